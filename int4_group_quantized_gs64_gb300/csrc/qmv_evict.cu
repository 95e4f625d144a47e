// qmv_evict.cu - eviction from the cache by accumulated attention weight.
//
// Of a sequence's `len` tokens each key/value head keeps `budget`: the first
// `sink`, the last `recent`, and of those between the ones with the largest
// sums, equal sums keeping the lower slot (a NaN sum counts as the lowest, -0
// as +0). The kept tokens keep their order and are copied, with their sums,
// to fresh pages: source pages may be shared with other sequences, and a
// token keeps the rotation of its own position, so its slot may change.
//
// k_evict_select finds the smallest kept sum of a (sequence, head) by radix
// selection on order-preserving 32-bit keys (11, 11 and 10 bits, a histogram
// each, largest bins first), then lists the kept slots in order. The sums are
// read once: their keys stay in shared memory. A cluster of blocks shares a
// list, each with its own stretch of slots; histograms and counts are read
// across the cluster. k_evict_copy moves the rows.
#include <cooperative_groups.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_launch.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace attn {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32, kBins = 2048;
constexpr int kCachedMax = 50 * 1024;  // keys a block keeps in shared memory (200 KB)

struct EvictArgs {
    const float *acc;
    const int32_t *table, *lens;
    int B, Hkv, max_pages, page, lpage, pages;
    int budget, sink, recent;
    int32_t *keep, *new_lens;
    int32_t *status;
    // the copy
    const uint16_t *k, *v;
    uint16_t *dk, *dv;
    float *dacc;
    const int32_t *dst_table;
    int dst_max_pages, dst_pages, dpage, dlpage;
};

// Larger float, larger key; NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t sum_key(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t slot_key(const EvictArgs &a, const int32_t *row, int h, int i) {
    const int pid = __ldg(row + (i >> a.lpage));
    if ((unsigned)pid >= (unsigned)a.pages) return 0u;
    return sum_key(__ldg(a.acc + ((long long)pid * a.Hkv + h) * a.page + (i & (a.page - 1))));
}

struct SelSmem {
    uint32_t hist[3][kBins];
    uint32_t wsum[kSelWarps];
    uint32_t found[2];           // bin, and how many are still wanted from it
    uint32_t mine[2];            // this block's (above the threshold, equal to it)
    uint32_t wcnt[kSelWarps][2];
};

// Adds one to the lanes' bins; a warp whose lanes all have the same bin (many
// equal sums) adds once.
__device__ __forceinline__ void count_bin(uint32_t *hist, uint32_t bin, bool valid, int lane) {
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, valid);
    if (who == 0) return;
    const int first = __ffs(who) - 1;
    const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, bin, first);
    if (__all_sync(0xFFFFFFFFu, !valid || bin == b0)) {
        if (lane == first) atomicAdd(hist + b0, (uint32_t)__popc(who));
    } else if (valid) {
        atomicAdd(hist + bin, 1u);
    }
}

// cached: the keys of a block's stretch that its shared memory holds (all of
// them up to cached * blocks slots; the rest are read again where needed).
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictArgs a, int cached) {
    extern __shared__ __align__(16) uint8_t smem[];
    SelSmem *m = reinterpret_cast<SelSmem *>(smem);
    uint32_t *keys = reinterpret_cast<uint32_t *>(m + 1);
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank();
    const int bh = blockIdx.x / C, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&m->hist[0][0])[i] = 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int len = a.lens[b];
    const bool ok = len >= 0 && (long long)len <= ((long long)a.max_pages << a.lpage);
    if (!ok) {
        len = 0;
        if (tid == 0 && rank == 0) set_status(a.status, kStLength);
    }
    const int kept = min(len, a.budget);
    if (tid == 0 && rank == 0 && h == 0) a.new_lens[b] = kept;
    int32_t *keep = a.keep + (long long)bh * a.budget;
    const int32_t *row = a.table + (long long)b * a.max_pages;
    if (len <= a.budget) {  // the whole cluster
        for (int i = rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads)
            keep[i] = i < kept ? i : -1;
        return;
    }
    for (int i = rank * kSelThreads + tid; i < a.sink + a.recent; i += C * kSelThreads)
        keep[i < a.sink ? i : a.budget - a.recent + (i - a.sink)] =
            i < a.sink ? i : len - a.recent + (i - a.sink);

    const int lo = a.sink, hi = len - a.recent;
    uint32_t want = a.budget - a.sink - a.recent;  // of slots [lo, hi)
    // this warp's stretch [w0, w1), a multiple of 32 slots long; slot i's key is
    // keys[i - c0] while that is below `cached`
    const int per = (((hi - lo + C * kSelWarps - 1) / (C * kSelWarps)) + 31) & ~31;
    const int c0 = (int)min((long long)lo + (long long)rank * kSelWarps * per, (long long)hi);
    const int w0 = (int)min((long long)c0 + (long long)warp * per, (long long)hi);
    const int w1 = (int)min((long long)w0 + per, (long long)hi);
    auto key_at = [&](int i) {
        return i - c0 < cached ? keys[i - c0] : slot_key(a, row, h, i);
    };
    __syncthreads();

    // keys to shared memory, eight loads a lane under way, and the first histogram
    constexpr int kU = 8;
    for (int i0 = w0; i0 < w1; i0 += 32 * kU) {
        int pid[kU];
        float v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * 32 + lane;
            pid[u] = __ldg(row + (min(i, hi - 1) >> a.lpage));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = min(i0 + u * 32 + lane, hi - 1);
            const bool good = (unsigned)pid[u] < (unsigned)a.pages;
            v[u] = good ? __ldg(a.acc + ((long long)pid[u] * a.Hkv + h) * a.page + (i & (a.page - 1)))
                        : __int_as_float(0x7FC00000);  // no page: the lowest
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * 32 + lane;
            const uint32_t k = sum_key(v[u]);
            if (i < w1 && i - c0 < cached) keys[i - c0] = k;
            count_bin(m->hist[0], k >> 21, i < w1, lane);
        }
    }
    __syncwarp();
    uint32_t prefix = 0, mask = 0;  // the bits found so far
    for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : p == 1 ? 10 : 0, bits = p == 2 ? 10 : 11;
        if (p > 0)
            for (int i0 = w0; i0 < w1; i0 += 32) {
                const int i = i0 + lane;
                const uint32_t k = i < w1 ? key_at(i) : 0u;
                count_bin(m->hist[p], (k >> shift) & ((1u << bits) - 1), i < w1 && (k & mask) == prefix, lane);
            }
        cl.sync();
        // bins from the top: thread t takes the kPer below kBins - kPer * t
        constexpr int kPer = kBins / kSelThreads;
        static_assert(kPer == 4 || kPer == 2, "");
        const int bin0 = kBins - (tid + 1) * kPer;
        uint32_t n[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) n[j] = 0;
        for (int r = 0; r < C; ++r) {
            const uint32_t *hr = cl.map_shared_rank(&m->hist[p][0], r) + bin0;
            if (kPer == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(hr);
                n[kPer - 1] += x.x; n[kPer - 2] += x.y; n[1] += x.z; n[0] += x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(hr);
                n[1] += x.x; n[0] += x.y;
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += n[j];
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) m->wsum[warp] = inc;
        if (tid == 0) {  // wanted 0: a threshold above every key
            m->found[0] = (1u << bits) - 1;
            m->found[1] = 0;
        }
        __syncthreads();
        uint32_t before = inc - sum;
        for (int w = 0; w < warp; ++w) before += m->wsum[w];
        // the bin that holds the want-th largest
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (before < want && before + n[j] >= want) {
                m->found[0] = kBins - 1 - (tid * kPer + j);
                m->found[1] = want - before;
            }
            before += n[j];
        }
        __syncthreads();
        prefix |= m->found[0] << shift;
        mask |= ((1u << bits) - 1) << shift;
        want = m->found[1];
        __syncthreads();
    }
    // keys above `prefix` are kept, and the first `want` equal to it
    uint32_t above = 0, equal = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key_at(i);
        above += k > prefix;
        equal += k == prefix;
    }
    above = __reduce_add_sync(0xFFFFFFFFu, above);
    equal = __reduce_add_sync(0xFFFFFFFFu, equal);
    if (lane == 0) {
        m->wcnt[warp][0] = above;
        m->wcnt[warp][1] = equal;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t s = 0;
        for (int w = 0; w < kSelWarps; ++w) s += m->wcnt[w][tid];
        m->mine[tid] = s;
    }
    cl.sync();
    uint32_t pa = 0, pe = 0;  // above / equal before this warp's stretch
    for (int r = 0; r < rank; ++r) {
        const uint32_t *x = cl.map_shared_rank(&m->mine[0], r);
        pa += x[0];
        pe += x[1];
    }
    for (int w = 0; w < warp; ++w) {
        pa += m->wcnt[w][0];
        pe += m->wcnt[w][1];
    }
    if (C > 1) cl.sync();  // no block leaves while its counts are read
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? key_at(i) : 0u;
        const uint32_t ba = __ballot_sync(0xFFFFFFFFu, i < w1 && k > prefix);
        const uint32_t be = __ballot_sync(0xFFFFFFFFu, i < w1 && k == prefix);
        const uint32_t below = (1u << lane) - 1;
        const uint32_t na = pa + __popc(ba & below), ne = pe + __popc(be & below);
        if (((ba >> lane) & 1u) || (((be >> lane) & 1u) && ne < want))
            keep[a.sink + na + min(ne, want)] = i;
        pa += __popc(ba);
        pe += __popc(be);
    }
}

// Rows of kept tokens to their new places: D / 8 lanes a row, kRows rows in
// flight a lane group.
template <int D>
__global__ void __launch_bounds__(256) k_evict_copy(const EvictArgs a) {
    constexpr int kLanes = D / 8, kRows = 4, kGroups = 256 / kLanes;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int grp = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int i0 = (blockIdx.x * kGroups + grp) * kRows;
    if (i0 >= a.budget) return;
    const int32_t *keep = a.keep + (long long)bh * a.budget;
    long long src[kRows], dst[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        src[j] = dst[j] = -1;
        const int i = i0 + j, s = i < a.budget ? keep[i] : -1;
        if (s < 0) continue;
        const int pid = a.table[(long long)b * a.max_pages + (s >> a.lpage)];
        const int did = (long long)i < ((long long)a.dst_max_pages << a.dlpage)
                            ? a.dst_table[(long long)b * a.dst_max_pages + (i >> a.dlpage)]
                            : -1;
        if ((unsigned)pid >= (unsigned)a.pages || (unsigned)did >= (unsigned)a.dst_pages) {
            if (lane == 0) set_status(a.status, kStPage);
            continue;
        }
        src[j] = ((long long)pid * a.Hkv + h) * a.page + (s & (a.page - 1));
        dst[j] = ((long long)did * a.Hkv + h) * a.dpage + (i & (a.dpage - 1));
    }
    uint4 kv[kRows], vv[kRows];
    float w[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        if (src[j] >= 0) {
            kv[j] = __ldg(reinterpret_cast<const uint4 *>(a.k + src[j] * D) + lane);
            vv[j] = __ldg(reinterpret_cast<const uint4 *>(a.v + src[j] * D) + lane);
            if (lane == 0) w[j] = __ldg(a.acc + src[j]);
        }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        if (src[j] >= 0) {
            reinterpret_cast<uint4 *>(a.dk + dst[j] * D)[lane] = kv[j];
            reinterpret_cast<uint4 *>(a.dv + dst[j] * D)[lane] = vv[j];
            if (lane == 0) a.dacc[dst[j]] = w[j];
        }
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_evict(const AttnCache &src, const float *acc, const int32_t *table,
                              int max_pages, const int32_t *lens, int B, int budget, int sink,
                              int recent, const AttnCache &dst, float *dst_acc,
                              const int32_t *dst_table, int dst_max_pages, int32_t *keep,
                              int32_t *new_lens, int32_t *status, cudaStream_t st) {
    using namespace attn;
    auto log2of = [](int x) { int l = 0; while ((1 << l) < x) ++l; return l; };
    EvictArgs a;
    a.acc = acc; a.table = table; a.lens = lens;
    a.B = B; a.Hkv = src.Hkv; a.max_pages = max_pages; a.page = src.page; a.lpage = log2of(src.page);
    a.pages = src.pages;
    a.budget = budget; a.sink = sink; a.recent = recent;
    a.keep = keep; a.new_lens = new_lens; a.status = status;
    a.k = static_cast<const uint16_t *>(src.k); a.v = static_cast<const uint16_t *>(src.v);
    a.dk = static_cast<uint16_t *>(dst.k); a.dv = static_cast<uint16_t *>(dst.v);
    a.dacc = dst_acc; a.dst_table = dst_table;
    a.dst_max_pages = dst_max_pages; a.dst_pages = dst.pages;
    a.dpage = dst.page; a.dlpage = log2of(dst.page);
    // Blocks a list: while the lists alone do not fill the GPU, and a block has
    // some thousand slots (a cluster's barriers cost as much as reading those).
    const long long longest = (long long)max_pages << a.lpage;
    int C = 1;
    while (C < 8 && longest / C > 8192 && (long long)B * src.Hkv * C * 2 <= sm_count()) C *= 2;
    // as many of its keys as fit in shared memory
    const long long stretch = (longest + C - 1) / C + 32 * kSelWarps;
    const int cached = (int)(stretch < kCachedMax ? stretch : kCachedMax);
    const size_t smem = sizeof(SelSmem) + (size_t)cached * 4;
    cudaError_t e = set_smem(k_evict_select, smem);
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * src.Hkv * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_evict_select, a, cached);
    if (e != cudaSuccess) return e;
    const int per = 256 / (src.D / 8) * 4;
    const dim3 grid((unsigned)((budget + per - 1) / per), (unsigned)(B * src.Hkv));
    return src.D == 64 ? launch(k_evict_copy<64>, grid, dim3(256), 0, st, true, a)
                       : launch(k_evict_copy<128>, grid, dim3(256), 0, st, true, a);
}

}  // namespace qmv
