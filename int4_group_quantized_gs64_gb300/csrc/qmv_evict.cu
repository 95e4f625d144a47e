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
// each, largest bins first), then lists the kept slots in order. A cluster of
// blocks shares one list, each with its own stretch of slots; histograms and
// counts are read across the cluster. k_evict_copy moves the rows.
#include <cooperative_groups.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_launch.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace attn {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kBins = 2048;

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

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictArgs a) {
    __shared__ uint32_t hist[3][kBins];
    __shared__ uint32_t wsum[kSelWarps];
    __shared__ uint32_t found[2];       // bin, and how many are still wanted from it
    __shared__ uint32_t mine[2];        // this block's (kept outright, equal to the threshold)
    __shared__ uint32_t wcnt[kSelWarps][2];
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank();
    const int bh = blockIdx.x / C, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    for (int i = rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads)
        if (i >= kept || len <= a.budget) keep[i] = i < kept ? i : -1;
    if (len <= a.budget) return;  // the whole cluster

    const int lo = a.sink, hi = len - a.recent;
    uint32_t want = a.budget - a.sink - a.recent;  // of slots [lo, hi)
    // this block's stretch, a multiple of 32 slots a warp
    const int per = (((hi - lo + C * kSelWarps - 1) / (C * kSelWarps)) + 31) & ~31;
    const long long w0l = lo + (long long)(rank * kSelWarps + warp) * per;
    const int w0 = (int)min(w0l, (long long)hi), w1 = (int)min(w0l + per, (long long)hi);

    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0u;
    __syncthreads();
    uint32_t prefix = 0, mask = 0;  // the bits found so far
    for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : p == 1 ? 10 : 0, bits = p == 2 ? 10 : 11;
        for (int i = w0 + lane; i < w1; i += 32) {
            const uint32_t k = slot_key(a, row, h, i);
            if ((k & mask) == prefix) atomicAdd(&hist[p][(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        cl.sync();
        // bins from the top: thread t takes bins top - 4t .. top - 4t - 3
        constexpr int kPer = kBins / kSelThreads;
        uint32_t n[kPer], sum = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int bin = kBins - 1 - (tid * kPer + j);
            uint32_t s = 0;
            for (int r = 0; r < C; ++r) s += cl.map_shared_rank(&hist[p][0], r)[bin];
            n[j] = s;
            sum += s;
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        uint32_t before = inc - sum;
        for (int w = 0; w < warp; ++w) before += wsum[w];
        // the bin that holds the want-th largest (none when want is 0)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (before < want && before + n[j] >= want) {
                found[0] = kBins - 1 - (tid * kPer + j);
                found[1] = want - before;
            }
            before += n[j];
        }
        if (tid == 0 && want == 0) {  // nothing between: a threshold above every key
            found[0] = (1u << bits) - 1;
            found[1] = 0;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= ((1u << bits) - 1) << shift;
        want = found[1];
        __syncthreads();
    }
    // keys above `prefix` are kept, and the first `want` equal to it
    uint32_t above = 0, equal = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = slot_key(a, row, h, i);
        above += k > prefix;
        equal += k == prefix;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
        equal += __shfl_xor_sync(0xFFFFFFFFu, equal, o);
    }
    if (lane == 0) {
        wcnt[warp][0] = above;
        wcnt[warp][1] = equal;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t s = 0;
        for (int w = 0; w < kSelWarps; ++w) s += wcnt[w][tid];
        mine[tid] = s;
    }
    cl.sync();
    uint32_t pa = 0, pe = 0;  // kept outright / equal before this warp's stretch
    for (int r = 0; r < rank; ++r) {
        const uint32_t *m = cl.map_shared_rank(&mine[0], r);
        pa += m[0];
        pe += m[1];
    }
    for (int w = 0; w < warp; ++w) {
        pa += wcnt[w][0];
        pe += wcnt[w][1];
    }
    cl.sync();  // no block leaves while its counts are read
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? slot_key(a, row, h, i) : 0u;
        const uint32_t ba = __ballot_sync(0xFFFFFFFFu, i < w1 && k > prefix);
        const uint32_t be = __ballot_sync(0xFFFFFFFFu, i < w1 && k == prefix);
        const uint32_t below = (1u << lane) - 1;
        const uint32_t na = pa + __popc(ba & below), ne = pe + __popc(be & below);
        if (((ba >> lane) & 1u) || (((be >> lane) & 1u) && ne < want))
            keep[a.sink + na + min(ne, want)] = i;
        pa += __popc(ba);
        pe += __popc(be);
    }
    for (int i = rank * kSelThreads + tid; i < a.sink + a.recent; i += C * kSelThreads)
        keep[i < a.sink ? i : a.budget - a.recent + (i - a.sink)] =
            i < a.sink ? i : len - a.recent + (i - a.sink);
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
    // blocks a list: enough stretches of some thousand slots, while the lists
    // alone do not fill the GPU
    const long long longest = (long long)max_pages << a.lpage;
    int C = 1;
    while (C < 8 && longest / C > 8192 && (long long)B * src.Hkv * C < sm_count()) C *= 2;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * src.Hkv * C));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_select, a);
    if (e != cudaSuccess) return e;
    const int per = 256 / (src.D / 8) * 4;
    const dim3 grid((unsigned)((budget + per - 1) / per), (unsigned)(B * src.Hkv));
    return src.D == 64 ? launch(k_evict_copy<64>, grid, dim3(256), 0, st, true, a)
                       : launch(k_evict_copy<128>, grid, dim3(256), 0, st, true, a);
}

}  // namespace qmv
