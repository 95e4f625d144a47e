// qmv_evict.cu - eviction from the cache by accumulated attention weight.
//
// Of a sequence's `len` tokens each key/value head keeps `budget`: the first
// `sink`, the last `recent`, and of those between the ones with the largest
// sums, equal sums keeping the lower slot (a NaN sum counts as the lowest, -0
// as +0). The kept tokens keep their order and are copied, with their sums,
// to fresh pages: the source stays as it is (other sequences may read its pages),
// and a token keeps the rotation of its own position, so its slot may change.
//
// k_evict_select finds the smallest kept sum of a (sequence, head) by radix
// selection on order-preserving 32-bit keys (11, 11 and 10 bits, a histogram
// each, largest bins first), then lists the kept slots in order. The sums are
// read once, four slots a load; the upper halves of their keys stay in shared
// memory, eight of which a lane looks at together. After the first histogram a
// pass lists the few slots that share the threshold's bin, and only those are
// looked at whole for the other bits (all of the bin's again where too many
// share it). A cluster of blocks shares a list, each with its own stretch of
// slots; sums of 32 bins, and then one such group, are read across the cluster.
// Half a key a slot lets two blocks share an SM: with whole keys 16 clusters of
// 8 ran in two waves.
//
// What bounds it: the latencies of its steps. 16 lists of 300,007 sums (19 MB)
// take 33 us of which reading and counting 11, the pass that lists 8 and the one
// that writes 7; 4,099 sums take 8 us in one block a list, 2 of them the first
// sums' way from memory. k_evict_copy moves the rows, 16 bytes a lane and four
// rows in flight: 82 us for the 549 MB of a batch of 16 with 4096 kept a head,
// which is the rate of a plain copy.
#include <cooperative_groups.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_launch.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace attn {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kBins = 2048;
constexpr uint32_t kCand = 160;         // listed slots a warp
constexpr int kCached = 39552;          // slots a block keeps 16 key bits of (77 KB)

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
    if ((unsigned)pid >= (unsigned)a.pages) return 0u;  // no page: the lowest
    return sum_key(__ldg(a.acc + ((long long)pid * a.Hkv + h) * a.page + (i & (a.page - 1))));
}

struct alignas(16) SelSmem {  // (the key halves after it are read 16 bytes at a time)
    uint32_t hist[3][kBins];
    uint32_t group[3][kBins / 32];  // sums of 32 bins
    uint32_t found[2];           // bin, and how many are still wanted from it
    uint32_t mine[2];            // this block's (above the threshold, equal to it)
    uint32_t wcnt[2][32];        // the same of each warp
    // slots whose key shares the threshold's first bits, each warp its own, while
    // they fit
    int32_t cand[kSelWarps][kCand];
};

static_assert(sizeof(SelSmem) % 16 == 0, "");
static_assert(sizeof(SelSmem) + kCached * 2 <= 113 * 1024, "two blocks an SM");

// Inclusive sum over a warp's lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// cached: the slots (a multiple of 8) of a block's stretch whose upper 16 key
// bits its shared memory holds; beyond them the sums are read again.
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictArgs a, int cached) {
    extern __shared__ __align__(16) uint8_t smem[];
    SelSmem *m = reinterpret_cast<SelSmem *>(smem);
    uint16_t *upper = reinterpret_cast<uint16_t *>(m + 1);
    cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank();
    const int bh = blockIdx.x / C, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&m->hist[0][0])[i] = 0u;
    if (tid < 64) m->wcnt[tid >> 5][tid & 31] = 0u;
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
    // this warp's stretch [w0, w1): `per` slots from a multiple of 128 on; the
    // block's starts at c0
    const int base = lo & ~127;
    const int per = (((hi - base + C * kSelWarps - 1) / (C * kSelWarps)) + 127) & ~127;
    const int end = base + ((hi - base + 127) & ~127);
    const int c0 = (int)min((long long)base + (long long)rank * kSelWarps * per, (long long)end);
    const int w0 = (int)min((long long)c0 + (long long)warp * per, (long long)end);
    const int w1 = (int)min((long long)w0 + per, (long long)end);
    auto pack16 = [](const uint4 &k) {
        return make_uint2(__byte_perm(k.x, k.y, 0x7632), __byte_perm(k.z, k.w, 0x7632));
    };
    __syncthreads();

    // The sums, kU groups of four slots a lane a round (loads a round ahead, their
    // page ids two): upper halves of the keys to shared memory, and the histogram of
    // the first 11 bits. Sums share bins, so the lanes spread over the three
    // histograms, and a warp whose slots all have the same bin (many equal sums)
    // adds once.
    constexpr int kU = 4;
    float4 v[2][kU];
    int pid[kU];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
            pid[u] = __ldg(row + (min(i0 + u * 128 + lane * 4, hi - 1) >> a.lpage));
    };
    auto load = [&](int i0, float4 (&d)[kU]) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * 128 + lane * 4;
            const float no = __int_as_float(0x7FC00000);  // no page: the lowest
            d[u] = make_float4(no, no, no, no);
            if (i < min(w1, hi) && (unsigned)pid[u] < (unsigned)a.pages)
                d[u] = __ldg(reinterpret_cast<const float4 *>(
                    a.acc + ((long long)pid[u] * a.Hkv + h) * a.page + (i & (a.page - 1))));
        }
    };
    uint32_t *h0 = m->hist[lane % 3];
    auto count = [&](int i0, const float4 (&d)[kU]) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (i0 + u * 128 >= w1) break;
            const int i = i0 + u * 128 + lane * 4;
            const uint4 k = make_uint4(sum_key(d[u].x), sum_key(d[u].y), sum_key(d[u].z), sum_key(d[u].w));
            if (i - c0 < cached) *reinterpret_cast<uint2 *>(upper + (i - c0)) = pack16(k);
            const uint32_t x[4] = {k.x >> 21, k.y >> 21, k.z >> 21, k.w >> 21};
            const uint32_t b0 = __shfl_sync(0xFFFFFFFFu, x[0], 0);
            const bool all_in = i >= lo && i + 4 <= hi;
            if (__all_sync(0xFFFFFFFFu, all_in && x[0] == b0 && x[1] == b0 && x[2] == b0 && x[3] == b0)) {
                if (lane == 0) atomicAdd(&m->hist[0][b0], 128u);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (all_in || (i + e >= lo && i + e < hi)) atomicAdd(h0 + x[e], 1u);
            }
        }
    };
    constexpr int kRound = 128 * kU;
    if (w0 < w1) {
        fetch(w0);
        load(w0, v[0]);
        if (w0 + kRound < w1) fetch(w0 + kRound);
    }
    for (int i0 = w0; i0 < w1; i0 += 2 * kRound) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int i = i0 + s * kRound;
            if (i >= w1) break;
            if (i + kRound < w1) load(i + kRound, v[s ^ 1]);
            if (i + 2 * kRound < w1) fetch(i + 2 * kRound);
            count(i, v[s]);
        }
    }
    __syncthreads();
    // Sums of 32 bins, eight threads' n each.
    auto group_sum = [&](int p, const uint4 &n) {
        uint32_t x = n.x + n.y + n.z + n.w;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        if ((lane & 7) == 0) m->group[p][tid >> 3] = x;
    };
    static_assert(kBins == 4 * kSelThreads, "");
    {
        uint4 *s0 = reinterpret_cast<uint4 *>(m->hist[0]) + tid, *s1 = reinterpret_cast<uint4 *>(m->hist[1]) + tid,
              *s2 = reinterpret_cast<uint4 *>(m->hist[2]) + tid;
        const uint4 x = *s0, y = *s1, z = *s2;
        const uint4 n = make_uint4(x.x + y.x + z.x, x.y + y.y + z.y, x.z + y.z + z.z, x.w + y.w + z.w);
        *s0 = n;
        *s1 = *s2 = make_uint4(0u, 0u, 0u, 0u);
        group_sum(0, n);
    }
    // Which of eight slots from i are inside and have upper halves in [from, to) (eq)
    // or from `to` on (above), bit e for slot i + e; where the halves are not kept,
    // f(slot) says it: 1, 2, or 0.
    auto classes = [&](int i, uint32_t from, uint32_t to, uint32_t &above, uint32_t &eq, auto &&f) {
        above = eq = 0;
        if (i >= w1) return;
        if (i - c0 + 8 <= cached) {
            const uint4 x = *reinterpret_cast<const uint4 *>(upper + (i - c0));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w}, f = from << 16, t = to << 16;
            uint32_t some = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // the half in the upper 16 bits (an odd slot's with its neighbour's below)
                const uint32_t v = e & 1 ? w[e >> 1] : w[e >> 1] << 16;
                if (v >= f) some |= 1u << e;
                if (v >= t) above |= 1u << e;
            }
            if (to > 0xFFFFu) above = 0;
            eq = some & ~above;
        } else {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const int c = i + e >= lo && i + e < hi ? f(i + e) : 0;
                if (c == 1) eq |= 1u << e;
                if (c == 2) above |= 1u << e;
            }
        }
        if (i < lo || i + 8 > hi) {
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e >= lo && i + e < hi) in |= 1u << e;
            above &= in;
            eq &= in;
        }
    };
    uint32_t prefix = 0;  // the bits found so far
    // The slots that share the threshold's first bits, where they are listed: this
    // lane's, with their whole keys.
    bool listed = false;
    constexpr int kMine = kCand / 32;
    int cslot[kMine];
    uint32_t ckey[kMine];
    // Their whole keys: f(slot, key).
    auto candidates = [&](auto &&f) {
        __syncwarp();
        if (listed) {
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                if (cslot[j] >= 0) f(cslot[j], ckey[j]);
        } else {
            const uint32_t t = prefix >> 21;
            for (int i = w0 + lane * 8; i < w1; i += 256) {
                uint32_t above, eq;
                classes(i, t << 5, (t + 1) << 5, above, eq, [&](int s) { return slot_key(a, row, h, s) >> 21 == t; });
                for (; eq; eq &= eq - 1) {
                    const int s = i + __ffs(eq) - 1;
                    f(s, slot_key(a, row, h, s));
                }
            }
        }
    };
    for (int p = 0; p < 3; ++p) {
        const int shift = p == 0 ? 21 : p == 1 ? 10 : 0, bits = p == 2 ? 10 : 11;
        if (p > 0) {
            candidates([&](int, uint32_t k) {
                if (k >> (shift + bits) == prefix >> (shift + bits))
                    atomicAdd(&m->hist[p][(k >> shift) & ((1u << bits) - 1)], 1u);
            });
            __syncthreads();
            group_sum(p, *(reinterpret_cast<const uint4 *>(m->hist[p]) + tid));
        }
        if (C > 1)
            cl.sync();
        else
            __syncthreads();
        // the bin that holds the want-th largest: its group of 32 first (a block
        // that read all the others' bins took 5,000 to 9,000 cycles a histogram)
        if (warp == 0) {
            uint32_t bin = (1u << bits) - 1, left = 0;  // wanted 0: a threshold above every key
            if (want > 0) {
                uint2 n = make_uint2(0u, 0u);  // groups from the top, two a lane
#pragma unroll 8
                for (int r = 0; r < C; ++r) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(cl.map_shared_rank(&m->group[p][0], r) + 62 - 2 * lane);
                    n.x += x.x;
                    n.y += x.y;
                }
                uint32_t before = warp_scan(n.x + n.y, lane) - n.x - n.y;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, before + n.x + n.y >= want);
                const int src = __ffs(who) - 1;
                const bool second = before + n.y < want;
                const int grp = __shfl_sync(0xFFFFFFFFu, 63 - 2 * lane - (second ? 1 : 0), src);
                left = want - __shfl_sync(0xFFFFFFFFu, before + (second ? n.y : 0u), src);
                uint32_t c = 0;
#pragma unroll 8
                for (int r = 0; r < C; ++r)
                    c += cl.map_shared_rank(&m->hist[p][0], r)[grp * 32 + 31 - lane];
                const uint32_t inc = warp_scan(c, lane);
                const int at = __ffs(__ballot_sync(0xFFFFFFFFu, inc >= left)) - 1;
                left -= __shfl_sync(0xFFFFFFFFu, inc - c, at);
                bin = grp * 32 + 31 - at;
            }
            if (lane == 0) {
                m->found[0] = bin;
                m->found[1] = left;
            }
        }
        __syncthreads();
        prefix |= m->found[0] << shift;
        want = m->found[1];
        if (p == 0) {
            // each warp's keys above this bin, and a list of the slots in it
            uint32_t above = 0, n = 0;
            const uint32_t t = prefix >> 21;
            for (int i0 = w0; i0 < w1; i0 += 256) {
                uint32_t ab, eq;
                const int i = i0 + lane * 8;
                classes(i, t << 5, (t + 1) << 5, ab, eq, [&](int s) {
                    const uint32_t x = slot_key(a, row, h, s) >> 21;
                    return x > t ? 2 : x == t;
                });
                above += __popc(ab);
                if (__any_sync(0xFFFFFFFFu, eq != 0)) {
                    const uint32_t mine = __popc(eq), inc = warp_scan(mine, lane);
                    uint32_t at = n + inc - mine;
                    for (; eq; eq &= eq - 1, ++at)
                        if (at < kCand) m->cand[warp][at] = i + __ffs(eq) - 1;
                    n += __shfl_sync(0xFFFFFFFFu, inc, 31);
                }
            }
            above = __reduce_add_sync(0xFFFFFFFFu, above);
            if (lane == 0) m->wcnt[0][warp] = above;
            listed = __syncthreads_and(n <= kCand);
            if (listed) {
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const bool have = lane + j * 32 < n;
                    cslot[j] = have ? m->cand[warp][lane + j * 32] : -1;
                    ckey[j] = have ? slot_key(a, row, h, cslot[j]) : 0u;
                }
            }
        }
    }
    // keys above `prefix` are kept, and the first `want` equal to it: both in
    // each warp's stretch
    candidates([&](int s, uint32_t k) {
        const int w = (s - c0) / per;
        if (k > prefix) atomicAdd(&m->wcnt[0][w], 1u);
        if (k == prefix) atomicAdd(&m->wcnt[1][w], 1u);
        // its upper half, where that alone does not decide, moves to the right side
        if (k >> 16 == prefix >> 16 && k != prefix && s - c0 < cached)
            upper[s - c0] = (uint16_t)((k >> 16) + (k > prefix ? 1 : -1));
    });
    __syncthreads();
    const uint32_t wa = lane < kSelWarps ? m->wcnt[0][lane] : 0u, we = lane < kSelWarps ? m->wcnt[1][lane] : 0u;
    uint32_t pa = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wa : 0u);  // before this warp's stretch
    uint32_t pe = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? we : 0u);
    if (C > 1) {
        if (warp == 0) {
            const uint32_t ta = __reduce_add_sync(0xFFFFFFFFu, wa), te = __reduce_add_sync(0xFFFFFFFFu, we);
            if (lane == 0) {
                m->mine[0] = ta;
                m->mine[1] = te;
            }
        }
        cl.sync();
        uint32_t ra = 0, re = 0;
        if (lane < rank) {
            const uint32_t *x = cl.map_shared_rank(&m->mine[0], lane);
            ra = x[0];
            re = x[1];
        }
        pa += __reduce_add_sync(0xFFFFFFFFu, ra);
        pe += __reduce_add_sync(0xFFFFFFFFu, re);
        cl.sync();  // no block leaves while its counts are read
    }
    const uint32_t t16 = prefix >> 16;
    keep += a.sink;
    for (int i0 = w0; i0 < w1; i0 += 256) {
        uint32_t ab, eq;
        const int i = i0 + lane * 8;
        classes(i, t16, t16 + 1, ab, eq, [&](int s) {  // (not kept: the whole key decides)
            const uint32_t k = slot_key(a, row, h, s);
            return k > prefix ? 2 : k == prefix;
        });
        if (__any_sync(0xFFFFFFFFu, (ab | eq) != 0)) {
            const uint32_t mine = __popc(ab) | __popc(eq) << 16, inc = warp_scan(mine, lane);
            uint32_t na = pa + ((inc - mine) & 0xFFFFu), ne = pe + ((inc - mine) >> 16);
            for (uint32_t some = ab | eq; some; some &= some - 1) {
                const int e = __ffs(some) - 1;
                const bool tie = (eq >> e) & 1u;
                if (!tie || ne < want) keep[na + min(ne, want)] = i + e;
                na += !tie;
                ne += tie;
            }
            const uint32_t all = __shfl_sync(0xFFFFFFFFu, inc, 31);
            pa += all & 0xFFFFu;
            pe += all >> 16;
        }
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
    // some thousand slots, since a cluster's barriers cost as much as reading those
    // (4,099 slots in one block 12.3 us, in two 16.4; 65,536 in 8 blocks 20.5 us, in
    // 16 23.2; 16 lists of 300,007 in 16 blocks each 88 us, in 4 156).
    const long long longest = (long long)max_pages << a.lpage;
    int C = 1;
    while (C < 16 && longest / C > 8192 && (long long)B * src.Hkv * C <= sm_count()) C *= 2;
    // the upper halves of a block's keys, as many as leave room for two blocks an SM
    const long long stretch = (longest + C - 1) / C + 128 * kSelWarps + 128;
    const int cached = (int)(stretch < kCached ? stretch : kCached) & ~7;
    const size_t smem = sizeof(SelSmem) + (size_t)cached * 2;
    cudaError_t e = set_smem(k_evict_select, smem);
    if (e == cudaSuccess && C > 8)  // more than the portable size
        e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
