// qmv_attn_plan.cuh - the arguments of the attention kernels, how the thread
// blocks share the work out, and which keys a row sees.
//
// The kernels come in two forms (kWin): trees of drafts, whose rows see all
// cached keys and the drafts of a mask, and causal rows with a sliding window
// and a few first keys. In the second form the keys of an item (and their
// number) depend on its block of rows, and slots that none of its rows sees are
// not looked at, nor are their page ids.
#pragma once

#include "qmv_attn.cuh"
#include "qmv_attn.h"

namespace qmv {
namespace attn {

constexpr uint32_t kPoll = 1u << 22;  // polls of a copy's barrier before giving up

// A segment that is not its whole item: units [u0, u0 + n) of nu (n 0: none).
struct PartInfo {
    int b, h, rb, u0, n, nu, quota, pad;
};

struct TreeArgs {
    Seqs s;
    const uint16_t *q;
    long long q_stride;
    int Hq, Hkv, G, pages;
    uint32_t ginv;  // ceil(2^32 / G), for div_g (G > 1)
    const uint32_t *mask;
    int words;
    // |scale| * log2(e), so that a masked score can be -inf before the scaling;
    // the sign goes to the queries (xor), a scale of zero clears them (and)
    float sl2;
    uint32_t qxor, qand;
    void *o;
    int o_f32;
    float *lse;
    // segments' sums, [grid][2][D / 4][rows][4]: a thread a row or a lane group a
    // row, stores and loads fill their sectors
    float *part_o;
    float *part_ml;  // [grid][2][rows][2]
    int grid, rows, unit;
    const uint16_t *vpool;
    const float *acc_in;
    float *acc_out;
    float decay;
    float *stash;  // scores for the weights, [B][Hkv][16 keys][max_rows][16], or null
    int max_rows;
    int32_t *status;
    // kWin: a row at slot p sees j <= p with j > p - window or j < sinks
    int window, sinks;
    int lunit;       // unit = 1 << lunit
    int align;       // slots in a row that are copied together, a power of two
    // Rows come in tiles of whole tokens: tile x of a sequence holds the tokens from
    // x / hs * tb on, tb of them, and of their G query heads those from x % hs * hb
    // on, hb of them (all, unless G is above 128). An item is tpi tiles.
    int tb, hb, hs, tpi;
    uint32_t hinv;   // ceil(2^32 / hb)
    float flip;      // what scores are multiplied by before sl2: 1, or -1 or 0 for such a scale
    PartInfo *info;  // which items the segments in part_o belong to, [grid][2]
};

// r / G for a row r < 2^18 and G <= 1024: the rounding of ginv adds less than
// r * 2^10 / 2^32 < 1 / G.
__device__ __forceinline__ int div_g(const TreeArgs &a, int r) {
    return a.G == 1 ? r : (int)__umulhi((uint32_t)r, a.ginv);
}

__device__ __forceinline__ int row_blocks(const Seq &q, int G, int rows) {
    return (q.T * G + rows - 1) / rows;
}
__device__ __forceinline__ int key_units(const Seq &q, int unit) {
    return (q.ctx + q.T + unit - 1) / unit;
}

// kWin: a sequence's tiles of rows, and its items a head.
__device__ __forceinline__ int row_tiles(const TreeArgs &a, const Seq &q) {
    return (q.T + a.tb - 1) / a.tb * a.hs;
}
__device__ __forceinline__ int window_items(const TreeArgs &a, const Seq &q) {
    return (row_tiles(a, q) + a.tpi - 1) / a.tpi;
}
// Token and head (among the G) of row i < 128 of a tile; false: there is none.
__device__ __forceinline__ bool tile_row(const TreeArgs &a, const Seq &q, int tile, int i, int &t, int &g) {
    const int x = a.hb == 1 ? i : (int)__umulhi((uint32_t)i, a.hinv), k = tile / a.hs;
    t = k * a.tb + x;
    g = (tile - k * a.hs) * a.hb + i - x * a.hb;
    return x < a.tb && t < q.T && g < a.G;
}

__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// kWin: which of the 32 slots from `slot` on a row at slot p sees.
__device__ __forceinline__ uint32_t window_word(const TreeArgs &a, int p, int slot) {
    const int lo = max(0, p - a.window + 1);
    return bits_below(p + 1 - slot) & (~bits_below(lo - slot) | bits_below(a.sinks - slot));
}

// kWin: the keys of an item, those that some row of it sees: slots below a.sinks and
// slots [lo, p1]. Both stretches, to whole pieces of a.align slots, are put side by
// side (sp slots from 0 on, then those from sw on); units count along that row of
// places, so that a few first tokens cost a piece and not a unit.
struct Reach {
    int p0, p1, lo, sp, sw, nu;
    __device__ __forceinline__ void set(const TreeArgs &a, const Seq &q, int item) {
        const int x = item * a.tpi;
        if (a.hs == 1) {  // (no divisions: planning goes through all items)
            p0 = q.ctx + x * a.tb;
            p1 = q.ctx + min((x + a.tpi) * a.tb, q.T) - 1;
        } else {
            const int y = min(x + a.tpi, row_tiles(a, q)) - 1;
            p0 = q.ctx + x / a.hs * a.tb;
            p1 = q.ctx + min(y / a.hs * a.tb + a.tb, q.T) - 1;
        }
        lo = max(0, p0 - a.window + 1);
        sw = lo & -a.align;
        sp = (min(a.sinks, lo) + a.align - 1) & -a.align;
        if (sp >= sw) sp = sw = 0;  // one stretch
        nu = ((sp + p1 - sw) >> a.lunit) + 1;
    }
    __device__ __forceinline__ int slot(int place) const { return place < sp ? place : place - sp + sw; }
    __device__ __forceinline__ int place(int slot) const { return slot < sp ? slot : slot - sw + sp; }
    // Whether some row sees a slot of [s0, s1), and whether all rows see all of them.
    __device__ __forceinline__ bool some(const TreeArgs &a, int s0, int s1) const {
        return s0 <= p1 && (s1 > lo || s0 < a.sinks);
    }
    __device__ __forceinline__ bool all(const TreeArgs &a, int s0, int s1) const {
        return s1 - 1 <= p0 && (s0 > p1 - a.window || s1 <= a.sinks);
    }
    // Whether all rows see n places from `at` on (both stretches: no, to be looked at).
    __device__ __forceinline__ bool all_at(const TreeArgs &a, int at, int n) const {
        return (at >= sp || at + n <= sp) && all(a, slot(at), slot(at) + n);
    }
    // Which of 32 places from `at` on (a multiple of 16) a row at slot p sees.
    __device__ __forceinline__ uint32_t word(const TreeArgs &a, int p, int at) const {
        return (window_word(a, p, slot(at)) & 0xFFFFu) | window_word(a, p, slot(at + 16)) << 16;
    }
};

// kWin: the units of one head of a sequence. A thread adds up the items `from`,
// `from` + step, ...
__device__ __forceinline__ long long window_units(const TreeArgs &a, const Seq &q, int from, int step) {
    long long n = 0;
    const int nrb = window_items(a, q);
#pragma unroll 1
    for (int rb = from; rb < nrb; rb += step) {
        Reach r;
        r.set(a, q, rb);
        n += r.nu;
    }
    return n;
}
// Items that a thread adds up by itself for every sequence that a warp would else add up
// together: some 40 cycles each, against 600 a sequence.
constexpr int kAlone = 16;

// All units of a sequence, by one thread.
template <bool kWin>
__device__ __forceinline__ long long seq_units(const TreeArgs &a, const Seq &q) {
    if (q.T <= 0) return 0;
    if (kWin) return window_units(a, q, 0, 1) * a.Hkv;
    return (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv;
}
// A lane's sequence each; the whole warp helps with long ones where they are few.
template <bool kWin>
__device__ __forceinline__ long long lane_units(const TreeArgs &a, const Seq &q) {
    if (!kWin) return seq_units<false>(a, q);
    const int items = q.T > 0 ? window_items(a, q) : 0;
    const int several = __popc(__ballot_sync(0xFFFFFFFFu, items > kAlone / 4));
    const bool big = items > kAlone * max(several, 1);
    long long n = big ? 0 : seq_units<true>(a, q);
    for (uint32_t who = __ballot_sync(0xFFFFFFFFu, big); who; who &= who - 1) {
        const int from = __ffs(who) - 1, lane = threadIdx.x & 31;
        Seq o;
        o.ctx = __shfl_sync(0xFFFFFFFFu, q.ctx, from);
        o.first = 0;
        o.T = __shfl_sync(0xFFFFFFFFu, q.T, from);
        long long x = window_units(a, o, lane, 32);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, k);
        if (lane == from) n = x * a.Hkv;
    }
    return n;
}

// All items' units, and those before sequence `upto`. A thread of the block
// handles ceil(B / threads) sequences (up to 32 of them: each warp for itself);
// sh: two long longs a warp.
template <int kThreads>
__device__ __forceinline__ long long count_units(const TreeArgs &a, int upto, long long *sh,
                                                 long long &before) {
    if (a.s.B <= 32) {
        const int lane = threadIdx.x & 31;
        bool ok = false;
        Seq q;
        q.ctx = q.first = q.T = 0;
        if (lane < a.s.B) q = get_seq(a.s, lane, ok);
        long long n = q.T > 0 ? (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv : 0;
        before = lane < upto ? n : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
            before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        }
        return n;
    }
    const int per = (a.s.B + kThreads - 1) / kThreads;
    long long n = 0, nb = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= a.s.B) break;
        bool ok;
        const Seq q = get_seq(a.s, b, ok);
        const long long x =
            q.T > 0 ? (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv : 0;
        n += x;
        if (b < upto) nb += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        nb += __shfl_xor_sync(0xFFFFFFFFu, nb, o);
    }
    if ((threadIdx.x & 31) == 0) {
        sh[threadIdx.x >> 5] = n;
        sh[kThreads / 32 + (threadIdx.x >> 5)] = nb;
    }
    __syncthreads();
    n = 0;
    before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        n += sh[w];
        before += sh[kThreads / 32 + w];
    }
    return n;
}

// This block's share [u0, u1) of all units, and where it starts.
struct Share {
    long long u0, u1, rest, quota;  // rest: u0's place among its sequence's units
    int padded;  // > 0: an item's units, filled up to whole quotas
    int b;
};
template <int kWarps>
struct ShareScratch {
    long long sums[kWarps];
    long long rest;
    int b;
};

// Each thread of the block counts ceil(B / threads) sequences in a row; the
// one whose units hold u0 says where they start. Up to 32 sequences each warp
// counts for itself, which saves two barriers.
template <int kThreads, bool kWin = false>
__device__ __forceinline__ Share find_share(const TreeArgs &a, ShareScratch<kThreads / 32> *sh) {
    if (a.s.B <= 32) {
        const int lane = threadIdx.x & 31;
        bool ok = false;
        Seq q;
        q.ctx = q.first = q.T = 0;
        if (lane < a.s.B) q = get_seq(a.s, lane, ok);
        if (kWin && a.tpi == 1 && a.hs == 1 && a.tb >= a.s.N) {
            // One item a head and sequence. A block whose share ends one item and
            // begins another has two segments to finish, which costs it more than
            // another unit: if whole blocks an item take at most one unit more than
            // even shares, each item gets whole blocks (one token over 4100 keys, 8
            // items of 65 units for 304 blocks: 18.3 us with shares of 2 units across
            // items, 14.9 without).
            uint32_t nu = 0;
            if (q.T > 0) {
                Reach r;
                r.set(a, q, 0);
                nu = r.nu;
            }
            const uint32_t items = __reduce_add_sync(0xFFFFFFFFu, q.T > 0 ? 1u : 0u) * a.Hkv;
            const long long all = (long long)__reduce_add_sync(0xFFFFFFFFu, nu) * a.Hkv;
            const uint32_t grid = a.grid;
            if (items > 0 && items < grid && all < 1 << 30) {
                const uint32_t even = ((uint32_t)all + grid - 1) / grid;
                const uint32_t whole = ((uint32_t)all + grid - items - 1) / (grid - items);
                if (whole <= even + 1) {
                    const uint32_t blocks = (nu + whole - 1) / whole;  // an item
                    uint32_t inc = blocks * a.Hkv;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                        if (lane >= o) inc += v;
                    }
                    const uint32_t who = __ballot_sync(0xFFFFFFFFu, inc > blockIdx.x);
                    Share s;
                    s.quota = whole;
                    s.b = who ? __ffs(who) - 1 : 0;
                    const uint32_t per = __shfl_sync(0xFFFFFFFFu, blocks, s.b);
                    const uint32_t units = __shfl_sync(0xFFFFFFFFu, nu, s.b);
                    // among the sequence's blocks
                    const uint32_t at = blockIdx.x - (__shfl_sync(0xFFFFFFFFu, inc, s.b) - per * a.Hkv);
                    s.padded = (int)(per * whole);
                    s.rest = s.u0 = at * whole;
                    s.u1 = who ? s.u0 + min(whole, units - at % per * whole) : s.u0;
                    return s;
                }
            }
        }
        const long long n = lane_units<kWin>(a, q);
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        const long long total = __shfl_sync(0xFFFFFFFFu, inc, 31), quota = (total + a.grid - 1) / a.grid;
        Share s;
        s.padded = 0;
        s.quota = quota;
        s.u0 = quota * blockIdx.x;
        s.u1 = min(s.u0 + quota, total);
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, inc > s.u0);
        s.b = who ? __ffs(who) - 1 : 0;
        s.rest = s.u0 - __shfl_sync(0xFFFFFFFFu, inc - n, s.b);
        return s;
    }
    const int per = (a.s.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto units = [&](int b) -> long long {
        bool ok;
        const Seq q = get_seq(a.s, b, ok);
        return seq_units<kWin>(a, q);
    };
    long long n = 0;
#pragma unroll 1
    for (int i = 0; i < per && b0 + i < a.s.B; ++i) n += units(b0 + i);
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sh->sums[warp] = inc;
    __syncthreads();
    long long total = 0, before = inc - n;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh->sums[w];
        total += sh->sums[w];
    }
    Share s;
    s.padded = 0;
    const long long quota = (total + a.grid - 1) / a.grid;
    s.quota = quota;
    s.u0 = quota * blockIdx.x;
    s.u1 = min(s.u0 + quota, total);
    if (s.u0 < s.u1 && before <= s.u0 && s.u0 < before + n) {
#pragma unroll 1
        for (int i = 0;; ++i) {
            const long long v = units(b0 + i);
            if (s.u0 < before + v) {
                sh->b = b0 + i;
                sh->rest = s.u0 - before;
                break;
            }
            before += v;
        }
    }
    __syncthreads();
    s.b = sh->b;
    s.rest = sh->rest;
    return s;
}

// kWin: shares that 31 bits do not count. The launcher refuses them; only sequences that
// overlap (cu not ascending) add up to more than it knows of. Whole grid.
__device__ __forceinline__ bool too_long(const TreeArgs &a, const Share &s) {
    if (s.quota <= 0x7FFFFFFFLL) return false;
    if (threadIdx.x == 0) set_status(a.status, kStLength);
    return true;
}

// The place of a unit: sequence, head, row block (item), unit of the item's keys.
template <bool kWin>
struct CursorOf {
    int b, h, rb, u;
    int nu, nrb;
    Seq q;
    Reach r;  // kWin
    __device__ __forceinline__ void load(const TreeArgs &a) {
        bool ok;
        q = get_seq(a.s, b, ok);
        nrb = kWin ? window_items(a, q) : row_blocks(q, a.G, a.rows);
        if (!kWin) nu = key_units(q, a.unit);
    }
    __device__ __forceinline__ void reach(const TreeArgs &a) {
        if (kWin) {
            r.set(a, q, rb);
            nu = r.nu;
        }
    }
    // The slot at a place among the item's keys.
    __device__ __forceinline__ int slot(int place) const { return kWin ? r.slot(place) : place; }
    // Whether some row of the item may see a slot of [s0, s1).
    __device__ __forceinline__ bool some(const TreeArgs &a, int s0, int s1) const {
        return kWin ? r.some(a, s0, s1) : s0 < q.ctx + q.T;
    }
    __device__ __forceinline__ void next_item(const TreeArgs &a) {
        u = 0;
        if (++rb < nrb) return reach(a);
        rb = 0;
        if (++h < a.Hkv) return reach(a);
        h = 0;
        do {
            ++b;
            if (b >= a.s.B) return;
            load(a);
        } while (q.T == 0);
        reach(a);
    }
    __device__ __forceinline__ void start(const TreeArgs &a, const Share &s) {
        b = s.b;
        load(a);
        if (kWin) return start_window(a, s.rest, s.padded);
        const int item = (int)(s.rest / nu);
        u = (int)(s.rest - (long long)item * nu);
        h = item / nrb;
        rb = item - h * nrb;
    }
    // kWin, whole warp: the head from the units of one, then its block of rows, 32 at a time.
    __device__ __forceinline__ void start_window(const TreeArgs &a, long long rest, int padded) {
        const int lane = threadIdx.x & 31;
        if (nrb == 1) {
            rb = 0;
            reach(a);
            const int n = padded ? padded : nu;
            h = (int)(rest / n);
            u = (int)(rest - (long long)h * n);
            return;
        }
        long long n = window_units(a, q, lane, 32);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, k);
        h = (int)(rest / n);
        rest -= h * n;
#pragma unroll 1
        for (rb = 0;; rb += 32) {
            Reach x;
            x.nu = 0;
            if (rb + lane < nrb) x.set(a, q, rb + lane);
            int inc = x.nu;
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, k);
                if (lane >= k) inc += v;
            }
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, inc > rest);
            if (who || rb + 32 >= nrb) {
                const int l = who ? __ffs(who) - 1 : 0;
                rest -= __shfl_sync(0xFFFFFFFFu, inc - x.nu, l);
                rb += l;
                break;
            }
            rest -= __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        u = (int)rest;
        reach(a);
    }
};
using Cursor = CursorOf<false>;

// Element `col` (a multiple of 4) of row r of a block's first or last segment.
template <int D>
__device__ __forceinline__ float *part_at(const TreeArgs &a, int block, int last, int r, int col) {
    return a.part_o +
           (((long long)block * 2 + last) * (D / 4) + (col >> 2)) * (a.rows * 4LL) + r * 4;
}

// A pool as a tensor map (128 bytes, row, 128-byte chunk of a row), boxes of
// box_rows rows of one chunk, or of all (chunks), 128-byte swizzle.
bool encode_pool(CUtensorMap *map, const void *pool, const AttnCache &c, int box_rows, bool all_chunks);

// Queries as a tensor map (128 bytes, head, token, 128-byte chunk of a head), boxes
// of some heads of some tokens, one chunk, 128-byte swizzle.
bool encode_heads(CUtensorMap *map, const void *q, int N, int Hq, int D, long long q_stride, int heads,
                  int tokens);

// The scores of 16 keys from `slot` (a multiple of 16): [max_rows][16].
__device__ __forceinline__ float *stash_at(const TreeArgs &a, int b, int h, int slot) {
    const long long slices = ((long long)a.s.max_pages << a.s.lpage) >> 4;
    return a.stash + (((long long)b * a.Hkv + h) * slices + (slot >> 4)) * (a.max_rows * 16LL);
}

// The attention weights, once every row's lse is there (qmv_attn_weights.cu).
cudaError_t launch_tree_weights(const AttnCache &c, const TreeArgs &a, int max_rows,
                                cudaStream_t st);

// Launches the tcgen05 kernel (qmv_attn_tc.cu) for a.rows = 128 or 256.
cudaError_t launch_tree_tc(const AttnCache &c, const TreeArgs &a, cudaStream_t st);

// Which of the 32 slots from `slot` on a row of draft t sees, as bits: all
// before ctx, drafts by the mask (or the chain), nothing past the end.
__device__ __forceinline__ uint32_t seen_word(const TreeArgs &a, const Seq &q, int t, int slot) {
    const int d = slot - q.ctx;
    if (d <= -32) return 0xFFFFFFFFu;
    const uint32_t *m = a.mask ? a.mask + (long long)(q.first + t) * a.words : nullptr;
    auto word = [&](int i) -> uint32_t {  // drafts 32 i .. 32 i + 31
        if (i < 0) return 0xFFFFFFFFu;
        const int n = (m ? q.T : t + 1) - 32 * i;  // how many of them there are (chain: 0 .. t)
        if (n <= 0) return 0u;
        const uint32_t w = m ? __ldg(m + i) : 0xFFFFFFFFu;
        return n >= 32 ? w : w & ((1u << n) - 1);
    };
    const int i = d >> 5;  // floor
    return __funnelshift_r(word(i), (d & 31) ? word(i + 1) : 0u, d & 31);
}

}  // namespace attn
}  // namespace qmv
