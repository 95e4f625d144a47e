// qmv_attn_plan.cuh - the arguments of the tree attention kernels, how the
// thread blocks share the work out, and which drafts a row sees.
#pragma once

#include "qmv_attn.cuh"
#include "qmv_attn.h"

namespace qmv {
namespace attn {

constexpr uint32_t kPoll = 1u << 22;  // polls of a copy's barrier before giving up

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
    long long u0, u1, rest;  // rest: u0's place among its sequence's units
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
template <int kThreads>
__device__ __forceinline__ Share find_share(const TreeArgs &a, ShareScratch<kThreads / 32> *sh) {
    if (a.s.B <= 32) {
        const int lane = threadIdx.x & 31;
        bool ok = false;
        Seq q;
        q.ctx = q.first = q.T = 0;
        if (lane < a.s.B) q = get_seq(a.s, lane, ok);
        const long long n =
            q.T > 0 ? (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv : 0;
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        const long long total = __shfl_sync(0xFFFFFFFFu, inc, 31), quota = (total + a.grid - 1) / a.grid;
        Share s;
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
        return q.T > 0 ? (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv : 0;
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
    const long long quota = (total + a.grid - 1) / a.grid;
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

// The place of a unit: sequence, head, row block, unit of the item's keys.
struct Cursor {
    int b, h, rb, u;
    int nu, nrb;
    Seq q;
    __device__ __forceinline__ void load(const TreeArgs &a) {
        bool ok;
        q = get_seq(a.s, b, ok);
        nu = key_units(q, a.unit);
        nrb = row_blocks(q, a.G, a.rows);
    }
    __device__ __forceinline__ void next_item(const TreeArgs &a) {
        u = 0;
        if (++rb < nrb) return;
        rb = 0;
        if (++h < a.Hkv) return;
        h = 0;
        do {
            ++b;
            if (b >= a.s.B) return;
            load(a);
        } while (q.T == 0);
    }
    __device__ __forceinline__ void start(const TreeArgs &a, const Share &s) {
        b = s.b;
        load(a);
        const int item = (int)(s.rest / nu);
        u = (int)(s.rest - (long long)item * nu);
        h = item / nrb;
        rb = item - h * nrb;
    }
};

// Element `col` (a multiple of 4) of row r of a block's first or last segment.
template <int D>
__device__ __forceinline__ float *part_at(const TreeArgs &a, int block, int last, int r, int col) {
    return a.part_o +
           (((long long)block * 2 + last) * (D / 4) + (col >> 2)) * (a.rows * 4LL) + r * 4;
}

// A pool as a tensor map (128 bytes, row, 128-byte chunk of a row), boxes of
// box_rows rows of one chunk, or of all (chunks), 128-byte swizzle.
bool encode_pool(CUtensorMap *map, const void *pool, const AttnCache &c, int box_rows, bool all_chunks);

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
