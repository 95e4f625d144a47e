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
    const uint32_t *mask;
    int words;
    // |scale| * log2(e), so that a masked score can be -inf before the scaling;
    // the sign goes to the queries (xor), a scale of zero clears them (and)
    float sl2;
    uint32_t qxor, qand;
    void *o;
    int o_f32;
    float *lse;
    float *part_o;   // [grid][2][rows][D]
    float *part_ml;  // [grid][2][rows][2]
    int grid, rows, unit;
    const uint16_t *kpool, *vpool;
    const float *acc_in;
    float *acc_out;
    float decay;
    int32_t *status;
};

__device__ __forceinline__ int row_blocks(const Seq &q, int G, int rows) {
    return (q.T * G + rows - 1) / rows;
}
__device__ __forceinline__ int key_units(const Seq &q, int unit) {
    return (q.ctx + q.T + unit - 1) / unit;
}

// All items' units before sequence `upto` (B: all of them). One thread of the
// block handles ceil(B / threads) sequences; sh: a long long per warp.
template <int kThreads>
__device__ long long units_before(const TreeArgs &a, int upto, long long *sh) {
    const int per = (a.s.B + kThreads - 1) / kThreads;
    long long n = 0;
    for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        if (b >= upto) break;
        bool ok;
        const Seq q = get_seq(a.s, b, ok);
        n += (long long)key_units(q, a.unit) * row_blocks(q, a.G, a.rows) * a.Hkv * (q.T > 0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) n += sh[w];
    return n;
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
    // To unit x of all (whose sequence exists).
    __device__ __forceinline__ void seek(const TreeArgs &a, long long x) {
        for (b = 0; b < a.s.B; ++b) {
            load(a);
            const long long n = q.T > 0 ? (long long)nu * nrb * a.Hkv : 0;
            if (x < n) break;
            x -= n;
        }
        const long long item = x / nu;
        u = (int)(x - item * nu);
        h = (int)(item / nrb);
        rb = (int)(item - (long long)h * nrb);
    }
};

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
