// qmv_attn_tree.cu - attention of drafted tokens over a paged cache.
//
// For sequence b with ctx cached tokens and T drafted ones, the rows of
// key/value head h are the T * G pairs (draft t, query head h * G + g),
// G = Hq / Hkv: they share the keys, so one pass over the keys serves them
// all. Row r sees key j when j < ctx, or when j = ctx + d and bit d of its
// token's mask is set:
//     x_j = scale * q . k_j,   o = sum_j exp(x_j - M) v_j / sum_j exp(x_j - M)
// with the running maximum M and sum of the softmax carried along the keys
// (in units of log2, so the exponential is one ex2), in fp32.
//
// Work: an item is (b, h, block of rows); its keys come in units. All items'
// units in order are one sequence that the thread blocks share out evenly, so
// ragged contexts and few heads fill the GPU alike. A block's part of an item
// is a segment; a segment that is not the whole item leaves its unnormalised
// sum, maximum and sum of exponentials in the workspace, and k_attn_join adds
// them up in key order (the same order every time).
#include <cudaTypedefs.h>
#include <math.h>
#include <string.h>

#include <mutex>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_plan.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

// Byte offset of 16-byte chunk c of row r in a copied slice of `rows` rows:
// [chunk of 128 bytes][row][128 bytes], the 16-byte units XOR-ed with row mod 8.
template <int kRows>
__device__ __forceinline__ uint32_t slice_ofs(int r, int c) {
    return (uint32_t)((c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ------------------------------------------------------------------ few rows

// Up to 16 * MT rows an item, on the warp MMA. Each of the NW warps takes 16
// keys of every unit through its own ring of kStages copies and keeps its own
// maximum, sum and output accumulators, so the warps meet only at a segment's
// end. What bounds it is the stream of keys and values: 16 rows need 4 x 16
// multiply-adds per loaded value, far below the warp MMA's rate.
//
// The exponentials go to the second product as two 16-bit numbers each (the
// rounded value and the rounded rest), so the output carries no more than its
// own rounding; the extra products are free next to the copies.
template <int D, int MT, int NW>
struct RowsShape {
    static constexpr int kRows = 16 * MT;
    static constexpr int kSlice = 16 * D * 2;         // bytes of 16 keys (or values)
    static constexpr int kStages = 3 * 128 / D;
    static constexpr int kRing = NW * kStages * 2 * kSlice;
    static constexpr int kBuf = kRows * D * 4;
    static constexpr int kMl = NW * kRows * 8;
    static constexpr int kSmem = kRing + kBuf + kMl + NW * kStages * 12 + 8 * NW + 32;
};

template <int D, int MT, int NW, bool kBf16>
__global__ void __launch_bounds__(32 * NW, NW == 4 ? 2 : 1)
    k_attn_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const TreeArgs a) {
    using S = RowsShape<D, MT, NW>;
    // fp16 weights are held 2^15 times larger: the small ones would lose bits
    // below fp16's range
    constexpr float kBoost = kBf16 ? 0.f : 15.f;
    constexpr int kRows = S::kRows, kStages = S::kStages, KK = D / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *buf = reinterpret_cast<float *>(smem + S::kRing);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kRing + S::kBuf);
    auto *share = reinterpret_cast<ShareScratch<NW> *>(smem + S::kRing + S::kBuf + S::kMl);
    uint64_t *bars = reinterpret_cast<uint64_t *>(share + 1);
    int *flags = reinterpret_cast<int *>(bars + NW * kStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    uint64_t *bar = bars + warp * kStages;
    int *flag = flags + warp * kStages;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc05::mbar_init(bar + i, 1);
        tc05::fence_mbar_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && a.status) {
        for (int b = threadIdx.x; b < a.s.B; b += 32 * NW) {
            bool ok;
            get_seq(a.s, b, ok);
            if (!ok) set_status(a.status, kStLength);
        }
    }
    const Share sh = find_share<32 * NW>(a, share);
    const long long u0 = sh.u0, u1 = sh.u1;
    if (u0 >= u1) return;

    Cursor pc, cc;  // of the copies, of the products
    cc.start(a, sh);
    pc = cc;
    long long pu = u0;  // next unit to copy
    int pstage = 0, pid = 0;
    const uint32_t ring = tc05::smem_addr(smem) + warp * (kStages * 2 * S::kSlice);

    auto fetch_page = [&]() {
        const int s0 = pc.u * a.unit + warp * 16;
        pid = s0 < pc.q.ctx + pc.q.T
                  ? __ldg(a.s.table + (long long)pc.b * a.s.max_pages + (s0 >> a.s.lpage))
                  : 0;
    };
    // Issues the copies of this warp's 16 keys and values of unit pu, then
    // starts the load of the next unit's page id.
    auto issue = [&]() {
        const int s0 = pc.u * a.unit + warp * 16;
        const bool live = s0 < pc.q.ctx + pc.q.T;
        const bool good = live && (unsigned)pid < (unsigned)a.pages;
        if (lane == 0) {
            flag[pstage] = good;
            uint64_t *br = bar + pstage;
            if (good) {
                const int row = (pid * a.Hkv + pc.h) * a.s.page + (s0 & (a.s.page - 1));
                const uint32_t dst = ring + pstage * (2 * S::kSlice);
                mbar_expect_tx(br, 2 * S::kSlice);
                tma_load3(dst, &kmap, 0, row, 0, br);
                tma_load3(dst + S::kSlice, &vmap, 0, row, 0, br);
            } else {
                mbar_arrive(br);
                if (live) set_status(a.status, kStPage);
            }
        }
        if (++pstage == kStages) pstage = 0;
        ++pu;
        if (++pc.u == pc.nu) pc.next_item(a);
        if (pu < u1) fetch_page();
    };

    fetch_page();
    for (int i = 0; i < kStages - 1 && pu < u1; ++i) issue();

    // key and 16-byte chunk of this lane's row in the 8x8 matrices of an ldmatrix
    const int kkey = (lane & 7) + ((lane >> 4) << 3), kchk = (lane >> 3) & 1;
    const int vkey = (lane & 7) + (((lane >> 3) & 1) << 3), vchk = lane >> 4;
    const int g = lane >> 2, c = lane & 3;

    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    long long u = u0;
    while (u < u1) {
        // ---- one segment
        const bool at_start = cc.u == 0, first_seg = u == u0;
        const int seg_b = cc.b, seg_h = cc.h, seg_rb = cc.rb;
        const Seq sq = cc.q;
        const int nrows = sq.T * a.G;
        uint32_t qf[MT][KK][4];
        int rt[MT][2];  // draft of each of this lane's rows, -1: no row
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = seg_rb * kRows + m * 16 + e * 8 + g;
                const bool have = r < nrows;
                const int t = have ? r / a.G : 0;
                rt[m][e] = have ? t : -1;
                const uint16_t *p = a.q + (long long)(sq.first + t) * a.q_stride +
                                    (long long)(seg_h * a.G + (have ? r - t * a.G : 0)) * D;
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(p + k * 16 + c * 2);
                    qf[m][k][e] = have ? (w[0] ^ a.qxor) & a.qand : 0u;
                    qf[m][k][e + 2] = have ? (w[4] ^ a.qxor) & a.qand : 0u;
                }
            }
        }
        float o[MT][D / 8][4];
        float mx[MT][2], l[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
            mx[m][0] = mx[m][1] = -INFINITY;
            l[m][0] = l[m][1] = 0.f;
        }
        bool done = false;
        while (!done) {
            if (pu < u1 && !dead) issue();
            if (!dead && !tc05::mbar_wait(bar + stage, phase, kPoll)) {
                // give up: flag it, and wait (bounded as well) for the copies in flight
                dead = true;
                if (lane == 0) set_status(a.status, kStTimeout);
                int ds = stage;
                uint32_t dp = phase;
                for (long long x = u; x < pu; ++x) {
                    tc05::mbar_wait(bar + ds, dp, kPoll);
                    if (++ds == kStages) {
                        ds = 0;
                        dp ^= 1;
                    }
                }
            }
            dead = __any_sync(0xFFFFFFFFu, dead);
            const int s0 = cc.u * a.unit + warp * 16;
            if (!dead && flag[stage]) {
                const uint32_t ks = ring + stage * (2 * S::kSlice), vs = ks + S::kSlice;
                float s[MT][2][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[m][n][i] = 0.f;
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    uint32_t kb[4];
                    ldmatrix4(kb, ks + slice_ofs<16>(kkey, 2 * k + kchk));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816<kBf16>(s[m][0], qf[m][k], kb[0], kb[1]);
                        mma16816<kBf16>(s[m][1], qf[m][k], kb[2], kb[3]);
                    }
                }
                if (s0 + 16 > sq.ctx) {  // drafts, or the end of the sequence, in this slice
                    const int len = sq.ctx + sq.T;
                    uint32_t see[MT][2];  // of this slice's 16 keys, by row
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            see[m][e] = rt[m][e] >= 0 ? seen_word(a, sq, rt[m][e], s0) : 0u;
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (!((see[m][e] >> (n * 8 + c * 2 + i)) & 1u))
                                        s[m][n][2 * e + i] = -INFINITY;
                        }
                    // Values that some row must not see are kept out of the
                    // product where zero times them is not zero: rows past the
                    // end (whatever an unused slot holds) become zeros, and a
                    // draft's infinities and NaNs are added to the rows that
                    // see it and replaced by zeros.
                    for (int j = 0; j < 16; ++j) {
                        const int key = s0 + j;
                        if (key < sq.ctx) continue;
                        bool bad = false;
                        for (int w = lane; w < D / 2; w += 32) {
                            const uint32_t ad = vs + slice_ofs<16>(j, w >> 2) + (w & 3) * 4;
                            if (key >= len)
                                sts32(ad, 0u);
                            else
                                bad |= nonfinite2<kBf16>(lds32(ad));
                        }
                        if (__any_sync(0xFFFFFFFFu, bad)) {
                            __syncwarp();
#pragma unroll
                            for (int m = 0; m < MT; ++m)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if ((see[m][e] >> j) & 1u)
#pragma unroll
                                        for (int n = 0; n < D / 8; ++n) {
                                            const float2 f = unpack2<kBf16>(
                                                lds32(vs + slice_ofs<16>(j, n) + c * 4));
                                            if (!isfinite(f.x)) o[m][n][2 * e] += f.x;
                                            if (!isfinite(f.y)) o[m][n][2 * e + 1] += f.y;
                                        }
                            __syncwarp();
                            for (int w = lane; w < D / 2; w += 32) {
                                const uint32_t ad = vs + slice_ofs<16>(j, w >> 2) + (w & 3) * 4;
                                uint32_t v = lds32(ad);
                                if (nonfinite2<kBf16>(v & 0xFFFFu)) v &= 0xFFFF0000u;
                                if (nonfinite2<kBf16>(v & 0xFFFF0000u)) v &= 0x0000FFFFu;
                                sts32(ad, v);
                            }
                        }
                    }
                    // the next copy into this slot comes from the async proxy
                    tc05::fence_proxy_async();
                    __syncwarp();
                }
                if (a.stash) {  // the masked scores, for the weights' own pass
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (rt[m][e] >= 0) {
                                float *p = stash_at(a, seg_b, seg_h, s0) + (m * 16 + e * 8 + g) * 16 + c * 2;
                                *reinterpret_cast<float2 *>(p) = make_float2(s[m][0][2 * e], s[m][0][2 * e + 1]);
                                *reinterpret_cast<float2 *>(p + 8) = make_float2(s[m][1][2 * e], s[m][1][2 * e + 1]);
                            }
                }
                uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = fmaxf(fmaxf(s[m][0][2 * e] * a.sl2, s[m][0][2 * e + 1] * a.sl2),
                                        fmaxf(s[m][1][2 * e] * a.sl2, s[m][1][2 * e + 1] * a.sl2));
                        t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
                        t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                        const float mn = fmaxf(mx[m][e], t);
                        if (__any_sync(0xFFFFFFFFu, mn > mx[m][e])) {
                            const float al = mn == mx[m][e] ? 1.f : ex2(mx[m][e] - mn);
                            mx[m][e] = mn;
                            l[m][e] *= al;
#pragma unroll
                            for (int n = 0; n < D / 8; ++n) {
                                o[m][n][2 * e] *= al;
                                o[m][n][2 * e + 1] *= al;
                            }
                        }
                        const float base = mx[m][e] == -INFINITY ? 0.f : mx[m][e] - kBoost;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float p0 = ex2(fmaf(s[m][n][2 * e], a.sl2, -base));
                            const float p1 = ex2(fmaf(s[m][n][2 * e + 1], a.sl2, -base));
                            l[m][e] += p0 + p1;
                            const uint32_t hi = pack2<kBf16>(p0, p1);
                            const float2 f = unpack2<kBf16>(hi);
                            ph[m][2 * n + e] = hi;
                            pl[m][2 * n + e] = pack2<kBf16>(p0 - f.x, p1 - f.y);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    uint32_t vb[4];
                    ldmatrix4_trans(vb, vs + slice_ofs<16>(vkey, 2 * k + vchk));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816<kBf16>(o[m][2 * k], ph[m], vb[0], vb[1]);
                        mma16816<kBf16>(o[m][2 * k + 1], ph[m], vb[2], vb[3]);
                        mma16816<kBf16>(o[m][2 * k], pl[m], vb[0], vb[1]);
                        mma16816<kBf16>(o[m][2 * k + 1], pl[m], vb[2], vb[3]);
                    }
                }
            }
            __syncwarp();  // the slot may be copied into again
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
            ++u;
            done = ++cc.u == cc.nu || u == u1;
        }
        const bool whole = at_start && cc.u == cc.nu;
        if (cc.u == cc.nu) cc.next_item(a);

        // ---- the segment's end: the warps' sums, one warp after the other
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (mx[m][e] != -INFINITY) mx[m][e] -= kBoost;
                l[m][e] += __shfl_xor_sync(0xFFFFFFFFu, l[m][e], 1);
                l[m][e] += __shfl_xor_sync(0xFFFFFFFFu, l[m][e], 2);
                if (c == 0) ml[warp * kRows + m * 16 + e * 8 + g] = make_float2(mx[m][e], l[m][e]);
            }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w)
                    M = fmaxf(M, ml[w * kRows + m * 16 + e * 8 + g].x);
                const float f = mx[m][e] == -INFINITY ? 1.f : ex2(mx[m][e] - M);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[m][n][2 * e] *= f;
                    o[m][n][2 * e + 1] *= f;
                }
            }
        for (int w = 0; w < NW; ++w) {
            if (warp == w) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            const int r = m * 16 + e * 8 + g;
                            float2 *p = reinterpret_cast<float2 *>(
                                buf + r * D + ((n * 8 + c * 2) ^ ((r & 3) << 3)));
                            float2 v = make_float2(o[m][n][2 * e], o[m][n][2 * e + 1]);
                            if (w > 0) {
                                v.x += p->x;
                                v.y += p->y;
                            }
                            *p = v;
                        }
            }
            __syncthreads();
        }
        // rows out: two columns a thread
        const int used = min(kRows, nrows - seg_rb * kRows);
        for (int i = threadIdx.x; i < used * (D / 2); i += 32 * NW) {
            const int r = i / (D / 2), col = (i - r * (D / 2)) * 2;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w * kRows + r].x);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float2 v = ml[w * kRows + r];
                L += v.x == -INFINITY ? v.y : v.y * ex2(v.x - M);
            }
            float2 v = *reinterpret_cast<const float2 *>(buf + r * D + (col ^ ((r & 3) << 3)));
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                v.x *= inv;
                v.y *= inv;
                const int rr = seg_rb * kRows + r, t = rr / a.G;
                const long long row = (long long)(sq.first + t) * a.Hq + seg_h * a.G + rr - t * a.G;
                if (a.o_f32)
                    *reinterpret_cast<float2 *>(static_cast<float *>(a.o) + row * D + col) = v;
                else
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.o) + row * D + col) =
                        pack2<kBf16>(v.x, v.y);
                if (col == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
            } else {
                const int last = first_seg ? 0 : 1;
                *reinterpret_cast<float2 *>(part_at<D>(a, blockIdx.x, last, r, col & ~3) + (col & 3)) = v;
                if (col == 0)
                    *reinterpret_cast<float2 *>(
                        a.part_ml + (((long long)blockIdx.x * 2 + last) * kRows + r) * 2) = make_float2(M, L);
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ joining segments

// Adds up the segments of an item that several blocks shared, in key order,
// kXb blocks' segments at a time (their loads in flight together). A warp takes
// 8 rows: lane l has row l % 8 and every fourth group of 4 columns, kCols of
// them (the rest of a row's columns are other warps'). kSplit warps share a
// long row of segments and meet in shared memory. The call's inputs are older
// than its first kernel, so everything up to the segments is read before the
// wait for it.
template <int D, int kCols, int kXb, int kSplit>
__global__ void __launch_bounds__(128 * kSplit) k_attn_join(const TreeArgs a, bool bf16) {
    constexpr int kParts = D / 16 / kCols;  // warps a row
    __shared__ long long scan[8 * kSplit];
    __shared__ float meet[kSplit > 1 ? (kSplit - 1) * 128 * (kCols * 4 + 2) : 1];
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv, rb = blockIdx.y;
    bool ok;
    const Seq q = get_seq(a.s, b, ok);
    const int nu = key_units(q, a.unit), nrb = row_blocks(q, a.G, a.rows);
    long long before;
    const long long total = count_units<128 * kSplit>(a, b, scan, before);
    const long long quota = (total + a.grid - 1) / a.grid;
    const long long i0 = before + ((long long)h * nrb + rb) * nu, i1 = i0 + nu;
    const bool any = q.T > 0 && rb < nrb;
    const int c0 = any ? (int)(i0 / quota) : 0, c1 = any ? (int)((i1 - 1) / quota) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (c0 == c1) return;  // nothing here, or one segment, written by its block
    const int rows = min(a.rows, q.T * a.G - rb * a.rows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.z * 4 + (warp & 3), split = warp >> 2;
    const int r = (w / kParts) * 8 + (lane & 7), col0 = (w % kParts) * (kCols * 16) + (lane >> 3) * 4;
    const bool have_row = r < rows;
    // this warp's stretch of the segments
    const int per = (c1 - c0 + kSplit) / kSplit;
    const int x_begin = c0 + split * per, x_end = min(c1 + 1, x_begin + per);

    float M = -INFINITY, L = 0.f, acc[kCols][4];
#pragma unroll
    for (int i = 0; i < kCols; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    auto add = [&](float m, float l, const float (&v)[kCols][4]) {
        const float mn = fmaxf(M, m);
        const float f0 = M == mn ? 1.f : ex2(M - mn), f1 = m == mn ? 1.f : ex2(m - mn);
        M = mn;
        L = L * f0 + l * f1;
#pragma unroll
        for (int i = 0; i < kCols; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = acc[i][e] * f0 + v[i][e] * f1;
    };
    for (int x0 = x_begin; x0 < x_end; x0 += kXb) {
        float2 ml[kXb];
        float v[kXb][kCols][4];
#pragma unroll
        for (int j = 0; j < kXb; ++j) {
            const int x = x0 + j, last = (long long)x * quota >= i0 ? 0 : 1;
            const bool have = x < x_end && have_row;
            ml[j] = have ? *reinterpret_cast<const float2 *>(
                               a.part_ml + (((long long)x * 2 + last) * a.rows + r) * 2)
                         : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                const float4 f = have ? *reinterpret_cast<const float4 *>(
                                            part_at<D>(a, x, last, r, col0 + 16 * i))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                v[j][i][0] = f.x; v[j][i][1] = f.y; v[j][i][2] = f.z; v[j][i][3] = f.w;
            }
        }
#pragma unroll
        for (int j = 0; j < kXb; ++j) add(ml[j].x, ml[j].y, v[j]);
    }
    if (kSplit > 1) {
        constexpr int kWords = kCols * 4 + 2;
        const int at = threadIdx.x & 127;
        if (split > 0) {
            float *p = meet + (split - 1) * 128 * kWords + at;
            p[0] = M;
            p[128] = L;
#pragma unroll
            for (int i = 0; i < kCols * 4; ++i) p[(2 + i) * 128] = acc[i >> 2][i & 3];
        }
        __syncthreads();
        if (split > 0) return;
#pragma unroll
        for (int k = 0; k < kSplit - 1; ++k) {
            const float *p = meet + k * 128 * kWords + at;
            float v[kCols][4];
#pragma unroll
            for (int i = 0; i < kCols * 4; ++i) v[i >> 2][i & 3] = p[(2 + i) * 128];
            add(p[0], p[128], v);
        }
    }
    if (!have_row) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int rr = rb * a.rows + r, t = rr / a.G;
    const long long row = (long long)(q.first + t) * a.Hq + h * a.G + rr - t * a.G;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        const float x0 = acc[i][0] * inv, x1 = acc[i][1] * inv, x2 = acc[i][2] * inv, x3 = acc[i][3] * inv;
        const long long at = row * D + col0 + 16 * i;
        if (a.o_f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = make_float4(x0, x1, x2, x3);
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o) + at) =
                bf16 ? make_uint2(pack2<true>(x0, x1), pack2<true>(x2, x3))
                     : make_uint2(pack2<false>(x0, x1), pack2<false>(x2, x3));
    }
    if (col0 == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------ host

template <int D, int MT, int NW, bool kBf16>
cudaError_t run_rows(const CUtensorMap &km, const CUtensorMap &vm, const TreeArgs &a,
                     cudaStream_t st) {
    auto *k = k_attn_rows<D, MT, NW, kBf16>;
    constexpr int smem = RowsShape<D, MT, NW>::kSmem;
    cudaError_t e = set_smem(k, smem);
    if (e == cudaSuccess) e = launch(k, dim3(a.grid), dim3(32 * NW), smem, st, true, km, vm, a);
    return e;
}

template <int D, bool kBf16>
cudaError_t run_tree(const AttnCache &c, const CUtensorMap &km, const CUtensorMap &vm,
                     const TreeArgs &a, int max_rows, cudaStream_t st) {
    cudaError_t e = a.rows == 16   ? run_rows<D, 1, 4, kBf16>(km, vm, a, st)
                    : a.rows == 32 ? run_rows<D, 2, 8, kBf16>(km, vm, a, st)
                                   : launch_tree_tc(c, a, st);
    const int nrb = (max_rows + a.rows - 1) / a.rows;
    // many rows: a warp 8 of them whole, two blocks' segments at a time; few rows:
    // a warp a part of 8 rows, four warps sharing the blocks' segments where items
    // are so few that each has many (8 items of 38 segments: 10.8 -> 5.8 us)
    const bool many = a.rows > 32, longs = a.grid > 8 * a.s.B * a.Hkv * nrb;
    const int warps = ((max_rows < a.rows ? max_rows : a.rows) + 7) / 8 * (many ? 1 : D / 32);
    const dim3 grid(a.s.B * a.Hkv, nrb, (warps + 3) / 4);
    if (e == cudaSuccess)
        e = many ? launch(k_attn_join<D, D / 16, 2, 1>, grid, dim3(128), 0, st, true, a, (bool)kBf16)
            : longs ? launch(k_attn_join<D, 2, 5, 4>, grid, dim3(512), 0, st, true, a, (bool)kBf16)
                    : launch(k_attn_join<D, 2, 8, 1>, grid, dim3(128), 0, st, true, a, (bool)kBf16);
    if (e == cudaSuccess && a.acc_out) e = launch_tree_weights(c, a, max_rows, st);
    return e;
}

// Rows an item: up to 32 on the warp MMA, more on tcgen05 (qmv_attn_tc.cu).
int tree_rows(int max_rows) {
    return max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : max_rows <= 128 ? 128 : 256;
}
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

int tree_grid_max(int rows) { return sm_count() * (rows == 16 ? 2 : 1); }

}  // namespace
}  // namespace attn

namespace attn {

bool encode_pool(CUtensorMap *map, const void *pool, const AttnCache &c, int box_rows, bool all_chunks) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)c.D * 2, chunks = row / 128;
    cuuint64_t dims[3] = {128, (cuuint64_t)c.pages * c.Hkv * c.page, chunks};
    cuuint64_t strides[2] = {row, 128};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, all_chunks ? (cuuint32_t)chunks : 1u};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pool), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// Where the weights come from with up to 32 rows: scores that the attention
// leaves in the workspace, or a second product of queries and keys. A score
// costs 4 bytes written and 4 read a row, a key's second reading 2 D bytes; the
// workspace is kept within kStashMax.
constexpr size_t kStashMax = (size_t)1 << 30;
size_t stash_bytes(const AttnCache &c, int max_rows, int B, int max_pages) {
    if (max_rows > 32) return 0;
    const size_t n = (size_t)B * c.Hkv * max_pages * c.page * max_rows * 4;
    return n <= kStashMax ? n : 0;
}

size_t part_bytes(const AttnCache &c, int rows) {
    const size_t slots = (size_t)tree_grid_max(rows) * 2 * rows;
    return (slots * (c.D + 2) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace attn

size_t attn_tree_ws_bytes(const AttnCache &c, int Hq, int B, int N, int max_draft, int max_pages,
                          bool acc) {
    (void)N;
    const int max_rows = max_draft * (Hq / c.Hkv);
    return attn::part_bytes(c, attn::tree_rows(max_rows)) +
           (acc ? attn::stash_bytes(c, max_rows, B, max_pages) : 0);
}

cudaError_t launch_attn_tree(const AttnCache &c, const TreeCall &t, cudaStream_t st) {
    using namespace attn;
    TreeArgs a;
    memset(&a, 0, sizeof(a));
    int lpage = 0;
    while ((1 << lpage) < c.page) ++lpage;
    a.s = Seqs{t.s.table, t.s.ctx, t.s.cu, t.s.B, t.s.N, t.s.max_draft, t.s.max_pages, c.page, lpage};
    a.q = static_cast<const uint16_t *>(t.q);
    a.q_stride = t.q_stride;
    a.Hq = t.Hq; a.Hkv = c.Hkv; a.G = t.Hq / c.Hkv; a.pages = c.pages;
    a.mask = t.mask; a.words = t.words;
    a.sl2 = t.scale == 0.f ? 1.f : fabsf(t.scale) * kLog2e;
    a.qxor = t.scale < 0.f ? 0x80008000u : 0u;
    a.qand = t.scale == 0.f ? 0u : 0xFFFFFFFFu;
    a.o = t.o; a.o_f32 = t.o_f32; a.lse = t.lse;
    a.kpool = static_cast<const uint16_t *>(c.k);
    a.vpool = static_cast<const uint16_t *>(c.v);
    a.acc_in = t.acc_in; a.acc_out = t.acc_out; a.decay = t.decay;
    a.status = t.status;
    const int max_rows = t.s.max_draft * a.G;
    a.rows = tree_rows(max_rows);
    a.unit = a.rows == 16 ? 64 : 128;  // keys a unit
    const long long most = (long long)t.s.B * c.Hkv * ((max_rows + a.rows - 1) / a.rows) *
                           ((((long long)t.s.max_pages << lpage) + a.unit - 1) / a.unit);
    const int gmax = tree_grid_max(a.rows);
    a.grid = most < gmax ? (int)most : gmax;
    a.part_o = static_cast<float *>(t.ws);
    a.part_ml = a.part_o + (size_t)gmax * 2 * a.rows * c.D;
    a.max_rows = max_rows;
    if (a.acc_out && stash_bytes(c, max_rows, t.s.B, t.s.max_pages))
        a.stash = reinterpret_cast<float *>(static_cast<char *>(t.ws) + part_bytes(c, a.rows));
    CUtensorMap km, vm;
    if (!encode_pool(&km, c.k, c, 16, true) || !encode_pool(&vm, c.v, c, 16, true))
        return cudaErrorNotSupported;
    if (c.D == 64)
        return c.bf16 ? run_tree<64, true>(c, km, vm, a, max_rows, st)
                      : run_tree<64, false>(c, km, vm, a, max_rows, st);
    return c.bf16 ? run_tree<128, true>(c, km, vm, a, max_rows, st)
                  : run_tree<128, false>(c, km, vm, a, max_rows, st);
}

}  // namespace qmv
