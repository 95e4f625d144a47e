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

// Up to 16 rows an item, on the warp MMA. Each of the four warps takes a slice
// of every unit (16 keys, 32 of 64 elements) through its own ring of kStages
// copies and keeps its own maximum, sum and output accumulators, so the warps
// meet only at a segment's end. What bounds it is the stream of keys and
// values: 16 rows need 4 x 16 multiply-adds per loaded value, far below the
// warp MMA's rate. 64 sequences of up to 8191 keys, 4 rows, take 247 us (6.3
// TB/s), one of 200,003 keys, 6 rows, 133 (6.2 TB/s), one of 777 10.6, joins
// included. (32 rows a warp measured 452 us where the tcgen05 kernel takes 244,
// 64 sequences of 8191 keys: registers leave one block an SM.)
//
// The exponentials go to the second product as two 16-bit numbers each (the
// rounded value and the rounded rest), so that a 16-bit output carries no more
// than its own rounding; the extra products are free next to the copies. For an
// fp32 output (kExact) there is a third bf16 number, and a slice's products are
// summed up by themselves and then added: the MMA cuts off what falls below its
// sum's last bit, and with that carried along all keys the output was three
// times as far off as with fp32 sums (one token over 200,000 keys: 3.9e-6 of the
// output's norm, against 1.4e-6).
constexpr int kRows = 16, kWarps = 4;
template <int D>
struct RowsShape {
    static constexpr int kSub = 128 / D;              // 16-key parts of a slice
    static constexpr int kPart = 16 * D * 2;          // bytes of 16 keys (or values)
    static constexpr int kSlice = kSub * kPart;
    static constexpr int kStages = 3;
    static constexpr int kUnit = kWarps * kSub * 16;  // keys a unit
    static constexpr int kRing = kWarps * kStages * 2 * kSlice;
    static constexpr int kBuf = 2 * kRows * D * 4;    // two warps' sums
    static constexpr int kMl = kWarps * kRows * 8;
    static constexpr int kSmem =
        kRing + kBuf + kMl + kWarps * kStages * 12 + (int)sizeof(ShareScratch<kWarps>);
};

template <int D, bool kBf16, bool kExact>
__global__ void __launch_bounds__(32 * kWarps, 2)
    k_attn_rows(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const TreeArgs a) {
    using S = RowsShape<D>;
    // fp16 weights are held 2^15 times larger: the small ones would lose bits
    // below fp16's range
    constexpr float kBoost = kBf16 ? 0.f : 15.f;
    constexpr int kStages = S::kStages, KK = D / 16, kSub = S::kSub, kNt = 2 * kSub;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *buf = reinterpret_cast<float *>(smem + S::kRing);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kRing + S::kBuf);
    auto *share = reinterpret_cast<ShareScratch<kWarps> *>(smem + S::kRing + S::kBuf + S::kMl);
    uint64_t *bars = reinterpret_cast<uint64_t *>(share + 1);
    int *flags = reinterpret_cast<int *>(bars + kWarps * kStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    uint64_t *bar = bars + warp * kStages;
    int *flag = flags + warp * kStages;  // which 16-key parts of a slice were copied
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc05::mbar_init(bar + i, 1);
        tc05::fence_mbar_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && a.status) {
        for (int b = threadIdx.x; b < a.s.B; b += 32 * kWarps) {
            bool ok;
            get_seq(a.s, b, ok);
            if (!ok) set_status(a.status, kStLength);
        }
    }
    const Share sh = find_share<32 * kWarps>(a, share);
    if (sh.u0 >= sh.u1) return;
    const int units = (int)(sh.u1 - sh.u0);  // (the launcher keeps this below 2^31)

    // keys and values are read once here, and must not push the scores kept for
    // the weights out of L2
    const uint64_t policy = evict_first_policy();
    Cursor pc, cc;  // of the copies, of the products
    cc.start(a, sh);
    pc = cc;
    int to_copy = units, pstage = 0, pid = 0;
    const uint32_t ring = tc05::smem_addr(smem) + warp * (kStages * 2 * S::kSlice);
    // this lane's 16-key part of the slice (lanes 0 .. kSub - 1 copy one each)
    const int part = kSub > 1 ? min(lane, kSub - 1) : 0;
    auto part_slot = [&](int u) { return (u * kWarps + warp) * (kSub * 16) + part * 16; };

    auto fetch_page = [&]() {
        const int s0 = part_slot(pc.u);
        pid = s0 < pc.q.ctx + pc.q.T
                  ? __ldg(a.s.table + (long long)pc.b * a.s.max_pages + (s0 >> a.s.lpage))
                  : 0;
    };
    // Issues the copies of this warp's slice of the next unit, then starts the
    // load of the page ids of the one after.
    auto issue = [&]() {
        const int s0 = part_slot(pc.u);
        const bool mine = lane < kSub, live = mine && s0 < pc.q.ctx + pc.q.T;
        const bool good = live && (unsigned)pid < (unsigned)a.pages;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, good);
        uint64_t *br = bar + pstage;
        if (lane == 0) {
            flag[pstage] = (int)who;
            if (who)
                mbar_expect_tx(br, __popc(who) * 2 * S::kPart);
            else
                mbar_arrive(br);
        }
        __syncwarp();
        if (good) {
            const int row = (pid * a.Hkv + pc.h) * a.s.page + (s0 & (a.s.page - 1));
            const uint32_t dst = ring + pstage * (2 * S::kSlice) + part * S::kPart;
            tma_load3_once(dst, &kmap, 0, row, 0, br, policy);
            tma_load3_once(dst + S::kSlice, &vmap, 0, row, 0, br, policy);
        } else if (live) {
            set_status(a.status, kStPage);
        }
        __syncwarp();
        if (++pstage == kStages) pstage = 0;
        --to_copy;
        if (++pc.u == pc.nu) pc.next_item(a);
        if (to_copy > 0) fetch_page();
    };

    fetch_page();
    for (int i = 0; i < kStages - 1 && to_copy > 0; ++i) issue();

    // key and 16-byte chunk of this lane's row in the 8x8 matrices of an ldmatrix
    const int kkey = (lane & 7) + ((lane >> 4) << 3), kchk = (lane >> 3) & 1;
    const int vkey = (lane & 7) + (((lane >> 3) & 1) << 3), vchk = lane >> 4;
    const int g = lane >> 2, c = lane & 3;

    int stage = 0, left = units;
    uint32_t phase = 0;
    bool dead = false;
    while (left > 0) {
        // ---- one segment
        const bool at_start = cc.u == 0, first_seg = left == units;
        const int seg_b = cc.b, seg_h = cc.h;
        const Seq sq = cc.q;
        const int nrows = sq.T * a.G;  // at most 16
        uint32_t qf[KK][4];
        int rt[2];  // draft of each of this lane's rows, -1: no row
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = e * 8 + g;
            const bool have = r < nrows;
            const int t = have ? div_g(a, r) : 0;
            rt[e] = have ? t : -1;
            const uint16_t *p = a.q + (long long)(sq.first + t) * a.q_stride +
                                (long long)(seg_h * a.G + (have ? r - t * a.G : 0)) * D;
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(p + k * 16 + c * 2);
                qf[k][e] = have ? (w[0] ^ a.qxor) & a.qand : 0u;
                qf[k][e + 2] = have ? (w[4] ^ a.qxor) & a.qand : 0u;
            }
        }
        float *kept = a.stash ? stash_at(a, seg_b, seg_h, 0) + g * 16 + c * 2 : nullptr;
        float o[D / 8][4];
        float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        bool done = false;
        while (!done) {
            if (to_copy > 0 && !dead) issue();
            if (!dead && !tc05::mbar_wait(bar + stage, phase, kPoll)) {
                // give up: flag it, and wait (bounded as well) for the copies in flight
                dead = true;
                if (lane == 0) set_status(a.status, kStTimeout);
                int ds = stage;
                uint32_t dp = phase;
                for (int x = left; x > to_copy; --x) {
                    tc05::mbar_wait(bar + ds, dp, kPoll);
                    if (++ds == kStages) {
                        ds = 0;
                        dp ^= 1;
                    }
                }
            }
            dead = __any_sync(0xFFFFFFFFu, dead);
            const int s0 = (cc.u * kWarps + warp) * (kSub * 16);
            const int copied = dead ? 0 : flag[stage];
            if (copied) {
                const uint32_t ks = ring + stage * (2 * S::kSlice), vs = ks + S::kSlice;
                float s[kNt][4];
#pragma unroll
                for (int n = 0; n < kNt; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int j = 0; j < kSub; ++j) {
                        uint32_t kb[4];
                        ldmatrix4(kb, ks + j * S::kPart + slice_ofs<16>(kkey, 2 * k + kchk));
                        mma16816<kBf16>(s[2 * j], qf[k], kb[0], kb[1]);
                        mma16816<kBf16>(s[2 * j + 1], qf[k], kb[2], kb[3]);
                    }
                // drafts, the end of the sequence or a missing page in this slice
                const bool special = s0 + kSub * 16 > sq.ctx || copied != (1 << kSub) - 1;
                auto there = [&]() {  // its keys that were copied
                    uint32_t w = 0;
#pragma unroll
                    for (int j = 0; j < kSub; ++j)
                        if ((copied >> j) & 1) w |= 0xFFFFu << (16 * j);
                    return w;
                };
                auto sees = [&](int e) {  // and those that this lane's row sees
                    return rt[e] >= 0 ? seen_word(a, sq, rt[e], s0) & there() : 0u;
                };
                if (special) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t see = sees(e);
#pragma unroll
                        for (int n = 0; n < kNt; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!((see >> (n * 8 + c * 2 + i)) & 1u)) s[n][2 * e + i] = -INFINITY;
                    }
                }
                if (a.stash) {  // the masked scores, for the weights' own pass
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (rt[e] >= 0)
#pragma unroll
                            for (int j = 0; j < kSub; ++j)
                                if (kSub == 1 || s0 + j * 16 < sq.ctx + sq.T) {
                                    float *p = kept + (long long)((s0 >> 4) + j) * (a.max_rows * 16) + e * 128;
                                    *reinterpret_cast<float2 *>(p) = make_float2(s[2 * j][2 * e], s[2 * j][2 * e + 1]);
                                    *reinterpret_cast<float2 *>(p + 8) =
                                        make_float2(s[2 * j + 1][2 * e], s[2 * j + 1][2 * e + 1]);
                                }
                }
                constexpr int kTerms = kExact && kBf16 ? 3 : 2;
                uint32_t ph[kTerms][kSub][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = -INFINITY;
#pragma unroll
                    for (int n = 0; n < kNt; ++n) t = fmaxf(t, fmaxf(s[n][2 * e], s[n][2 * e + 1]));
                    t *= a.sl2;
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                    const float mn = fmaxf(mx[e], t);
                    if (__any_sync(0xFFFFFFFFu, mn > mx[e])) {
                        const float al = mn == mx[e] ? 1.f : ex2(mx[e] - mn);
                        mx[e] = mn;
                        l[e] *= al;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][2 * e] *= al;
                            o[n][2 * e + 1] *= al;
                        }
                    }
                    const float base = mx[e] == -INFINITY ? 0.f : mx[e] - kBoost;
#pragma unroll
                    for (int n = 0; n < kNt; ++n) {
                        float p0 = ex2(fmaf(s[n][2 * e], a.sl2, -base));
                        float p1 = ex2(fmaf(s[n][2 * e + 1], a.sl2, -base));
                        l[e] += p0 + p1;
#pragma unroll
                        for (int i = 0; i < kTerms; ++i) {
                            const uint32_t w = pack2<kBf16>(p0, p1);
                            const float2 f = unpack2<kBf16>(w);
                            ph[i][n >> 1][2 * (n & 1) + e] = w;
                            p0 -= f.x;
                            p1 -= f.y;
                        }
                    }
                }
                if (special) {
                    // Values that some row must not see are kept out of the
                    // product where zero times them is not zero: rows past the
                    // end (whatever an unused slot holds) and missing ones become
                    // zeros, and a draft's infinities and NaNs are added to the
                    // rows that see it (after the move of the maximum, whose factor
                    // may be zero) and replaced by zeros.
                    const int len = sq.ctx + sq.T;
                    const uint32_t all = there(), see[2] = {sees(0), sees(1)};
                    for (int j = 0; j < kSub * 16; ++j) {
                        const int key = s0 + j;
                        const bool none = key >= len || !((all >> j) & 1u);
                        if (key < sq.ctx && !none) continue;
                        const uint32_t row = vs + (j >> 4) * S::kPart;
                        bool bad = false;
                        for (int w = lane; w < D / 2; w += 32) {
                            const uint32_t ad = row + slice_ofs<16>(j & 15, w >> 2) + (w & 3) * 4;
                            if (none)
                                sts32(ad, 0u);
                            else
                                bad |= nonfinite2<kBf16>(lds32(ad));
                        }
                        if (__any_sync(0xFFFFFFFFu, bad)) {
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if ((see[e] >> j) & 1u)
#pragma unroll
                                    for (int n = 0; n < D / 8; ++n) {
                                        const float2 f = unpack2<kBf16>(
                                            lds32(row + slice_ofs<16>(j & 15, n) + c * 4));
                                        if (!isfinite(f.x)) o[n][2 * e] += f.x;
                                        if (!isfinite(f.y)) o[n][2 * e + 1] += f.y;
                                    }
                            __syncwarp();
                            for (int w = lane; w < D / 2; w += 32) {
                                const uint32_t ad = row + slice_ofs<16>(j & 15, w >> 2) + (w & 3) * 4;
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
#pragma unroll
                for (int k = 0; k < KK; ++k) {
                    float part[2][4] = {};
                    float(&o0)[4] = kExact ? part[0] : o[2 * k], (&o1)[4] = kExact ? part[1] : o[2 * k + 1];
                    uint32_t vb[kSub][4];
#pragma unroll
                    for (int j = 0; j < kSub; ++j)
                        ldmatrix4_trans(vb[j], vs + j * S::kPart + slice_ofs<16>(vkey, 2 * k + vchk));
#pragma unroll
                    for (int i = kTerms - 1; i >= 0; --i)  // small ones first
#pragma unroll
                        for (int j = 0; j < kSub; ++j) {
                            mma16816<kBf16>(o0, ph[i][j], vb[j][0], vb[j][1]);
                            mma16816<kBf16>(o1, ph[i][j], vb[j][2], vb[j][3]);
                        }
                    if (kExact)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[2 * k][i] += o0[i];
                            o[2 * k + 1][i] += o1[i];
                        }
                }
            }
            __syncwarp();  // the slot may be copied into again
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
            --left;
            done = ++cc.u == cc.nu || left == 0;
        }
        const bool whole = at_start && cc.u == cc.nu;
        if (left > 0) cc.next_item(a);

        // ---- the segment's end: the warps' sums, one warp after the other
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (mx[e] != -INFINITY) mx[e] -= kBoost;
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
            if (c == 0) ml[warp * kRows + e * 8 + g] = make_float2(mx[e], l[e]);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + e * 8 + g].x);
            const float f = mx[e] == -INFINITY ? 1.f : ex2(mx[e] - M);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][2 * e] *= f;
                o[n][2 * e + 1] *= f;
            }
        }
        // (in pairs: 2 and 3 to 0 and 1, then 1 to 0; rows that do not exist are left out)
        auto place = [&](int half, int e, int n) {
            const int r = e * 8 + g;
            return reinterpret_cast<float2 *>(buf + (half * kRows + r) * D +
                                              ((n * 8 + c * 2) ^ ((r & 3) << 3)));
        };
        auto give = [&](int half) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (e * 8 < nrows)
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *place(half, e, n) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
        };
        auto take = [&](int half) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (e * 8 < nrows) {
                    float2 v[D / 8];
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) v[n] = *place(half, e, n);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * e] += v[n].x;
                        o[n][2 * e + 1] += v[n].y;
                    }
                }
        };
        if (warp >= 2) give(warp - 2);
        __syncthreads();
        if (warp < 2) take(warp);
        if (warp == 1) give(1);
        __syncthreads();
        if (warp == 0) {
            take(1);
            give(0);
        }
        __syncthreads();
        // rows out: two columns a thread
        for (int i = threadIdx.x; i < nrows * (D / 2); i += 32 * kWarps) {
            const int r = i / (D / 2), col = (i - r * (D / 2)) * 2;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * kRows + r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 v = ml[w * kRows + r];
                L += v.x == -INFINITY ? v.y : v.y * ex2(v.x - M);
            }
            float2 v = *reinterpret_cast<const float2 *>(buf + r * D + (col ^ ((r & 3) << 3)));
            if (whole) {
                // (no weight: zero, where a value's infinity has made a NaN of 0 x inf too)
                v.x = L == 0.f ? 0.f : v.x * (1.f / L);
                v.y = L == 0.f ? 0.f : v.y * (1.f / L);
                const int t = div_g(a, r);
                const long long row = (long long)(sq.first + t) * a.Hq + seg_h * a.G + r - t * a.G;
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
// wait for it. What bounds it is latency: 7.6 us from cold for the 304 blocks'
// parts of 512 items (2.5 MB), 13.5 us for 31 MB of 128 items of 256 rows.
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
    if (L == 0.f)  // no weight: zero, where a value's infinity has made a NaN of 0 x inf too
#pragma unroll
        for (int i = 0; i < kCols; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int rr = rb * a.rows + r, t = div_g(a, rr);
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

template <int D, bool kBf16>
cudaError_t run_rows(const AttnCache &c, const TreeArgs &a, cudaStream_t st) {
    CUtensorMap km, vm;
    if (!encode_pool(&km, c.k, c, 16, true) || !encode_pool(&vm, c.v, c, 16, true))
        return cudaErrorNotSupported;
    auto *k = a.o_f32 ? k_attn_rows<D, kBf16, true> : k_attn_rows<D, kBf16, false>;
    constexpr int smem = RowsShape<D>::kSmem;
    cudaError_t e = set_smem(k, smem);
    if (e == cudaSuccess) e = launch(k, dim3(a.grid), dim3(32 * kWarps), smem, st, true, km, vm, a);
    return e;
}

template <int D, bool kBf16>
cudaError_t run_tree(const AttnCache &c, const TreeArgs &a, int max_rows, cudaStream_t st) {
    cudaError_t e = a.rows == kRows ? run_rows<D, kBf16>(c, a, st) : launch_tree_tc(c, a, st);
    const int nrb = (max_rows + a.rows - 1) / a.rows;
    // many rows: a warp 8 of them whole, two blocks' segments at a time; few rows:
    // a warp a part of 8 rows, four warps sharing the blocks' segments where items
    // are so few that each has many (8 items of 38 segments: 10.8 -> 5.8 us)
    const bool many = a.rows > kRows, longs = a.grid > 8 * a.s.B * a.Hkv * nrb;
    const int warps = ((max_rows < a.rows ? max_rows : a.rows) + 7) / 8 * (many ? 1 : D / 32);
    const dim3 grid(a.s.B * a.Hkv, nrb, (warps + 3) / 4);
    if (e == cudaSuccess)
        e = many ? launch(k_attn_join<D, D / 16, 2, 1>, grid, dim3(128), 0, st, true, a, (bool)kBf16)
            : longs ? launch(k_attn_join<D, 2, 5, 4>, grid, dim3(512), 0, st, true, a, (bool)kBf16)
                    : launch(k_attn_join<D, 2, 8, 1>, grid, dim3(128), 0, st, true, a, (bool)kBf16);
    if (e == cudaSuccess && a.acc_out) e = launch_tree_weights(c, a, max_rows, st);
    return e;
}

// Rows an item: up to 16 on the warp MMA, more on tcgen05 (qmv_attn_tc.cu).
// With 16 rows the two measured 250 and 240 us (64 sequences of 8191 keys), 124
// and 156 with 64 elements a head, and 12.3 and 15.4 us (one of 777 keys); with 32
// rows 452 and 244. Above 128 rows two tiles share the keys: 192 rows over 16 x
// 8191 keys 106 us, in blocks of 128 150.
int tree_rows(int max_rows) { return max_rows <= kRows ? kRows : max_rows <= 128 ? 128 : 256; }
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

int tree_grid_max(int rows) { return sm_count() * (rows == kRows ? 2 : 1); }

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

// Where the weights come from with up to 16 rows: scores that the attention
// leaves in the workspace, or a second product of queries and keys. A score
// costs 4 bytes written and 4 read a row, a key's second reading 2 D bytes; the
// workspace is kept within kStashMax.
constexpr size_t kStashMax = (size_t)1 << 30;
size_t stash_bytes(const AttnCache &c, int max_rows, int B, int max_pages) {
    if (max_rows > kRows) return 0;
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
    a.s = Seqs{t.s.table, t.s.ctx, t.s.cu, t.s.B, t.s.N, t.s.max_draft, t.s.max_pages, c.page, lpage, 0};
    a.q = static_cast<const uint16_t *>(t.q);
    a.q_stride = t.q_stride;
    a.Hq = t.Hq; a.Hkv = c.Hkv; a.G = t.Hq / c.Hkv; a.pages = c.pages;
    a.ginv = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
    a.mask = t.mask; a.words = t.words;
    a.sl2 = t.scale == 0.f ? 1.f : fabsf(t.scale) * kLog2e;
    a.qxor = t.scale < 0.f ? 0x80008000u : 0u;
    a.qand = t.scale == 0.f ? 0u : 0xFFFFFFFFu;
    a.o = t.o; a.o_f32 = t.o_f32; a.lse = t.lse;
    a.vpool = static_cast<const uint16_t *>(c.v);
    a.acc_in = t.acc_in; a.acc_out = t.acc_out; a.decay = t.decay;
    a.status = t.status;
    const int max_rows = t.s.max_draft * a.G;
    a.rows = tree_rows(max_rows);
    a.unit = a.rows == kRows ? kWarps * 16 * (128 / c.D) : 128;  // keys a unit
    const long long most = (long long)t.s.B * c.Hkv * ((max_rows + a.rows - 1) / a.rows) *
                           ((((long long)t.s.max_pages << lpage) + a.unit - 1) / a.unit);
    const int gmax = tree_grid_max(a.rows);
    if (most / gmax >= 0x7FFFFFFFLL) return cudaErrorInvalidValue;  // a block's units fit 31 bits
    a.grid = most < gmax ? (int)most : gmax;
    a.part_o = static_cast<float *>(t.ws);
    a.part_ml = a.part_o + (size_t)gmax * 2 * a.rows * c.D;
    a.max_rows = max_rows;
    if (a.acc_out && stash_bytes(c, max_rows, t.s.B, t.s.max_pages))
        a.stash = reinterpret_cast<float *>(static_cast<char *>(t.ws) + part_bytes(c, a.rows));
    if (c.D == 64)
        return c.bf16 ? run_tree<64, true>(c, a, max_rows, st)
                      : run_tree<64, false>(c, a, max_rows, st);
    return c.bf16 ? run_tree<128, true>(c, a, max_rows, st)
                  : run_tree<128, false>(c, a, max_rows, st);
}

}  // namespace qmv
