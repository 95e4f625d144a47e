// qmv_rope.cu - rotary positions of new tokens and their append to the cache.
//
// A token at position p turns pair i of every query and key head by the angle
// p * inv_freq[i]:
//     (a, b) -> m * (a cos - b sin, b cos + a sin)
// with the pair at elements (i, i + rot/2), or (2i, 2i + 1) when interleaved;
// elements from rot on pass unchanged. The angle is formed in turns in 64
// bits (off by 3 x 2^-53 of the angle) and only its fraction is rounded to 32: at
// position 10^6 an fp32 angle would be off by hundredths of a radian, the turns by
// 1e-10, their fraction by 3e-8.
// All arithmetic on the elements is fp32, rounded once to the cache's type.
//
// With norms (kNorm) a query or key head x first becomes x * w / sqrt(mean(x^2) +
// eps), the mean over its D elements, w a weight an element: the lanes that share
// the head add up their squares and exchange them (three shuffles at 128 elements),
// and the result goes on to the turn in fp32. The head is in registers either way,
// so the norm costs no traffic. Where the sum of squares leaves fp32's range (elements
// near 1e19 or, with an eps as small, near 1e-16 and below) the head is scaled by a
// power of two first and its squares are added up again: a vote a pass, and code that
// ordinary heads do not run (14,839 tokens of 64 heads 92.6 -> 93.7 us).
//
// A warp takes one token (or a share of its heads, so that few tokens fill the
// GPU too). D / 16 lanes share a head, 16 elements each: a lane has the same
// place in every head that it meets, and so the same eight angles, which stay
// in registers: no shared memory, no barrier. The lanes that share a place
// divide its eight angles and exchange them. What bounds it is the copy: 14,839
// tokens of 64 heads take 82 us, 5.9 TB/s of the 486 MB they read and write; one
// token takes a launch (4.5 us).
#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

struct RopeArgs {
    Seqs s;
    const void *q, *k, *v;
    long long qs, ks, vs;  // elements between tokens
    int Hq, Hkv, D, rot, pages;
    const int32_t *pos;
    const double *inv_freq;
    float mscale;
    uint16_t *q_out, *kc, *vc;
    float *acc;
    int32_t *status;
    int parts;  // blocks a token
    const void *qw, *kw;  // norms' weights [D], null: ones
    int w_f32;            // they are fp32, else of the cache's type
    float eps;
    float low;            // a sum of squares below this lacks bits (0: eps hides them)
};

constexpr int kWarps = 4;  // a block
// Warps an SM that few tokens are split for (336 tokens of 48 heads: 8.2 us; with
// 4 8.3, with 64, whose warps find slots and angles for two heads each, 11.3).
constexpr int kFill = 16;

// Eight consecutive elements as they lie in memory, as fp32, and rounded.
template <bool kBf16, bool kF32>
struct Vec8 {
    uint4 raw[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, long long at) {
        const uint4 *u = kF32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at)
                              : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        raw[0] = __ldcs(u);
        if (kF32) raw[kF32 ? 1 : 0] = __ldcs(u + 1);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
        if (kF32) {
            const uint4 h = raw[kF32 ? 1 : 0];
            const uint32_t v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __uint_as_float(w[i]);
                x[4 + i] = __uint_as_float(v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<kBf16>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
};
template <bool kBf16>
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2<kBf16>(x[0], x[1]), pack2<kBf16>(x[2], x[3]), pack2<kBf16>(x[4], x[5]),
                   pack2<kBf16>(x[6], x[7]));
}

template <bool kBf16, bool kF32>
__device__ __forceinline__ float load1(const void *p, long long at) {
    return kF32 ? static_cast<const float *>(p)[at]
                : to_f32<kBf16>(static_cast<const uint16_t *>(p)[at]);
}

// Squares below 2^-126 lose bits, each less than 2^-150. Beside a sum, or an eps * D,
// of 2^-100 that is nothing (D <= 128).
constexpr float kLowSum = 0x1p-100f;
__device__ __forceinline__ bool out_of_range(const RopeArgs &a, float sum) {
    return !(sum >= a.low && sum <= 3.402823466e38f);
}
// The power of two that brings a head's largest magnitude, or the root of eps * D where
// that is larger, to [1, 4) (2^-22 at least where it is subnormal): the squares and
// eps * s * s are then in range. Infinities, NaNs and zeros stay what they are.
__device__ __forceinline__ float scale_of(const RopeArgs &a, float top, int D) {
    top = fmaxf(top, sqrtf(a.eps) * sqrtf((float)D));
    if (!(top > 0.f && top <= 3.402823466e38f)) return 1.f;
    const int e = (int)(__float_as_uint(top) >> 23);
    return __uint_as_float((uint32_t)max(254 - e, 1) << 23);
}
// The factor that makes a head's mean square (its sum / D, plus eps) one. A head
// of zeros stays zeros.
__device__ __forceinline__ float norm_of(float sum, int D, float eps) {
    const float m = fmaf(sum, 1.f / (float)D, eps);
    return m == 0.f ? 0.f : rsqrtf(m);
}
template <bool kBf16>
__device__ __forceinline__ float weight1(const RopeArgs &a, const void *w, int i) {
    if (!w) return 1.f;
    return a.w_f32 ? static_cast<const float *>(w)[i] : to_f32<kBf16>(static_cast<const uint16_t *>(w)[i]);
}
// Eight weights from element i on, on a 16-byte boundary.
template <bool kBf16>
__device__ __forceinline__ void weights8(const RopeArgs &a, const void *w, int i, float (&x)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 1.f;
    } else if (a.w_f32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + i);
        const float4 u = __ldg(p), v = __ldg(p + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + i));
        const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<kBf16>(r[e]);
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
}

// cos and sin of the angle of pair i at position pos, times mscale.
__device__ __forceinline__ float2 turn_of(const RopeArgs &a, double pos, int i) {
    double t = pos * (a.inv_freq[i] * 0.15915494309189533577);
    t -= floor(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    return make_float2(c * a.mscale, s * a.mscale);
}

// Where a token goes in the cache: its page and row; false if nowhere (the
// status says why). Whole warp.
__device__ __forceinline__ bool find_slot(const RopeArgs &a, int n, int lane, int &pid, int &row) {
    // its sequence holds it (the last of them, where cu is not ascending)
    int b = -1;
    for (int j0 = 0; j0 < a.s.B; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t who =
            __ballot_sync(0xFFFFFFFFu, j < a.s.B && a.s.cu[j] <= n && n < a.s.cu[j + 1]);
        if (who) b = j0 + 31 - __clz(who);
    }
    bool ok = false;
    Seq q;
    q.ctx = q.first = q.T = 0;
    if (b >= 0) q = get_seq(a.s, b, ok);
    ok = ok && n - q.first < q.T;
    pid = -1;
    row = 0;
    if (ok) {
        const int slot = q.ctx + n - q.first;
        pid = a.s.table[(long long)b * a.s.max_pages + (slot >> a.s.lpage)];
        row = slot & (a.s.page - 1);
    }
    const bool good = ok && (unsigned)pid < (unsigned)a.pages;
    if (lane == 0 && !good) set_status(a.status, ok ? kStPage : kStLength);
    return good;
}

// Lengths that do not fit, of sequences without tokens too (one warp of the
// grid, when its rows are on their way).
__device__ __forceinline__ void check_lengths(const RopeArgs &a, int lane) {
    if (!a.status) return;
    for (int b = lane; b < a.s.B; b += 32) {
        bool ok;
        get_seq(a.s, b, ok);
        if (!ok) set_status(a.status, kStLength);
    }
}

struct Head {
    const void *src;
    long long at;   // its first element
    uint16_t *dst;  // null: nowhere
    bool turn;
};
__device__ __forceinline__ Head head_of(const RopeArgs &a, int n, int hd, bool good, int pid, int row) {
    Head r;
    r.dst = nullptr;
    r.turn = hd < a.Hq + a.Hkv;
    if (hd < a.Hq) {
        r.src = a.q;
        r.at = (long long)n * a.qs + (long long)hd * a.D;
        r.dst = a.q_out + ((long long)n * a.Hq + hd) * a.D;
    } else {
        const int h = r.turn ? hd - a.Hq : hd - a.Hq - a.Hkv;
        r.src = r.turn ? a.k : a.v;
        r.at = (long long)n * (r.turn ? a.ks : a.vs) + (long long)h * a.D;
        if (good)
            r.dst = (r.turn ? a.kc : a.vc) + (((long long)pid * a.Hkv + h) * a.s.page + row) * a.D;
    }
    return r;
}

__device__ __forceinline__ void clear_sums(const RopeArgs &a, int lane, int pid, int row) {
    for (int h = lane; h < a.Hkv; h += 32) a.acc[((long long)pid * a.Hkv + h) * a.s.page + row] = 0.f;
}

// Rows and strides on 16-byte boundaries, rot a multiple of 16. kFew (with norms): for
// tokens whose heads are few passes of a warp, where a token's slot and angles are what
// it costs: more warps an SM, and no weights kept in registers (7 heads of 128, 70,803
// tokens: 137 -> 111 us; 4 + 4 heads, 20,361 tokens: 41 -> 30; 64 heads, 14 passes,
// 92 -> 97, so those go the other way).
constexpr int kFewPasses = 4;
template <int D, bool kBf16, bool kF32, bool kInter, bool kNorm, bool kFew>
__global__ void __launch_bounds__(32 * kWarps, kNorm ? (kFew ? 7 : 4) : 0) k_rope_append(const RopeArgs a) {
    constexpr int kPerHead = D / 16, kHeads = 32 / kPerHead;  // lanes a head, heads a pass
    constexpr int kAngles = 8 / kHeads, kAhead = kNorm ? (kF32 || kFew ? 1 : 2) : kF32 ? 2 : 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= (long long)a.s.N * a.parts) return;
    const int n = (int)(w / a.parts), part = (int)(w - (long long)n * a.parts);
    const int i = lane % kPerHead, g = lane / kPerHead, half = a.rot >> 1;
    const int lo = kInter || i * 8 >= half ? i * 16 : i * 8;
    const int hi = kInter || i * 8 >= half ? i * 16 + 8 : half + i * 8;
    const bool place_turns = i * 8 < half;
    const int heads = a.Hq + 2 * a.Hkv;
    const int hb = (int)((long long)heads * part / a.parts), he = (int)((long long)heads * (part + 1) / a.parts);

    Vec8<kBf16, kF32> next[kNorm ? kAhead : 1][2];
    auto load = [&](Vec8<kBf16, kF32> (*x)[2], int h0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int hd = h0 + j * kHeads + g;
            if (hd < he) {
                const Head s = head_of(a, n, hd, false, -1, 0);
                x[j][0].load(s.src, s.at + lo);
                x[j][1].load(s.src, s.at + hi);
            }
        }
    };
    // (norms take longer than the turns alone: the next heads are on their way meanwhile,
    // the first ones while slot and angles are found; 103 -> 92 us for 14,839 tokens)
    if (kNorm) load(next, hb);
    int pid, row;
    const bool good = find_slot(a, n, lane, pid, row);
    if (good && a.acc && part == 0) clear_sums(a, lane, pid, row);
    float2 cs[8];
    {
        const double pos = (double)a.pos[n];
        float2 mine[kAngles];
#pragma unroll
        for (int j = 0; j < kAngles; ++j)
            mine[j] = place_turns ? turn_of(a, pos, i * 8 + g * kAngles + j) : make_float2(1.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int from = (j / kAngles) * kPerHead + i;
            cs[j].x = __shfl_sync(0xFFFFFFFFu, mine[j % kAngles].x, from);
            cs[j].y = __shfl_sync(0xFFFFFFFFu, mine[j % kAngles].y, from);
        }
    }
    float w0[8], w1[8];  // queries' weights (the few key heads load theirs when they come)
    if (kNorm && !kFew) {
        weights8<kBf16>(a, a.qw, lo, w0);
        weights8<kBf16>(a, a.qw, hi, w1);
    }
    for (int h0 = hb; h0 < he; h0 += kHeads * kAhead) {
        Vec8<kBf16, kF32> r[kAhead][2];
        if constexpr (kNorm) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                r[j][0] = next[j][0];
                r[j][1] = next[j][1];
            }
            load(next, h0 + kHeads * kAhead);
        } else {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int hd = h0 + j * kHeads + g;
                if (hd < he) {
                    const Head s = head_of(a, n, hd, good, pid, row);
                    r[j][0].load(s.src, s.at + lo);
                    r[j][1].load(s.src, s.at + hi);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int hd = h0 + j * kHeads + g;
            if (!kNorm && hd >= he) continue;
            float x0[8], x1[8];
            r[j][0].unpack(x0);
            r[j][1].unpack(x1);
            if (kNorm) {  // (the whole warp: lanes past the last head take part)
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], sum));
#pragma unroll
                for (int o = kPerHead / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                float eps = a.eps;
                const bool far = hd < min(he, a.Hq + a.Hkv) && out_of_range(a, sum);
                if (__any_sync(0xFFFFFFFFu, far)) {
                    float top = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
#pragma unroll
                    for (int o = kPerHead / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const float up = far ? scale_of(a, top, D) : 1.f;
                    sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x0[e] *= up;
                        x1[e] *= up;
                        sum = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], sum));
                    }
#pragma unroll
                    for (int o = kPerHead / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    eps = eps * up * up;
                }
                if (hd >= he) continue;
                const float f = norm_of(sum, D, eps);
                if (!kFew && hd < a.Hq) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x0[e] *= f * w0[e];
                        x1[e] *= f * w1[e];
                    }
                } else if (hd < a.Hq + a.Hkv) {
                    const void *hw = kFew && hd < a.Hq ? a.qw : a.kw;
                    float k0[8], k1[8];
                    weights8<kBf16>(a, hw, lo, k0);
                    weights8<kBf16>(a, hw, hi, k1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x0[e] *= f * k0[e];
                        x1[e] *= f * k1[e];
                    }
                }
            }
            const Head s = head_of(a, n, hd, good, pid, row);
            if (s.turn && place_turns) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &p = kInter ? (e < 4 ? x0[2 * e] : x1[2 * e - 8]) : x0[e];
                    float &q = kInter ? (e < 4 ? x0[2 * e + 1] : x1[2 * e - 7]) : x1[e];
                    const float u = p, v = q;
                    p = u * cs[e].x - v * cs[e].y;
                    q = v * cs[e].x + u * cs[e].y;
                }
            }
            if (s.dst) {
                store8<kBf16>(s.dst + lo, x0);
                store8<kBf16>(s.dst + hi, x1);
            }
        }
    }
    if (w == 0) check_lengths(a, lane);
}

// Any alignment and any even rot: a lane takes a pair (or two elements past
// rot) at a time.
template <bool kBf16, bool kF32, bool kInter, bool kNorm>
__global__ void __launch_bounds__(32 * kWarps) k_rope_any(const RopeArgs a) {
    __shared__ float2 table[kWarps][64];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= (long long)a.s.N * a.parts) return;
    const int n = (int)(w / a.parts), part = (int)(w - (long long)n * a.parts), half = a.rot >> 1;
    const int heads = a.Hq + 2 * a.Hkv;
    const int hb = (int)((long long)heads * part / a.parts), he = (int)((long long)heads * (part + 1) / a.parts);
    int pid, row;
    const bool good = find_slot(a, n, lane, pid, row);
    if (good && a.acc && part == 0) clear_sums(a, lane, pid, row);
    float2 *cs = table[threadIdx.x >> 5];
    const double pos = (double)a.pos[n];
    for (int i = lane; i < half; i += 32) cs[i] = turn_of(a, pos, i);
    __syncwarp();
    for (int hd = hb; hd < he; ++hd) {
        const Head s = head_of(a, n, hd, good, pid, row);
        const void *w = hd < a.Hq ? a.qw : a.kw;
        float f = 1.f, up = 1.f;
        if (kNorm && s.turn) {
            auto squares = [&](float &top) {
                float sum = 0.f;
                top = 0.f;
                for (int i = lane; i < a.D; i += 32) {
                    const float x = load1<kBf16, kF32>(s.src, s.at + i) * up;
                    sum = fmaf(x, x, sum);
                    top = fmaxf(top, fabsf(x));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                }
                return sum;
            };
            float top, sum = squares(top);
            if (out_of_range(a, sum)) {
                up = scale_of(a, top, a.D);
                sum = squares(top);
            }
            f = norm_of(sum, a.D, a.eps * up * up);
        }
        for (int i = lane; i < a.D / 2; i += 32) {
            const bool t = i < half;
            const int lo = kInter || !t ? 2 * i : i, hi = kInter || !t ? 2 * i + 1 : half + i;
            float u = load1<kBf16, kF32>(s.src, s.at + lo), v = load1<kBf16, kF32>(s.src, s.at + hi);
            if (kNorm && s.turn) {
                u = u * up * (f * weight1<kBf16>(a, w, lo));
                v = v * up * (f * weight1<kBf16>(a, w, hi));
            }
            if (s.turn && t) {
                const float x = u;
                u = x * cs[i].x - v * cs[i].y;
                v = v * cs[i].x + x * cs[i].y;
            }
            if (s.dst) {
                s.dst[lo] = from_f32<kBf16>(u);
                s.dst[hi] = from_f32<kBf16>(v);
            }
        }
    }
    if (w == 0) check_lengths(a, lane);
}

template <bool kBf16, bool kF32, bool kInter, bool kNorm>
cudaError_t run(const RopeArgs &a, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)a.s.N * a.parts + kWarps - 1) / kWarps)), block(32 * kWarps);
    const bool few = kNorm && (a.Hq + 2 * a.Hkv) * (a.D / 16) <= 32 * kFewPasses;
    return launch(!vec ? k_rope_any<kBf16, kF32, kInter, kNorm>
                  : a.D == 64 ? (few ? k_rope_append<64, kBf16, kF32, kInter, kNorm, kNorm>
                                     : k_rope_append<64, kBf16, kF32, kInter, kNorm, false>)
                              : (few ? k_rope_append<128, kBf16, kF32, kInter, kNorm, kNorm>
                                     : k_rope_append<128, kBf16, kF32, kInter, kNorm, false>),
                  grid, block, 0, st, true, a);
}

template <bool kNorm>
cudaError_t run(const RopeArgs &a, bool bf16, bool f32, bool inter, bool vec, cudaStream_t st) {
    if (inter)
        return bf16 ? (f32 ? run<true, true, true, kNorm>(a, vec, st) : run<true, false, true, kNorm>(a, vec, st))
                    : (f32 ? run<false, true, true, kNorm>(a, vec, st) : run<false, false, true, kNorm>(a, vec, st));
    return bf16 ? (f32 ? run<true, true, false, kNorm>(a, vec, st) : run<true, false, false, kNorm>(a, vec, st))
                : (f32 ? run<false, true, false, kNorm>(a, vec, st) : run<false, false, false, kNorm>(a, vec, st));
}

}  // namespace
}  // namespace attn

cudaError_t launch_rope_append(const AttnCache &c, const AttnSeqs &s, const RopeIn &q,
                               const RopeIn &k, const RopeIn &v, int in_f32, int Hq,
                               const int32_t *pos, const double *inv_freq, int rot,
                               bool interleaved, float mscale, void *q_out, float *acc,
                               int32_t *status, cudaStream_t st, const RopeNorm *norm) {
    using namespace attn;
    int lpage = 0;
    while ((1 << lpage) < c.page) ++lpage;
    RopeArgs a;
    a.s = Seqs{s.table, s.ctx, s.cu, s.B, s.N, 0, s.max_pages, c.page, lpage, 0};
    a.q = q.p; a.k = k.p; a.v = v.p;
    a.qs = q.stride; a.ks = k.stride; a.vs = v.stride;
    a.Hq = Hq; a.Hkv = c.Hkv; a.D = c.D; a.rot = rot; a.pages = c.pages;
    a.pos = pos; a.inv_freq = inv_freq; a.mscale = mscale;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.kc = static_cast<uint16_t *>(c.k);
    a.vc = static_cast<uint16_t *>(c.v);
    a.acc = acc; a.status = status;
    a.qw = norm ? norm->qw : nullptr;
    a.kw = norm ? norm->kw : nullptr;
    a.w_f32 = norm ? norm->w_f32 : 0;
    a.eps = norm ? norm->eps : 0.f;
    a.low = a.eps * (float)c.D >= kLowSum ? 0.f : kLowSum;
    const int esize = in_f32 ? 4 : 2;
    auto vec = [&](const RopeIn &r) {
        return reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && r.stride * esize % 16 == 0;
    };
    const bool v8 = vec(q) && vec(k) && vec(v) && rot % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.qw) % 16 == 0 && reinterpret_cast<uintptr_t>(a.kw) % 16 == 0;
    // Warps a token: enough to give every SM some when tokens are few, each with
    // at least one pass over heads.
    const int heads = Hq + 2 * c.Hkv, pass = v8 ? 32 / (c.D / 16) : 1;
    const int most = (heads + pass - 1) / pass, want = (sm_count() * kFill + s.N - 1) / s.N;
    a.parts = want < most ? want : most;
    return norm ? run<true>(a, c.bf16, in_f32, interleaved, v8, st)
                : run<false>(a, c.bf16, in_f32, interleaved, v8, st);
}

}  // namespace qmv
