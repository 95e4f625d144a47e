// qmv_rope.cu - rotary positions of new tokens and their append to the cache.
//
// A token at position p turns pair i of every query and key head by the angle
// p * inv_freq[i]:
//     (a, b) -> m * (a cos - b sin, b cos + a sin)
// with the pair at elements (i, i + rot/2), or (2i, 2i + 1) when interleaved;
// elements from rot on pass unchanged. The angle is formed in turns in 64
// bits and only its fraction is rounded to 32: at position 10^6 an fp32 angle
// would be off by hundredths of a radian, the fraction of a turn by 1e-10.
// All arithmetic on the elements is fp32, rounded once to the cache's type.
//
// It is bound by memory at many tokens and by latency at few, so each block
// takes a share of one token's heads (as many blocks a token as fill the GPU)
// and issues its loads before it forms the angles.
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
};

constexpr int kRopeThreads = 256;

// Eight consecutive elements as fp32, and back.
template <bool kBf16, bool kF32>
struct Vec8 {
    float x[8];
    __device__ __forceinline__ void load(const void *p, long long at) {
        if (kF32) {
            const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            const float4 a = __ldg(f), b = __ldg(f + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const uint4 u = __ldg(
                reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<kBf16>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2<kBf16>(x[0], x[1]), pack2<kBf16>(x[2], x[3]),
                       pack2<kBf16>(x[4], x[5]), pack2<kBf16>(x[6], x[7]));
    }
};

template <bool kBf16, bool kF32>
__device__ __forceinline__ float load1(const void *p, long long at) {
    return kF32 ? static_cast<const float *>(p)[at]
                : to_f32<kBf16>(static_cast<const uint16_t *>(p)[at]);
}

// kVec: rows and strides 16-byte aligned and rot a multiple of 16, so a
// thread takes 16 elements of a head as two vectors (the two halves of eight
// pairs, or 16 in a row). Otherwise a thread takes one pair (or two elements
// past rot) at a time.
template <bool kBf16, bool kF32, bool kVec, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) k_rope_append(const RopeArgs a) {
    extern __shared__ float2 cs[];  // [rot / 2] (cos, sin) times mscale
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int n = blockIdx.x / a.parts, part = blockIdx.x - n * a.parts;
    const int heads = a.Hq + 2 * a.Hkv, half = a.rot >> 1;
    const int per_head = kVec ? a.D / 16 : a.D / 2;
    const int units = heads * per_head;
    const int ub = (int)((long long)units * part / a.parts);
    const int ue = (int)((long long)units * (part + 1) / a.parts);
    // where the first vectors are, so that their loads are under way first
    auto source = [&](int u, const void *&p, long long &at, int &hd, int &lo, int &hi, bool &turn) {
        hd = u / per_head;
        const int i = u - hd * per_head;
        if (kVec) {
            if (!kInter && i < half / 8) {
                lo = i * 8;
                hi = half + i * 8;
                turn = true;
            } else {
                lo = i * 16;
                hi = lo + 8;
                turn = kInter && lo < a.rot;
            }
        } else {
            turn = i < half;
            lo = kInter || !turn ? 2 * i : i;
            hi = kInter || !turn ? 2 * i + 1 : half + i;
        }
        if (hd < a.Hq) {
            p = a.q;
            at = (long long)n * a.qs + (long long)hd * a.D;
        } else if (hd < a.Hq + a.Hkv) {
            p = a.k;
            at = (long long)n * a.ks + (long long)(hd - a.Hq) * a.D;
        } else {
            p = a.v;
            at = (long long)n * a.vs + (long long)(hd - a.Hq - a.Hkv) * a.D;
            turn = false;
        }
    };
    Vec8<kBf16, kF32> x0, x1;
    const void *p;
    long long at;
    int hd = 0, lo = 0, hi = 0;
    bool turn = false;
    int u = ub + threadIdx.x;
    if (kVec && u < ue) {
        source(u, p, at, hd, lo, hi, turn);
        x0.load(p, at + lo);
        x1.load(p, at + hi);
    }
    const double pos = (double)a.pos[n];
    for (int i = threadIdx.x; i < half; i += kRopeThreads) {
        double t = pos * (a.inv_freq[i] * 0.15915494309189533577);
        t -= floor(t);
        float s, c;
        sincospif(2.f * (float)t, &s, &c);
        cs[i] = make_float2(c * a.mscale, s * a.mscale);
    }
    // the token's sequence: how many sequences start at or before it
    int b = 0;
    for (int i = 0; i < a.s.B; i += kRopeThreads) {
        const int j = i + threadIdx.x;
        b += __syncthreads_count(j < a.s.B && a.s.cu[j] <= n);
    }
    b -= 1;  // (the barrier also publishes cs)
    bool ok = false;
    Seq q;
    q.ctx = q.first = q.T = 0;
    if (b >= 0) q = get_seq(a.s, b, ok);
    ok = ok && n - q.first < q.T;
    int pid = -1, row = 0;
    if (ok) {
        const int slot = q.ctx + n - q.first;
        pid = a.s.table[(long long)b * a.s.max_pages + (slot >> a.s.lpage)];
        row = slot & (a.s.page - 1);
    }
    const bool good = ok && (unsigned)pid < (unsigned)a.pages;
    if (threadIdx.x == 0 && part == 0 && !good) set_status(a.status, ok ? kStPage : kStLength);
    if (good && a.acc && part == 0)
        for (int h = threadIdx.x; h < a.Hkv; h += kRopeThreads)
            a.acc[((long long)pid * a.Hkv + h) * a.s.page + row] = 0.f;
    for (; u < ue; u += kRopeThreads) {
        if (u >= ub + kRopeThreads || !kVec) {
            source(u, p, at, hd, lo, hi, turn);
            if (kVec) {
                x0.load(p, at + lo);
                x1.load(p, at + hi);
            }
        }
        uint16_t *d;
        if (hd < a.Hq) {
            d = a.q_out + ((long long)n * a.Hq + hd) * a.D;
        } else {
            if (!good) continue;
            const int h = hd < a.Hq + a.Hkv ? hd - a.Hq : hd - a.Hq - a.Hkv;
            d = (hd < a.Hq + a.Hkv ? a.kc : a.vc) +
                (((long long)pid * a.Hkv + h) * a.s.page + row) * a.D;
        }
        if (kVec) {
            if (turn) {
                if (kInter) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = cs[lo / 2 + i], g = cs[lo / 2 + 4 + i];
                        const float a0 = x0.x[2 * i], b0 = x0.x[2 * i + 1];
                        x0.x[2 * i] = a0 * f.x - b0 * f.y;
                        x0.x[2 * i + 1] = b0 * f.x + a0 * f.y;
                        const float a1 = x1.x[2 * i], b1 = x1.x[2 * i + 1];
                        x1.x[2 * i] = a1 * g.x - b1 * g.y;
                        x1.x[2 * i + 1] = b1 * g.x + a1 * g.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = cs[lo + i];
                        const float a0 = x0.x[i], b0 = x1.x[i];
                        x0.x[i] = a0 * f.x - b0 * f.y;
                        x1.x[i] = b0 * f.x + a0 * f.y;
                    }
                }
            }
            x0.store(d + lo);
            x1.store(d + hi);
        } else {
            const float va = load1<kBf16, kF32>(p, at + lo), vb = load1<kBf16, kF32>(p, at + hi);
            float ra = va, rb = vb;
            if (turn) {
                const float2 f = cs[kInter ? lo / 2 : lo];
                ra = va * f.x - vb * f.y;
                rb = vb * f.x + va * f.y;
            }
            d[lo] = from_f32<kBf16>(ra);
            d[hi] = from_f32<kBf16>(rb);
        }
    }
}

template <bool kBf16, bool kF32, bool kVec>
cudaError_t run(const RopeArgs &a, bool inter, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)a.s.N * a.parts)), block(kRopeThreads);
    const size_t smem = (size_t)(a.rot / 2) * sizeof(float2);
    return inter ? launch(k_rope_append<kBf16, kF32, kVec, true>, grid, block, smem, st, true, a)
                 : launch(k_rope_append<kBf16, kF32, kVec, false>, grid, block, smem, st, true, a);
}

}  // namespace
}  // namespace attn

cudaError_t launch_rope_append(const AttnCache &c, const AttnSeqs &s, const RopeIn &q,
                               const RopeIn &k, const RopeIn &v, int in_f32, int Hq,
                               const int32_t *pos, const double *inv_freq, int rot,
                               bool interleaved, float mscale, void *q_out, float *acc,
                               int32_t *status, cudaStream_t st) {
    using namespace attn;
    int lpage = 0;
    while ((1 << lpage) < c.page) ++lpage;
    RopeArgs a;
    a.s = Seqs{s.table, s.ctx, s.cu, s.B, s.N, 0, s.max_pages, c.page, lpage};
    a.q = q.p; a.k = k.p; a.v = v.p;
    a.qs = q.stride; a.ks = k.stride; a.vs = v.stride;
    a.Hq = Hq; a.Hkv = c.Hkv; a.D = c.D; a.rot = rot; a.pages = c.pages;
    a.pos = pos; a.inv_freq = inv_freq; a.mscale = mscale;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.kc = static_cast<uint16_t *>(c.k);
    a.vc = static_cast<uint16_t *>(c.v);
    a.acc = acc; a.status = status;
    const int esize = in_f32 ? 4 : 2;
    auto vec = [&](const RopeIn &r) {
        return reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && r.stride * esize % 16 == 0;
    };
    const bool v8 = vec(q) && vec(k) && vec(v) && rot % 16 == 0;
    const int units = (Hq + 2 * c.Hkv) * (v8 ? c.D / 16 : c.D / 2);
    // blocks a token: enough to give every SM one when tokens are few, each
    // with at least one pass of its threads
    const int most = (units + kRopeThreads - 1) / kRopeThreads, want = (sm_count() + s.N - 1) / s.N;
    a.parts = want < most ? want : most;
    if (c.bf16)
        return in_f32 ? (v8 ? run<true, true, true>(a, interleaved, st)
                            : run<true, true, false>(a, interleaved, st))
                      : (v8 ? run<true, false, true>(a, interleaved, st)
                            : run<true, false, false>(a, interleaved, st));
    return in_f32 ? (v8 ? run<false, true, true>(a, interleaved, st)
                        : run<false, true, false>(a, interleaved, st))
                  : (v8 ? run<false, false, true>(a, interleaved, st)
                        : run<false, false, false>(a, interleaved, st));
}

}  // namespace qmv
