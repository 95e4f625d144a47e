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
// A warp takes one token (or a share of its heads, so that few tokens fill the
// GPU too). D / 16 lanes share a head, 16 elements each: a lane has the same
// place in every head that it meets, and so the same eight angles, which stay
// in registers: no shared memory, no barrier. The lanes that share a place
// divide its eight angles and exchange them. What bounds it is the copy: 16,372
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

// Rows and strides on 16-byte boundaries, rot a multiple of 16.
template <int D, bool kBf16, bool kF32, bool kInter>
__global__ void __launch_bounds__(32 * kWarps) k_rope_append(const RopeArgs a) {
    constexpr int kPerHead = D / 16, kHeads = 32 / kPerHead;  // lanes a head, heads a pass
    constexpr int kAngles = 8 / kHeads, kAhead = kF32 ? 2 : 4;
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
    for (int h0 = hb; h0 < he; h0 += kHeads * kAhead) {
        Vec8<kBf16, kF32> r[kAhead][2];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int hd = h0 + j * kHeads + g;
            if (hd < he) {
                const Head s = head_of(a, n, hd, good, pid, row);
                r[j][0].load(s.src, s.at + lo);
                r[j][1].load(s.src, s.at + hi);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int hd = h0 + j * kHeads + g;
            if (hd >= he) continue;
            const Head s = head_of(a, n, hd, good, pid, row);
            float x0[8], x1[8];
            r[j][0].unpack(x0);
            r[j][1].unpack(x1);
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
template <bool kBf16, bool kF32, bool kInter>
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
        for (int i = lane; i < a.D / 2; i += 32) {
            const bool t = i < half;
            const int lo = kInter || !t ? 2 * i : i, hi = kInter || !t ? 2 * i + 1 : half + i;
            float u = load1<kBf16, kF32>(s.src, s.at + lo), v = load1<kBf16, kF32>(s.src, s.at + hi);
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

template <bool kBf16, bool kF32, bool kInter>
cudaError_t run(const RopeArgs &a, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)a.s.N * a.parts + kWarps - 1) / kWarps)), block(32 * kWarps);
    return launch(!vec        ? k_rope_any<kBf16, kF32, kInter>
                  : a.D == 64 ? k_rope_append<64, kBf16, kF32, kInter>
                              : k_rope_append<128, kBf16, kF32, kInter>,
                  grid, block, 0, st, true, a);
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
    a.s = Seqs{s.table, s.ctx, s.cu, s.B, s.N, 0, s.max_pages, c.page, lpage, 0};
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
    // Warps a token: enough to give every SM some when tokens are few, each with
    // at least one pass over heads.
    const int heads = Hq + 2 * c.Hkv, pass = v8 ? 32 / (c.D / 16) : 1;
    const int most = (heads + pass - 1) / pass, want = (sm_count() * kFill + s.N - 1) / s.N;
    a.parts = want < most ? want : most;
    if (interleaved)
        return c.bf16 ? (in_f32 ? run<true, true, true>(a, v8, st) : run<true, false, true>(a, v8, st))
                      : (in_f32 ? run<false, true, true>(a, v8, st) : run<false, false, true>(a, v8, st));
    return c.bf16 ? (in_f32 ? run<true, true, false>(a, v8, st) : run<true, false, false>(a, v8, st))
                  : (in_f32 ? run<false, true, false>(a, v8, st) : run<false, false, false>(a, v8, st));
}

}  // namespace qmv
