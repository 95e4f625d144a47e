// qmv_attn.cuh - shared by the attention operators over a paged key/value
// cache: the cache's addressing, the sequences of a call, and PTX wrappers.
//
// A pool is [pages][Hkv][page][D] (16-bit), so that the page-size rows of one
// head are one contiguous block: a tile of keys is then one tensor-map copy.
// Token `slot` of sequence b is row slot % page of page table[b][slot / page].
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tc05.cuh"

namespace qmv {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Bits of the attention operators' status word.
constexpr int kStPage = 1;     // a page id outside [0, pages): its tokens were left out
constexpr int kStLength = 2;   // a sequence whose lengths do not fit: it was left out
constexpr int kStTimeout = 4;  // a bounded wait ran out: outputs not valid

__device__ __forceinline__ void set_status(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------ 16-bit types

template <bool kBf16>
__device__ __forceinline__ float to_f32(uint16_t v) {
    if (kBf16) return __uint_as_float((uint32_t)v << 16);
    return __half2float(__ushort_as_half(v));
}

template <bool kBf16>
__device__ __forceinline__ uint16_t from_f32(float v) {
    if (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    return __half_as_ushort(__float2half_rn(v));
}

// (lo, hi) rounded to 16 bits each, lo in the low half.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    if (kBf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (kBf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

__device__ __forceinline__ float ex2(float v) {
    float d;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
    return d;
}

// Pairs of floats in one 64-bit register, two operations an instruction.
__device__ __forceinline__ uint64_t pack_u32x2(uint32_t a, uint32_t b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
    return pack_u32x2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &a, float &b) {
    uint32_t x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// All exponent bits set: an infinity or a NaN, in either half.
template <bool kBf16>
__device__ __forceinline__ bool nonfinite2(uint32_t v) {
    const uint32_t m = kBf16 ? 0x7F80u : 0x7C00u;
    return (v & m) == m || ((v >> 16) & m) == m;
}

// ------------------------------------------------------------------ the sequences of a call

struct Seqs {
    const int32_t *table;  // [B][max_pages]
    const int32_t *ctx;    // [B] cached tokens before the call
    const int32_t *cu;     // [B + 1] first new token of each sequence
    int B, N, max_draft, max_pages, page, lpage;  // page = 1 << lpage
    int min_draft;  // sequences of fewer new tokens count as empty
};

struct Seq {
    int ctx, first, T;  // cached tokens, first new token's index, new tokens (0: none, or not valid)
};

// A sequence whose new tokens do not lie inside [0, N), outnumber max_draft
// (0: any number), or do not fit its row of the table counts as empty.
__device__ __forceinline__ Seq get_seq(const Seqs &s, int b, bool &ok) {
    Seq q;
    q.ctx = s.ctx[b];
    q.first = s.cu[b];
    const int end = s.cu[b + 1];
    ok = q.ctx >= 0 && q.first >= 0 && end >= q.first && end <= s.N &&
         (s.max_draft == 0 || end - q.first <= s.max_draft) &&
         (long long)q.ctx + (end - q.first) <= ((long long)s.max_pages << s.lpage);
    q.T = ok && end - q.first >= s.min_draft ? end - q.first : 0;
    if (!ok) q.ctx = 0;
    return q;
}

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                          int c2, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc05::smem_addr(mbar))
        : "memory");
}

// The same, its lines the first to leave L2 (data read once).
__device__ __forceinline__ void tma_load3_once(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                               int c2, uint64_t *mbar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc05::smem_addr(mbar)),
        "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t *mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                     tc05::smem_addr(mbar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc05::smem_addr(mbar))
                 : "memory");
}

// One poll of a barrier's phase (it may suspend the thread for a short while).
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ void prefetch_tmap(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// d += A(16x16, row) * B(16x8, col), fp32 accumulators.
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if (kBf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

}  // namespace attn
}  // namespace qmv
