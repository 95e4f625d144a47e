// qmv_attn_join.cuh - adds up the segments of the attention kernels' items.
#pragma once

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_plan.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

// Adds up the segments of an item that several blocks shared, in key order,
// kXb blocks' segments at a time (their loads in flight together). A warp takes
// 8 rows: lane l has row l % 8 and every fourth group of 4 columns, kCols of
// them (the rest of a row's columns are other warps'). kSplit warps share a
// long row of segments and meet in shared memory. The call's inputs are older
// than its first kernel, so everything up to the segments is read before the
// wait for it. What bounds it is latency: 7.6 us from cold for the 304 blocks'
// parts of 512 items (2.5 MB), 13.5 us for 31 MB of 128 items of 256 rows.
//
// Trees (kWin false): a block an item, which works out the item's segments from the
// lengths. kWin: items may be many thousands, of which only those that a block's
// share ends inside have segments, so a block here goes with a block of the
// attention, which has left word of its segments (PartInfo), and joins the item
// whose first segment that one had.
template <int D, int kCols, int kXb, int kSplit, bool kWin>
__global__ void __launch_bounds__(128 * kSplit) k_attn_join(const TreeArgs a, bool bf16) {
    constexpr int kParts = D / 16 / kCols;  // warps a row
    __shared__ long long scan[kWin ? 1 : 8 * kSplit];
    __shared__ float meet[kSplit > 1 ? (kSplit - 1) * 128 * (kCols * 4 + 2) : 1];
    int b, h, rb, c0, c1, first = 0;  // first: which of block c0's two segments
    long long i0 = 0, quota = 1;
    Seq q;
    bool ok;
    if constexpr (kWin) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        c0 = blockIdx.x;
        const PartInfo s0 = a.info[c0 * 2], s1 = a.info[c0 * 2 + 1];
        first = s1.n > 0 && s1.u0 == 0;
        const PartInfo &s = first ? s1 : s0;
        if (s.n == 0 || s.u0 != 0) return;
        b = s.b;
        h = s.h;
        rb = s.rb;
        c1 = c0 + (s.nu - s.n + s.quota - 1) / s.quota;
        q = get_seq(a.s, b, ok);
    } else {
        b = blockIdx.x / a.Hkv;
        h = blockIdx.x - b * a.Hkv;
        rb = blockIdx.y;
        q = get_seq(a.s, b, ok);
        const int nu = key_units(q, a.unit), nrb = row_blocks(q, a.G, a.rows);
        long long before;
        const long long total = count_units<128 * kSplit>(a, b, scan, before);
        quota = (total + a.grid - 1) / a.grid;
        i0 = before + ((long long)h * nrb + rb) * nu;
        const long long i1 = i0 + nu;
        const bool any = q.T > 0 && rb < nrb;
        c0 = any ? (int)(i0 / quota) : 0;
        c1 = any ? (int)((i1 - 1) / quota) : 0;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (c0 == c1) return;  // nothing here, or one segment, written by its block
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = blockIdx.z * 4 + (warp & 3), split = warp >> 2;
    const int r = (w / kParts) * 8 + (lane & 7), col0 = (w % kParts) * (kCols * 16) + (lane >> 3) * 4;
    // the row's token and query head
    int t, g;
    bool have_row;
    if constexpr (kWin) {
        have_row = tile_row(a, q, rb * a.tpi + (r >> 7), r & 127, t, g);
    } else {
        const int rr = rb * a.rows + r;
        t = div_g(a, rr);
        g = rr - t * a.G;
        have_row = r < min(a.rows, q.T * a.G - rb * a.rows);
    }
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
            const int x = x0 + j;
            const int last = kWin ? (x == c0 ? first : 0) : (long long)x * quota >= i0 ? 0 : 1;
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
    const long long row = (long long)(q.first + t) * a.Hq + h * a.G + g;
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

// many rows: a warp 8 of them whole, two blocks' segments at a time; few rows:
// a warp a part of 8 rows, four warps sharing the blocks' segments where items
// are so few that each has many (8 items of 38 segments: 10.8 -> 5.8 us). nrb:
// blocks of rows a sequence, at most.
template <int D, bool kBf16, bool kWin>
cudaError_t run_join(const TreeArgs &a, bool many, int max_rows, long long nrb, cudaStream_t st) {
    const bool longs = a.grid > 8 * nrb * a.s.B * a.Hkv;
    const int warps = ((max_rows < a.rows ? max_rows : a.rows) + 7) / 8 * (many ? 1 : D / 32);
    const dim3 grid = kWin ? dim3(a.grid, 1, (warps + 3) / 4)
                           : dim3(a.s.B * a.Hkv, (unsigned)nrb, (warps + 3) / 4);
    return many  ? launch(k_attn_join<D, D / 16, 2, 1, kWin>, grid, dim3(128), 0, st, true, a, (bool)kBf16)
           : longs ? launch(k_attn_join<D, 2, 5, 4, kWin>, grid, dim3(512), 0, st, true, a, (bool)kBf16)
                   : launch(k_attn_join<D, 2, 8, 1, kWin>, grid, dim3(128), 0, st, true, a, (bool)kBf16);
}

}  // namespace
}  // namespace attn
}  // namespace qmv
