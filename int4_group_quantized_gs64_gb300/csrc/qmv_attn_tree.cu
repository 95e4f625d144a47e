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
#include "qmv_attn_join.cuh"
#include "qmv_attn_plan.cuh"
#include "qmv_attn_rows.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

template <int D, bool kBf16>
cudaError_t run_tree(const AttnCache &c, const TreeArgs &a, int max_rows, cudaStream_t st) {
    cudaError_t e = a.rows == kRows ? run_rows<D, kBf16, false>(c, a, st) : launch_tree_tc(c, a, st);
    if (e == cudaSuccess)
        e = run_join<D, kBf16, false>(a, a.rows > kRows, max_rows, (max_rows + a.rows - 1) / a.rows, st);
    if (e == cudaSuccess && a.acc_out) e = launch_tree_weights(c, a, max_rows, st);
    return e;
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

bool encode_heads(CUtensorMap *map, const void *q, int N, int Hq, int D, long long q_stride, int heads,
                  int tokens) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[4] = {128, (cuuint64_t)Hq, (cuuint64_t)N, (cuuint64_t)D / 64};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2, 128};
    cuuint32_t box[4] = {128, (cuuint32_t)heads, (cuuint32_t)tokens, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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
    const size_t slots = (size_t)attn_grid_max(rows) * 2 * rows;
    return (slots * (c.D + 2) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace attn

size_t attn_tree_ws_bytes(const AttnCache &c, int Hq, int B, int N, int max_draft, int max_pages,
                          bool acc) {
    (void)N;
    const int max_rows = max_draft * (Hq / c.Hkv);
    return attn::part_bytes(c, attn::rows_an_item(max_rows)) +
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
    a.rows = rows_an_item(max_rows);
    a.unit = a.rows == kRows ? kWarps * 16 * (128 / c.D) : 128;  // keys a unit
    const long long most = (long long)t.s.B * c.Hkv * ((max_rows + a.rows - 1) / a.rows) *
                           ((((long long)t.s.max_pages << lpage) + a.unit - 1) / a.unit);
    const int gmax = attn_grid_max(a.rows);
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
