// qmv_window.cu - causal attention of new tokens over a paged cache, with a
// sliding window and a few first tokens that stay visible.
//
// The token at slot p sees the slots j <= p with j > p - window or j < sinks;
//     x_j = scale * q . k_j,   o = sum_j exp(x_j - M) v_j / sum_j exp(x_j - M)
// as in qmv_attn_tree.cu. The rows of a key/value head are its tokens times G
// query heads; some of them are an item, and its keys are the union of what its
// rows see, in two stretches that are put side by side (Reach): first tokens, and
// those from the first row's window to the last row's slot. Units that every row
// sees whole need no mask; the others (the edges) are masked row by row.
// Units are shared out evenly over the blocks, so a prompt's early rows (short
// reach) and late ones, and sequences of any length, fill the GPU alike.
//
// Up to 16 rows a sequence: k_attn_rows (warp MMA, bound by the copy of keys
// and values); more: k_window_tc (tcgen05).
#include <math.h>
#include <string.h>

#include <algorithm>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_join.cuh"
#include "qmv_attn_plan.cuh"
#include "qmv_attn_rows.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {

// Launches the tcgen05 kernel (qmv_window_tc.cu).
cudaError_t launch_window_tc(const AttnCache &c, const TreeArgs &a, cudaStream_t st);

namespace {

// Items of a head of a sequence of T new tokens.
long long items_a_head(const TreeArgs &a, long long T) {
    return ((T + a.tb - 1) / a.tb * a.hs + a.tpi - 1) / a.tpi;
}

// The rows of an item: few, or one tile of 128 or two (rows_an_item says which
// kernel they measured best on).
void set_rows(TreeArgs &a, int max_new) {
    a.max_rows = max_new * a.G;
    if (a.max_rows <= kRows) {  // all of a sequence's
        a.rows = kRows;
        a.tb = 1 << 30;
        a.hb = a.G;
        a.hs = a.tpi = 1;
    } else {
        a.hb = a.G < 128 ? a.G : 128;
        a.tb = 128 / a.hb;
        a.hs = (a.G + 127) / 128;
        a.tpi = max_new <= a.tb && a.hs == 1 ? 1 : 2;
        a.rows = 128 * a.tpi;
    }
    a.hinv = (uint32_t)(((1ull << 32) + a.hb - 1) / a.hb);
}

// Rows and keys of a unit; a.s, a.G, a.window and a.sinks are set.
void set_units(TreeArgs &a, const AttnCache &c) {
    set_rows(a, a.s.max_draft);
    a.unit = a.rows == kRows ? kWarps * 16 * (128 / c.D) : 128;  // keys a unit
    a.lunit = 0;
    while ((1 << a.lunit) < a.unit) ++a.lunit;
    a.align = a.rows == kRows ? 16 : c.page < 128 ? c.page : 128;
}

// Units of a call, at most: the items of B sequences at their bound, or of N tokens (a
// sequence's last item may be short), each over what its tokens may see (Reach: first
// slots and those from the first token's window to the last token, each stretch to
// whole pieces of a.align slots), or over the table's row where that is less.
long long units_at_most(const TreeArgs &a, int Hkv) {
    const long long items = std::min(a.s.B * items_a_head(a, a.s.max_draft), items_a_head(a, a.s.N) + a.s.B);
    const long long tokens = std::min<long long>(a.s.max_draft, (long long)a.tpi * a.tb);
    const long long seen = (long long)a.window + a.sinks + tokens + 2 * a.align;
    const long long slots = std::min((long long)a.s.max_pages << a.s.lpage, seen);
    return items * Hkv * (((slots + a.unit - 1) >> a.lunit) + 2);
}

template <int D, bool kBf16>
cudaError_t run_window(const AttnCache &c, const TreeArgs &a, cudaStream_t st) {
    const bool few = a.rows == kRows;
    cudaError_t e = few ? run_rows<D, kBf16, true>(c, a, st) : launch_window_tc(c, a, st);
    if (e == cudaSuccess) e = run_join<D, kBf16, true>(a, !few, few ? a.max_rows : a.rows, items_a_head(a, a.s.max_draft), st);
    return e;
}

// Segments' sums, their maxima and sums of exponentials, and whose they are.
size_t part_floats(const AttnCache &c, int rows) {
    return (size_t)attn_grid_max(rows) * 2 * rows * (c.D + 2);
}

}  // namespace
}  // namespace attn

size_t attn_window_ws_bytes(const AttnCache &c, int Hq, int max_new) {
    attn::TreeArgs a;
    a.G = Hq / c.Hkv;
    attn::set_rows(a, max_new);
    const int rows = a.rows;
    const size_t n = attn::part_floats(c, rows) * 4 + (size_t)attn::attn_grid_max(rows) * 2 * sizeof(attn::PartInfo);
    return (n + 255) / 256 * 256;
}

// What the plan goes by.
static void plan_window(attn::TreeArgs &a, const AttnCache &c, const AttnSeqs &s, int Hq, int window, int sinks) {
    int lpage = 0;
    while ((1 << lpage) < c.page) ++lpage;
    a.s = attn::Seqs{s.table, s.ctx, s.cu, s.B, s.N, s.max_draft, s.max_pages, c.page, lpage, 0};
    a.G = Hq / c.Hkv;
    a.window = window;
    a.sinks = sinks;
    attn::set_units(a, c);
}

bool attn_window_fits(const AttnCache &c, const AttnSeqs &s, int Hq, int window, int sinks) {
    attn::TreeArgs a;
    plan_window(a, c, s, Hq, window, sinks);
    return attn::units_at_most(a, c.Hkv) / attn::attn_grid_max(a.rows) < 0x7FFFFFFFLL;
}

cudaError_t launch_attn_window(const AttnCache &c, const WindowCall &t, cudaStream_t st) {
    using namespace attn;
    TreeArgs a;
    memset(&a, 0, sizeof(a));
    plan_window(a, c, t.s, t.Hq, t.window, t.sinks);
    a.q = static_cast<const uint16_t *>(t.q);
    a.q_stride = t.q_stride;
    a.Hq = t.Hq; a.Hkv = c.Hkv; a.pages = c.pages;
    a.ginv = (uint32_t)(((1ull << 32) + a.G - 1) / a.G);
    // (k_attn_rows turns or clears the queries, k_window_tc the scores)
    a.sl2 = t.scale == 0.f ? 1.f : fabsf(t.scale) * kLog2e;
    a.qxor = t.scale < 0.f ? 0x80008000u : 0u;
    a.qand = t.scale == 0.f ? 0u : 0xFFFFFFFFu;
    a.flip = t.scale < 0.f ? -1.f : t.scale == 0.f ? 0.f : 1.f;
    a.o = t.o; a.o_f32 = t.o_f32; a.lse = t.lse;
    a.vpool = static_cast<const uint16_t *>(c.v);
    a.status = t.status;
    const int gmax = attn_grid_max(a.rows);
    a.grid = (int)std::min<long long>(units_at_most(a, c.Hkv), gmax);
    a.part_o = static_cast<float *>(t.ws);
    a.part_ml = a.part_o + (size_t)gmax * 2 * a.rows * c.D;
    a.info = reinterpret_cast<PartInfo *>(a.part_o + part_floats(c, a.rows));
    if (c.D == 64) return c.bf16 ? run_window<64, true>(c, a, st) : run_window<64, false>(c, a, st);
    return c.bf16 ? run_window<128, true>(c, a, st) : run_window<128, false>(c, a, st);
}

}  // namespace qmv
