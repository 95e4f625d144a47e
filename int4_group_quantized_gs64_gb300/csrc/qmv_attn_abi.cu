// qmv_attn_abi.cu - the extern "C" entry points of the attention operators
// (include/qmv.h): host-side checks, then the launchers of qmv_attn.h. As in
// qmv_abi.cu, a negative status means that nothing was enqueued.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/qmv.h"
#include "qmv_attn.h"

namespace {

constexpr int kMaxDraft = 256;
constexpr int kMaxHeads = 1024;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t cs(qmv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? QMV_OK : QMV_ECUDA; }

bool page_ok(int page) { return page >= 16 && page <= 256 && !(page & (page - 1)); }

int check_cache(const qmv_attn_cache *c) {
    if (!c || !c->k || !c->v || c->pages < 1 || c->Hkv < 1 || c->Hkv > kMaxHeads) return QMV_EINVAL;
    if (c->dtype != QMV_BF16 && c->dtype != QMV_F16) return QMV_EINVAL;
    if (c->D != 64 && c->D != 128) return QMV_ESHAPE;
    if (!page_ok(c->page)) return QMV_ESHAPE;
    if ((int64_t)c->pages * c->Hkv * c->page >= (int64_t)1 << 31) return QMV_ESHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return QMV_EALIGN;
    return QMV_OK;
}

// A batch of sequences against a table of max_pages pages each.
int check_batch(const qmv_attn_cache *c, int B, int max_pages) {
    if (B < 0 || max_pages < 1) return QMV_EINVAL;
    if ((int64_t)B * c->Hkv > 65535 || (int64_t)max_pages * c->page > (int64_t)1 << 30)
        return QMV_ESHAPE;
    return QMV_OK;
}

qmv::AttnCache cache(const qmv_attn_cache *c) {
    return qmv::AttnCache{c->k, c->v, c->pages, c->Hkv, c->page, c->D, c->dtype == QMV_BF16};
}

bool heads_ok(const qmv_attn_cache *c, int Hq) {
    return Hq >= 1 && Hq <= kMaxHeads && Hq % c->Hkv == 0;
}

// A bound of a sequence's new tokens: its rows a key/value head are counted in 31 bits.
bool new_ok(const qmv_attn_cache *c, int Hq, int max_new) {
    return max_new >= 1 && max_new <= 1 << 22 && (int64_t)max_new * (Hq / c->Hkv) <= (int64_t)1 << 30;
}

// A pool of pages and a table of n rows.
int check_pages(int pages, int page, int n, int max_pages) {
    if (pages < 1 || n < 0 || max_pages < 1) return QMV_EINVAL;
    if (!page_ok(page) || pages > 1 << 30 || n > 65535 || (int64_t)max_pages * page > (int64_t)1 << 30 ||
        (int64_t)n * max_pages > INT32_MAX)
        return QMV_ESHAPE;
    return QMV_OK;
}

// An int32 array of a call.
struct Ints {
    const int32_t *p;
    int64_t n;
};
// Blocks write `out` while others still read or write the `rest`: no shared bytes.
bool apart(const Ints &out, std::initializer_list<Ints> rest) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p), e = a + 4 * (uintptr_t)out.n;
    for (const Ints &r : rest) {
        const uintptr_t b = reinterpret_cast<uintptr_t>(r.p);
        if (a < b + 4 * (uintptr_t)r.n && b < e) return false;
    }
    return true;
}

// Both rotary appends; norm null: without norms.
int rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                const qmv::RopeNorm *norm, int w_dtype, const int32_t *pos, const double *inv_freq,
                int rot, int interleaved, float mscale, const int32_t *table, int max_pages,
                const int32_t *ctx, const int32_t *cu, int B, int N, void *q_out, float *acc,
                int32_t *status, qmv_stream_t stream) {
    int r = check_cache(c);
    if (r) return r;
    if ((r = check_batch(c, B, max_pages))) return r;
    if (N < 0 || !heads_ok(c, Hq) || rot < 2 || rot > c->D || rot % 2 || !isfinite(mscale))
        return QMV_EINVAL;
    if (in_dtype != QMV_F32 && in_dtype != c->dtype) return QMV_EINVAL;
    if (norm && ((w_dtype != QMV_F32 && w_dtype != c->dtype) || !isfinite(norm->eps) || norm->eps < 0.f))
        return QMV_EINVAL;
    if (N > 1 << 22) return QMV_ESHAPE;
    if (q_stride < (int64_t)Hq * c->D || k_stride < (int64_t)c->Hkv * c->D ||
        v_stride < (int64_t)c->Hkv * c->D)
        return QMV_ESHAPE;
    if (B == 0 || N == 0) return QMV_OK;
    if (!q || !k || !v || !pos || !inv_freq || !table || !ctx || !cu || !q_out) return QMV_EINVAL;
    const uintptr_t e = in_dtype == QMV_F32 ? 4 : 2;
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(pos, 4) ||
        !aligned(inv_freq, 8) || !aligned(table, 4) || !aligned(ctx, 4) || !aligned(cu, 4) ||
        !aligned(q_out, 16) || !aligned(acc, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    const uintptr_t we = norm && norm->w_f32 ? 4 : 2;
    if (norm && (!aligned(norm->qw, we) || !aligned(norm->kw, we))) return QMV_EALIGN;
    return from_cuda(qmv::launch_rope_append(
        cache(c), qmv::AttnSeqs{table, ctx, cu, B, N, 0, max_pages}, qmv::RopeIn{q, q_stride},
        qmv::RopeIn{k, k_stride}, qmv::RopeIn{v, v_stride}, in_dtype == QMV_F32, Hq, pos, inv_freq,
        rot, interleaved != 0, mscale, q_out, acc, status, cs(stream), norm));
}

}  // namespace

extern "C" {

int attn_rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                     int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                     const int32_t *pos, const double *inv_freq, int rot, int interleaved,
                     float mscale, const int32_t *table, int max_pages, const int32_t *ctx,
                     const int32_t *cu, int B, int N, void *q_out, float *acc, int32_t *status,
                     qmv_stream_t stream) {
    return rope_append(c, q, q_stride, k, k_stride, v, v_stride, in_dtype, Hq, nullptr, QMV_F32, pos,
                       inv_freq, rot, interleaved, mscale, table, max_pages, ctx, cu, B, N, q_out,
                       acc, status, stream);
}

int attn_norm_rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                          int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                          const void *q_weight, const void *k_weight, int w_dtype, float eps,
                          const int32_t *pos, const double *inv_freq, int rot, int interleaved,
                          float mscale, const int32_t *table, int max_pages, const int32_t *ctx,
                          const int32_t *cu, int B, int N, void *q_out, float *acc,
                          int32_t *status, qmv_stream_t stream) {
    const qmv::RopeNorm norm{q_weight, k_weight, w_dtype == QMV_F32, eps};
    return rope_append(c, q, q_stride, k, k_stride, v, v_stride, in_dtype, Hq, &norm, w_dtype, pos,
                       inv_freq, rot, interleaved, mscale, table, max_pages, ctx, cu, B, N, q_out,
                       acc, status, stream);
}

size_t attn_tree_workspace_bytes(const qmv_attn_cache *c, int Hq, int B, int N, int max_draft,
                                 int max_pages, int weights) {
    if (check_cache(c) || check_batch(c, B, max_pages) || !heads_ok(c, Hq) || N < 0 ||
        max_draft < 1 || max_draft > kMaxDraft)
        return 0;
    return qmv::attn_tree_ws_bytes(cache(c), Hq, B, N, max_draft, max_pages, weights != 0);
}

int attn_tree(const qmv_attn_cache *c, const void *q, int64_t q_stride, int Hq,
              const int32_t *table, int max_pages, const int32_t *ctx, const int32_t *cu, int B,
              int N, int max_draft, const uint32_t *mask, int mask_words, float scale, void *o,
              int o_dtype, float *lse, const float *acc_in, float *acc_out, float decay,
              int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream) {
    int r = check_cache(c);
    if (r) return r;
    if ((r = check_batch(c, B, max_pages))) return r;
    if (N < 0 || !heads_ok(c, Hq) || max_draft < 1 || !isfinite(scale) || !isfinite(decay))
        return QMV_EINVAL;
    if (o_dtype != QMV_F32 && o_dtype != c->dtype) return QMV_EINVAL;
    if (max_draft > kMaxDraft) return QMV_ESHAPE;
    if (mask && (mask_words < 1 || mask_words > kMaxDraft / 32 || mask_words * 32 < max_draft))
        return QMV_ESHAPE;
    if (q_stride < (int64_t)Hq * c->D) return QMV_ESHAPE;
    if (acc_in && !acc_out) return QMV_EINVAL;
    if (B == 0 || N == 0) return QMV_OK;
    if (!q || !table || !ctx || !cu || !o || !lse) return QMV_EINVAL;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(table, 4) || !aligned(ctx, 4) ||
        !aligned(cu, 4) || !aligned(mask, 4) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(acc_in, 4) || !aligned(acc_out, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    if (!ws || !aligned(ws, 256) ||
        ws_bytes < qmv::attn_tree_ws_bytes(cache(c), Hq, B, N, max_draft, max_pages,
                                           acc_out != nullptr))
        return QMV_EWORKSPACE;
    qmv::TreeCall t;
    t.s = qmv::AttnSeqs{table, ctx, cu, B, N, max_draft, max_pages};
    t.q = q; t.q_stride = q_stride; t.Hq = Hq;
    t.mask = mask; t.words = mask_words; t.scale = scale;
    t.o = o; t.o_f32 = o_dtype == QMV_F32; t.lse = lse;
    t.acc_in = acc_in; t.acc_out = acc_out; t.decay = decay;
    t.status = status; t.ws = ws;
    return from_cuda(qmv::launch_attn_tree(cache(c), t, cs(stream)));
}

size_t attn_window_workspace_bytes(const qmv_attn_cache *c, int Hq, int B, int N, int max_new,
                                   int max_pages) {
    if (check_cache(c) || check_batch(c, B, max_pages) || !heads_ok(c, Hq) || N < 0 ||
        !new_ok(c, Hq, max_new))
        return 0;
    return qmv::attn_window_ws_bytes(cache(c), Hq, max_new);
}

int attn_window(const qmv_attn_cache *c, const void *q, int64_t q_stride, int Hq,
                const int32_t *table, int max_pages, const int32_t *ctx, const int32_t *cu, int B,
                int N, int max_new, int window, int sinks, float scale, void *o, int o_dtype,
                float *lse, int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream) {
    int r = check_cache(c);
    if (r) return r;
    if ((r = check_batch(c, B, max_pages))) return r;
    if (N < 0 || !heads_ok(c, Hq) || max_new < 1 || window < 1 || sinks < 0 || !isfinite(scale))
        return QMV_EINVAL;
    if (o_dtype != QMV_F32 && o_dtype != c->dtype) return QMV_EINVAL;
    if (N > 1 << 22 || !new_ok(c, Hq, max_new)) return QMV_ESHAPE;
    if (q_stride < (int64_t)Hq * c->D) return QMV_ESHAPE;
    if (B == 0 || N == 0) return QMV_OK;
    if (!q || !table || !ctx || !cu || !o || !lse) return QMV_EINVAL;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(table, 4) || !aligned(ctx, 4) ||
        !aligned(cu, 4) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < qmv::attn_window_ws_bytes(cache(c), Hq, max_new))
        return QMV_EWORKSPACE;
    qmv::WindowCall t;
    t.s = qmv::AttnSeqs{table, ctx, cu, B, N, max_new, max_pages};
    if (!qmv::attn_window_fits(cache(c), t.s, Hq, window, sinks)) return QMV_ESHAPE;
    t.q = q; t.q_stride = q_stride; t.Hq = Hq;
    t.window = window; t.sinks = sinks; t.scale = scale;
    t.o = o; t.o_f32 = o_dtype == QMV_F32; t.lse = lse;
    t.status = status; t.ws = ws;
    return from_cuda(qmv::launch_attn_window(cache(c), t, cs(stream)));
}

int attn_evict(const qmv_attn_cache *src, const float *acc, const int32_t *table, int max_pages,
               const int32_t *lens, int B, int budget, int sink, int recent,
               const qmv_attn_cache *dst, float *dst_acc, const int32_t *dst_table,
               int dst_max_pages, int32_t *keep, int32_t *new_lens, int32_t *status,
               qmv_stream_t stream) {
    int r = check_cache(src);
    if (r) return r;
    if ((r = check_cache(dst))) return r;
    if ((r = check_batch(src, B, max_pages)) || (r = check_batch(dst, B, dst_max_pages))) return r;
    if (src->Hkv != dst->Hkv || src->D != dst->D || src->dtype != dst->dtype) return QMV_ESHAPE;
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget) return QMV_EINVAL;
    if (budget > 1 << 30) return QMV_ESHAPE;
    if (B == 0) return QMV_OK;
    if (!acc || !table || !lens || !dst_acc || !dst_table || !keep || !new_lens) return QMV_EINVAL;
    if (dst_table == table && dst->k == src->k) return QMV_EINVAL;  // pages onto themselves
    if (!aligned(acc, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(dst_acc, 4) ||
        !aligned(dst_table, 4) || !aligned(keep, 4) || !aligned(new_lens, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    return from_cuda(qmv::launch_attn_evict(cache(src), acc, table, max_pages, lens, B, budget,
                                            sink, recent, cache(dst), dst_acc, dst_table,
                                            dst_max_pages, keep, new_lens, status, cs(stream)));
}

size_t attn_pages_update_workspace_bytes(int pages, int B, int max_pages) {
    return check_pages(pages, 16, B, max_pages) ? 0 : qmv::pages_update_ws_bytes(pages, B, max_pages);
}

int attn_pages_update(int32_t *refs, int pages, int page, int32_t *table, int max_pages,
                      const int32_t *lens, const int32_t *more, int B, int window, int sinks,
                      int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream) {
    const int r = check_pages(pages, page, B, max_pages);
    if (r) return r;
    if (window < 1 || sinks < 0) return QMV_EINVAL;
    if (B == 0) return QMV_OK;
    if (!refs || !table || !lens || !more) return QMV_EINVAL;
    if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(more, 4) ||
        !aligned(status, 4))
        return QMV_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < qmv::pages_update_ws_bytes(pages, B, max_pages))
        return QMV_EWORKSPACE;
    const Ints ta{table, (int64_t)B * max_pages}, le{lens, B}, mo{more, B};
    if (!apart(ta, {le, mo}) || !apart(Ints{refs, pages}, {ta, le, mo})) return QMV_EINVAL;
    return from_cuda(qmv::launch_pages_update(refs, pages, page, table, max_pages, lens, more, B,
                                              window, sinks, status, ws, cs(stream)));
}

size_t attn_pages_fork_workspace_bytes(int pages, int F) {
    return check_pages(pages, 16, F, 1) ? 0 : qmv::pages_fork_ws_bytes(pages, F);
}

int attn_pages_fork(int32_t *refs, int pages, int page, const int32_t *table, int max_pages,
                    const int32_t *lens, int B, const int32_t *parent, int F, int32_t *new_table,
                    int32_t *new_lens, int32_t *moves, int32_t *status, void *ws, size_t ws_bytes,
                    qmv_stream_t stream) {
    int r = check_pages(pages, page, B, max_pages);
    if (r || (r = check_pages(pages, page, F, max_pages))) return r;
    if (F == 0) return QMV_OK;
    if (!refs || !table || !lens || !parent || !new_table || !new_lens || !moves) return QMV_EINVAL;
    if (!aligned(refs, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(parent, 4) ||
        !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(moves, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    if (!ws || !aligned(ws, 256) || ws_bytes < qmv::pages_fork_ws_bytes(pages, F))
        return QMV_EWORKSPACE;
    // (children read their parents' rows while others are written)
    const Ints re{refs, pages}, ta{table, (int64_t)B * max_pages}, le{lens, B}, pa{parent, F};
    const Ints nt{new_table, (int64_t)F * max_pages}, nl{new_lens, F}, mv{moves, (int64_t)F * 3};
    if (!apart(nt, {re, ta, le, pa, nl, mv}) || !apart(nl, {re, ta, le, pa, mv}) || !apart(mv, {re, ta, le, pa}))
        return QMV_EINVAL;
    return from_cuda(qmv::launch_pages_fork(refs, pages, page, table, max_pages, lens, B, parent, F,
                                            new_table, new_lens, moves, status, ws, cs(stream)));
}

int attn_pages_copy(const qmv_attn_cache *src, const qmv_attn_cache *dst, const int32_t *moves, int n,
                    const float *src_acc, float *dst_acc, int32_t *status, qmv_stream_t stream) {
    int r = check_cache(src);
    if (r) return r;
    if ((r = check_cache(dst))) return r;
    if (src->Hkv != dst->Hkv || src->D != dst->D || src->dtype != dst->dtype || src->page != dst->page)
        return QMV_ESHAPE;
    if (n < 0 || (src_acc && !dst_acc)) return QMV_EINVAL;
    if ((int64_t)n * src->Hkv > INT32_MAX) return QMV_ESHAPE;
    if (n == 0) return QMV_OK;
    if (!moves) return QMV_EINVAL;
    if (!aligned(moves, 4) || !aligned(src_acc, 4) || !aligned(dst_acc, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    return from_cuda(qmv::launch_pages_copy(cache(src), cache(dst), moves, n, src_acc, dst_acc, status,
                                            cs(stream)));
}

int attn_compact(const qmv_attn_cache *c, const int32_t *table, int max_pages, const int32_t *ctx,
                 const int32_t *cu, int B, int N, const int32_t *keep, const int32_t *kept, float *acc,
                 int32_t *new_ctx, int32_t *status, qmv_stream_t stream) {
    int r = check_cache(c);
    if (r) return r;
    if ((r = check_batch(c, B, max_pages))) return r;
    if (N < 0) return QMV_EINVAL;
    if (B == 0) return QMV_OK;
    if (!table || !ctx || !cu || (!keep && N) || !kept || !new_ctx) return QMV_EINVAL;
    if (!aligned(table, 4) || !aligned(ctx, 4) || !aligned(cu, 4) || !aligned(keep, 4) ||
        !aligned(kept, 4) || !aligned(acc, 4) || !aligned(new_ctx, 4) || !aligned(status, 4))
        return QMV_EALIGN;
    // (other blocks still read them)
    if (!apart(Ints{new_ctx, B}, {Ints{table, (int64_t)B * max_pages}, Ints{ctx, B}, Ints{cu, B + 1},
                                  Ints{keep, N}, Ints{kept, B}}))
        return QMV_EINVAL;
    return from_cuda(qmv::launch_attn_compact(cache(c), qmv::AttnSeqs{table, ctx, cu, B, N, 0, max_pages},
                                              keep, kept, acc, new_ctx, status, cs(stream)));
}

}  // extern "C"
