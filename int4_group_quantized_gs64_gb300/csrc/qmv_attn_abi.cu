// qmv_attn_abi.cu - the extern "C" entry points of the attention operators
// (include/qmv.h): host-side checks, then the launchers of qmv_attn.h. As in
// qmv_abi.cu, a negative status means that nothing was enqueued.
#include <math.h>
#include <stdint.h>

#include "../../include/qmv.h"
#include "qmv_attn.h"

namespace {

constexpr int kMaxDraft = 256;
constexpr int kMaxHeads = 1024;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t cs(qmv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? QMV_OK : QMV_ECUDA; }

int check_cache(const qmv_attn_cache *c) {
    if (!c || !c->k || !c->v || c->pages < 1 || c->Hkv < 1 || c->Hkv > kMaxHeads) return QMV_EINVAL;
    if (c->dtype != QMV_BF16 && c->dtype != QMV_F16) return QMV_EINVAL;
    if (c->D != 64 && c->D != 128) return QMV_ESHAPE;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return QMV_ESHAPE;
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

}  // namespace

extern "C" {

int attn_rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                     int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                     const int32_t *pos, const double *inv_freq, int rot, int interleaved,
                     float mscale, const int32_t *table, int max_pages, const int32_t *ctx,
                     const int32_t *cu, int B, int N, void *q_out, float *acc, int32_t *status,
                     qmv_stream_t stream) {
    int r = check_cache(c);
    if (r) return r;
    if ((r = check_batch(c, B, max_pages))) return r;
    if (N < 0 || !heads_ok(c, Hq) || rot < 2 || rot > c->D || rot % 2 || !isfinite(mscale))
        return QMV_EINVAL;
    if (in_dtype != QMV_F32 && in_dtype != c->dtype) return QMV_EINVAL;
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
    return from_cuda(qmv::launch_rope_append(
        cache(c), qmv::AttnSeqs{table, ctx, cu, B, N, 0, max_pages}, qmv::RopeIn{q, q_stride},
        qmv::RopeIn{k, k_stride}, qmv::RopeIn{v, v_stride}, in_dtype == QMV_F32, Hq, pos, inv_freq,
        rot, interleaved != 0, mscale, q_out, acc, status, cs(stream)));
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

}  // extern "C"
