// qmv_attn.h - launchers of the attention operators (host side, no validation
// here: the ABI layer checks every argument before calling these).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qmv {

struct AttnCache {
    void *k, *v;  // [pages][Hkv][page][D]
    int pages, Hkv, page, D;
    bool bf16;  // else fp16
};

struct AttnSeqs {
    const int32_t *table, *ctx, *cu;
    int B, N, max_draft, max_pages;
};

struct RopeIn {
    const void *p;
    long long stride;  // elements between tokens
};

// Norms of query and key heads before the turn.
struct RopeNorm {
    const void *qw, *kw;  // [D], or null: ones
    int w_f32;            // else of the cache's type
    float eps;
};

// in_type: 0 fp32, else the cache's type. acc (optional): cleared for the new tokens.
// norm (optional): query and key heads are normed first.
cudaError_t launch_rope_append(const AttnCache &c, const AttnSeqs &s, const RopeIn &q,
                               const RopeIn &k, const RopeIn &v, int in_f32, int Hq,
                               const int32_t *pos, const double *inv_freq, int rot,
                               bool interleaved, float mscale, void *q_out, float *acc,
                               int32_t *status, cudaStream_t st, const RopeNorm *norm = nullptr);

struct TreeCall {
    AttnSeqs s;
    const void *q;
    long long q_stride;
    int Hq;
    const uint32_t *mask;  // [N][words], or null: draft j sees drafts 0..j
    int words;
    float scale;
    void *o;
    int o_f32;
    float *lse;
    const float *acc_in;
    float *acc_out;  // null: no weights
    float decay;
    int32_t *status;
    void *ws;
};
size_t attn_tree_ws_bytes(const AttnCache &c, int Hq, int B, int N, int max_draft, int max_pages,
                          bool acc);
cudaError_t launch_attn_tree(const AttnCache &c, const TreeCall &t, cudaStream_t st);

struct WindowCall {
    AttnSeqs s;  // max_draft: the new tokens of a sequence, at most
    const void *q;
    long long q_stride;
    int Hq, window, sinks;
    float scale;
    void *o;
    int o_f32;
    float *lse;
    int32_t *status;
    void *ws;
};
size_t attn_window_ws_bytes(const AttnCache &c, int Hq, int max_new);
// Whether a block's share of the call's units can be counted in 31 bits.
bool attn_window_fits(const AttnCache &c, const AttnSeqs &s, int Hq, int window, int sinks);
cudaError_t launch_attn_window(const AttnCache &c, const WindowCall &t, cudaStream_t st);

cudaError_t launch_attn_evict(const AttnCache &src, const float *acc, const int32_t *table,
                              int max_pages, const int32_t *lens, int B, int budget, int sink,
                              int recent, const AttnCache &dst, float *dst_acc,
                              const int32_t *dst_table, int dst_max_pages, int32_t *keep,
                              int32_t *new_lens, int32_t *status, cudaStream_t st);

// Pages: page = tokens a page. (qmv_pages.cu)
size_t pages_update_ws_bytes(int pages, int B, int max_pages);
cudaError_t launch_pages_update(int32_t *refs, int pages, int page, int32_t *table, int max_pages,
                                const int32_t *lens, const int32_t *more, int B, int window, int sinks,
                                int32_t *status, void *ws, cudaStream_t st);
size_t pages_fork_ws_bytes(int pages, int F);
cudaError_t launch_pages_fork(int32_t *refs, int pages, int page, const int32_t *table, int max_pages,
                              const int32_t *lens, int B, const int32_t *parent, int F,
                              int32_t *new_table, int32_t *new_lens, int32_t *moves, int32_t *status,
                              void *ws, cudaStream_t st);
cudaError_t launch_pages_copy(const AttnCache &src, const AttnCache &dst, const int32_t *moves, int n,
                              const float *src_acc, float *dst_acc, int32_t *status, cudaStream_t st);
cudaError_t launch_attn_compact(const AttnCache &c, const AttnSeqs &s, const int32_t *keep,
                                const int32_t *kept, float *acc, int32_t *new_ctx, int32_t *status,
                                cudaStream_t st);

}  // namespace qmv
