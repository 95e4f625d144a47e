/*
 * qmv.h - C ABI of the GB300 (sm_103a) quantized matrix-vector library.
 *
 * Quantized formats (colibri PR #418 "Vulkan backend: expert tier + dense +
 * MLA attention on any Vulkan 1.2 GPU"):
 *   int4-gs64  two offset-binary nibbles per byte, value = nibble - 8
 *              (commit "opt-in Vulkan int4/int8 quantized GEMV"), element 2j
 *              in the LOW nibble of byte j and 2j+1 in the high nibble (the
 *              pages do not state the order; this is the library's reading),
 *              bytes in K order; one fp32 scale per 64 consecutive K values
 *              applied to that group's partial dot product (commit "grouped
 *              scales in the Vulkan kernels", fmt 4, group size 64).
 *              Weights [rows][K/2] uint8, scales [rows][K/64] fp32, row-major.
 *   int8-row   int8 weights [rows][K] with one fp32 scale per row (same
 *              GEMV commit, fmt 1).
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers (memory the caller allocated on
 *     the current CUDA device). The caller owns every buffer; the library
 *     never allocates, frees or synchronises.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and is complete when the stream is. Calls can be
 *     captured into CUDA graphs.
 *   - Arguments are validated on the host before anything is enqueued. On a
 *     nonzero return nothing was enqueued and no output was touched.
 *   - Shapes are row-major and contiguous. K, H and I must be multiples of 64.
 *   - Activations may have any finite fp32 value; each kernel rescales them
 *     by a power of two internally, which changes no result bit pattern beyond
 *     the stated tolerance.
 *   - Accuracy: the fp32 paths return y with
 *         |y - y_exact| <= 2e-5 * sum_k |w_k * x_k|
 *     per output (w the dequantized weight), the bf16 prefill path with 1e-2.
 */
#ifndef QMV_H
#define QMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, so CUDA callers pass their streams unchanged. */
typedef struct CUstream_st *qmv_stream_t;

typedef enum {
    QMV_OK = 0,
    QMV_EINVAL = -1,     /* null pointer, bad count, unsupported group size   */
    QMV_ESHAPE = -2,     /* a dimension is not a multiple of 64 or too large   */
    QMV_EWORKSPACE = -3, /* workspace pointer null, misaligned or too small    */
    QMV_ECUDA = -4,      /* a CUDA launch failed (see cudaGetLastError)        */
    QMV_ETIMEOUT = -5,   /* a bounded device-side wait gave up                 */
    QMV_EALIGN = -6      /* a pointer is not aligned as documented             */
} qmv_status;

/* Library version as 10000*major + 100*minor + patch. */
int qmv_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char *qmv_status_str(int status);

/* Test hook, not part of the method: from the next launch on, the compute
 * warps of every odd CTA of the tensor-map MoE and dense kernels start `ns`
 * nanoseconds late (0 turns it off; negative values are taken as 0). Items
 * whose stages two CTAs share then meet every order of arrival, so tests can
 * check that the output does not depend on it. Process-wide, host only,
 * enqueues nothing; not thread-safe against concurrent launches. Returns the
 * previous value. */
int qmv_test_split_skew(int ns);

/* ---------------------------------------------------------------- GEMV */

/* Scratch needed by qmv_int4_gs / qmv_int8_row for S tokens of length K, in
 * bytes (a multiple of 256; 0 for unsupported sizes). It holds a status word
 * (the first int32, cleared by every call: bit 1 = a bounded device wait ran
 * out and y is not valid), counters and partial sums for row tiles shared
 * between thread blocks (about 4 MB, independent of K and S), and the
 * activations, converted into fp16 hi/lo fragments with one power-of-two
 * factor per 64-wide group before the weights are streamed. */
size_t qmv_gemv_workspace_bytes(int K, int S);

/* Dense int4 grouped-scale GEMV (colibri PR #418, commits "opt-in Vulkan
 * int4/int8 quantized GEMV" and "grouped scales in the Vulkan kernels"):
 *     y[s][i] = sum_g scales[i][g] * sum_{k in group g} (nibble(i,k) - 8) * x[s][k]
 *   wq      [N][K/2] uint8, 16-byte aligned
 *   scales  [N][K/gs] fp32, 4-byte aligned
 *   x       [S][K] fp32, 4-byte aligned
 *   y       [S][N] fp32 (written, fp32-accumulated)
 *   ws      device scratch of at least qmv_gemv_workspace_bytes(K, S) bytes,
 *           256-byte aligned, not shared with a concurrent call
 *   gs must be 64; K a multiple of 64; 1 <= N, 1 <= S, K <= 65536.
 * Up to 4 tokens whose activations fit 64 KB of fragments (S * K <= 16384)
 * run as one launch: every thread block converts x itself and streams its
 * 16-row tiles through per-warp cp.async rings, K split over the warps.
 * Otherwise, when N is a multiple of 16, K/64 a multiple of 4 and wq and
 * scales are 16-byte aligned, the weights stream through tensor-map (TMA)
 * copies with the row tiles' work shared evenly over all SMs; other shapes
 * use per-warp cp.async rings. All give the same results up to fp32
 * summation order.
 * Errors: QMV_EINVAL (null pointer, gs != 64, N or S < 1), QMV_ESHAPE (K),
 *         QMV_EALIGN, QMV_EWORKSPACE, QMV_ECUDA. */
int qmv_int4_gs(const uint8_t *wq, const float *scales, int N, int K, int gs, const float *x,
                float *y, int S, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* qmv_int4_gs with a bf16 output (colibri PR #418: the commit "vk_matmul_qt
 * routes a resident int4/int8 matmul_qt through coli_vk_matmul", whose dense
 * projections feed the next layer, and the rmsnorm / coli_vk_attn_qprep
 * chain that consumes them on the device; bf16 is the reading of the
 * activation type that chain passes on). The sum is formed exactly as in
 * qmv_int4_gs, in fp32, and each output is then rounded to the nearest bf16
 * value, ties to even:
 *   y_bf16  [S][N] bf16 bit patterns (uint16_t, 2-byte aligned; written)
 *   every other argument, the workspace and the errors as qmv_int4_gs.
 * For the same inputs and workspace size the result is the fp32 output of
 * qmv_int4_gs rounded to bf16, bit for bit. */
int qmv_int4_gs_bf16(const uint8_t *wq, const float *scales, int N, int K, int gs, const float *x,
                     uint16_t *y_bf16, int S, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* Two int4-gs64 GEMVs against the same activations (colibri PR #418, commit
 * "qmatmul staged-x length fix": matmul_pair stages x once for the q_a and
 * kv_a projections, 6144 -> (2048, 576), and records both in one submit):
 *     y0 = W0 x and y1 = W1 x, each exactly as qmv_int4_gs computes it
 *   wq0 [N0][K/2] and wq1 [N1][K/2] uint8, 16-byte aligned
 *   s0 [N0][K/gs], s1 [N1][K/gs] fp32; x [S][K]; y0 [S][N0]; y1 [S][N1] fp32
 *   ws      device scratch of at least qmv_gemv_workspace_bytes(K, S) bytes
 *           (the same as one GEMV), 256-byte aligned
 * x is converted into fp16 hi/lo fragments once. For up to 4 tokens with
 * S * K <= 16384 (see qmv_int4_gs) the row tiles of both matrices are one
 * work sequence of the single-launch kernel; otherwise, when both matrices
 * qualify for the tensor-map path, of one tensor-map launch; otherwise the
 * two GEMVs run one after the other (the status word then reports the second).
 * Errors: as qmv_int4_gs. */
int qmv_int4_gs_pair(const uint8_t *wq0, const float *s0, int N0, const uint8_t *wq1,
                     const float *s1, int N1, int K, int gs, const float *x, float *y0, float *y1,
                     int S, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* Dense int3-g64 GEMV over two-plane rows (colibri PR #418, the fmt-5
 * commit: 24 bytes per 64-group, lanes striding the 16-value low-plane words,
 * the high-plane word pre-shifted to bit 0, group scales applied to the word
 * partials). The pages name the planes but print no byte; the layout read
 * here: in each 24-byte group, bytes 0..15 hold 2 low bits per element
 * (element e at bits 2(e%4) of byte e/4) and bytes 16..23 one high bit per
 * element (bit e%8 of byte 16 + e/8); code = low | high << 2, value = code - 4.
 *     y[s][i] = sum_g scales[i][g] * sum_{k in group g} (code(i,k) - 4) * x[s][k]
 *   wq3     [N][K/64 * 24] uint8, 4-byte aligned
 *   scales  [N][K/gs] fp32, 4-byte aligned
 *   x       [S][K] fp32, 16-byte aligned
 *   y       [S][N] fp32 (written, fp32-accumulated)
 *   gs must be 64; K a multiple of 64; 1 <= N, 1 <= S, K <= 65536. No
 *   workspace: on the CUDA cores, each warp walks its rows and decodes each
 *   32-bit low-plane word once for up to 4 tokens; x is staged per CTA in up
 *   to 96 KB of shared memory (read from global memory when K > 24576).
 * Errors: QMV_EINVAL, QMV_ESHAPE (K), QMV_EALIGN, QMV_ECUDA. */
int qmv_int3_gs(const uint8_t *wq3, const float *scales, int N, int K, int gs, const float *x,
                float *y, int S, qmv_stream_t stream);

/* Dense int8 per-row-scale GEMV (same commit, fmt 1):
 *     y[s][i] = row_scale[i] * sum_k w[i][k] * x[s][k]
 *   w [N][K] int8 (16-byte aligned), row_scale [N] fp32, x [S][K] fp32, y [S][N] fp32,
 *   ws as for qmv_int4_gs. K a multiple of 64, K <= 65536; N, S >= 1.
 *   Errors as qmv_int4_gs. */
int qmv_int8_row(const int8_t *w, const float *row_scale, int N, int K, const float *x,
                 float *y, int S, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* qmv_int8_row with a bf16 output (as qmv_int4_gs_bf16): the fp32 result of
 * qmv_int8_row rounded to the nearest bf16, ties to even, into
 *   y_bf16  [S][N] bf16 bit patterns (uint16_t, 2-byte aligned; written);
 *   every other argument, the workspace and the errors as qmv_int8_row. */
int qmv_int8_row_bf16(const int8_t *w, const float *row_scale, int N, int K, const float *x,
                      uint16_t *y_bf16, int S, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* The dense int4-gs64 GEMV of qmv_int4_gs for callers that cannot allocate
 * device memory: code that must never make the device synchronise (cudaMalloc
 * and cudaFree can), hosts that forbid device allocation after start-up, and
 * C callers with nowhere to keep a workspace between calls. Same arguments as
 * qmv_int4_gs, minus the workspace, and the same results up to the order of
 * the fp32 additions: it always runs the per-warp cp.async kernel, never the
 * tensor-map kernel that qmv_int4_gs takes when N % 16 == 0, so results are
 * not bit-identical to qmv_int4_gs and its speed differs on such shapes. The
 * pages have no counterpart of this entry point.
 *   Scratch: one file-scope device array inside the library (266,240 bytes,
 *   held by every GPU that loads the library until the process exits), so
 *   S * K must be at most 65536; larger calls return QMV_EWORKSPACE and
 *   enqueue nothing.
 *   Every call looks up the array's device address in the current context (a
 *   host call, cudaGetSymbolAddress), so a device reset does not leave a stale
 *   address behind. The first call on a device may load the library's module
 *   there, which allocates the array and can synchronise: make one call per
 *   device at start-up, before any stream capture and before any code that
 *   must not synchronise.
 *   Every call uses the same array and overwrites all of it that it reads, so
 *   nothing carries over between calls, but calls whose work overlaps on the
 *   GPU (different streams, or different host threads on one device) race on
 *   it: order them on one stream.
 *   Allocates nothing itself: no cudaMalloc, cudaFree or allocating library
 *   call. */
int qmv_int4_gs_noalloc(const uint8_t *wq, const float *scales, int N, int K, int gs,
                        const float *x, float *y, int S, qmv_stream_t stream);

/* ---------------------------------------------------------------- MoE */

/* Device-resident int4-gs64 expert weights (the analogue of the pages'
 * uploaded-once weight handle). All experts live in one pool each:
 *   gu_q [E][2I][H/2] uint8: gate rows 0..I-1, then up rows I..2I-1 (reading:
 *        the pages fuse gate and up but do not state the stacking order)
 *   gu_s [E][2I][H/64] fp32
 *   dn_q [E][H][I/2] uint8, dn_s [E][H][I/64] fp32
 * The descriptor itself is a HOST struct; it is read during the call only. */
typedef struct {
    const uint8_t *gu_q;
    const float *gu_s;
    const uint8_t *dn_q;
    const float *dn_s;
    int32_t E, H, I, gs;
} qmv_moe_int4;

/* Top-k routing: for each token, the k experts with the largest logits
 * (fp32 comparison; equal logits keep the lower expert index first), in
 * descending logit order, with weights = softmax over all experts restricted
 * to the chosen k and renormalised to sum to one (equivalently
 * exp(l_e - l_max) / sum over the chosen). NaN logits are never chosen
 * ahead of finite ones.
 *   logits [T][E] fp32; ids [T][k] int32 (written); w [T][k] fp32 (written).
 *   1 <= k <= min(E, 32), E <= 1024, T >= 0 (T == 0 enqueues nothing). */
int moe_route_topk(const float *logits, int T, int E, int k, int32_t *ids, float *w,
                   qmv_stream_t stream);

/* Token -> expert grouping (so each expert's weights are read once per batch,
 * colibri PR #418 "coli_vk_expert_group"). Pair p = t*k + j.
 *   offsets [E+1] int32: exclusive prefix sum of the per-expert pair counts
 *   list    [T*k] int32: pair ids grouped by expert, ascending inside a group
 *   uexp    [E]   int32: the experts with at least one pair, ascending
 *   n_used  [1]   int32: how many entries of uexp are valid
 *   status  [1]   int32: OR-ed with 1 when an id is outside [0, E); such a
 *                 pair is left out of every list. Not cleared by this call.
 *   T*k <= 1 << 20, E <= 1024. */
int moe_group(const int32_t *ids, int T, int k, int E, int32_t *offsets, int32_t *list,
              int32_t *uexp, int32_t *n_used, int32_t *status, qmv_stream_t stream);

/* Fused gate+up with SiLU*mul for every grouped pair (colibri PR #418,
 * commit "qmatmul_gate_up.comp + coli_vk_gate_up"): for each expert e in
 * uexp and each pair p = t*k + j routed to e,
 *     h[p][c] = SiLU(gate_e[c] . x[t]) * (up_e[c] . x[t]),   SiLU(g) = g / (1 + e^-g)
 *   x [T][H] fp32; h [T*k][I] fp32 (rows of pairs that no expert serves are
 *   left untouched). offsets/list/uexp/n_used as written by moe_group.
 *   ws: device scratch of at least moe_workspace_bytes(m, T, k) bytes,
 *   256-byte aligned (the activations are converted into it first). */
int moe_gate_up_silu(const qmv_moe_int4 *m, const float *x, int T, int k,
                     const int32_t *offsets, const int32_t *list, const int32_t *uexp,
                     const int32_t *n_used, float *h, void *ws, size_t ws_bytes,
                     qmv_stream_t stream);

/* Down projection of every grouped pair (colibri PR #418, "coli_vk_expert_group"):
 *     y[p][i] = down_e[i] . h[p]          y [T*k][H] fp32 (pairs not served: untouched)
 * and the weighted combine (PR #1338, weighted accumulation of expert outputs):
 *     out[t][i] = sum_{j < k, ids[t][j] valid} w[t][j] * y[t*k + j][i]
 *   summed in slot order, so results are deterministic. out [T][H] fp32.
 *   moe_down takes the same workspace as moe_gate_up_silu. moe_combine reads
 *   ids to skip pairs whose id is outside [0, E). */
int moe_down(const qmv_moe_int4 *m, const float *h, int T, int k, const int32_t *offsets,
             const int32_t *list, const int32_t *uexp, const int32_t *n_used, float *y,
             void *ws, size_t ws_bytes, qmv_stream_t stream);
int moe_combine(const float *y, const int32_t *ids, const float *w, int T, int k, int E, int H,
                float *out, qmv_stream_t stream);

/* Workspace of the MoE entry points that take one, in bytes (256-byte aligned segments). */
size_t moe_workspace_bytes(const qmv_moe_int4 *m, int T, int k);

/* Whole MoE expert FFN for a decode micro-batch (colibri PR #418,
 * "coli_vk_expert_group": fused gate+up+SiLU, then down, hidden kept on the
 * device; PR #1338: weighted accumulation). Equivalent to moe_group,
 * moe_gate_up_silu, moe_down and moe_combine in sequence:
 *     out[t] = sum_j w[t][j] * down_e(SiLU(gate_e x[t]) * up_e x[t]),  e = ids[t][j]
 *   x [T][H] fp32, ids [T][k] int32, w [T][k] fp32, out [T][H] fp32.
 *   ws: device workspace of at least moe_workspace_bytes(m, T, k) bytes,
 *   256-byte aligned, owned by the caller, not shared between concurrent calls.
 *   The first int32 of ws is a device status word, cleared at the start of
 *   the call: bit 0 = an id outside [0, E) (that pair skipped, as moe_group),
 *   bit 1 = a bounded wait on the weight stream ran out (out not valid).
 *   One token (T == 1) with moe_one_token_path(m, k) == 1 runs as a single
 *   cooperative kernel (all CTAs resident, one grid-wide barrier between
 *   gate+up and down); the result is the same. */
int moe_expert_ffn_int4(const qmv_moe_int4 *m, const float *x, int T, const int32_t *ids,
                        const float *w, int k, float *out, void *ws, size_t ws_bytes,
                        qmv_stream_t stream);

/* Routing and expert FFN of a decode micro-batch in one call: moe_route_topk
 * on logits [T][E] (ids [T][k] and w [T][k] are written, as that call writes
 * them), then moe_expert_ffn_int4 with those ids and weights; same
 * workspace, limits and status word (1 <= k <= min(E, 32)). With one token
 * and moe_one_token_path(m, k) == 1 the routing runs inside the
 * single-launch FFN kernel (every thread block routes the token itself; the
 * first writes ids and w), so the call is one kernel after the status clear.
 * With 2..32 tokens on the tensor-map path the grouping kernel routes the
 * tokens itself the same way, which saves the routing launch.
 * Errors: those of moe_route_topk and moe_expert_ffn_int4. */
int moe_route_expert_ffn_int4(const qmv_moe_int4 *m, const float *logits, const float *x, int T,
                              int k, int32_t *ids, float *w, float *out, void *ws, size_t ws_bytes,
                              qmv_stream_t stream);

/* moe_expert_ffn_int4 over the resident experts only (colibri PR #418,
 * "Vulkan expert tier ... overlapped with CPU rows": the GPU computes the
 * experts of its registry while the CPU computes the rest; PR #1338,
 * "Validation": a miss returns no mask bit):
 *     out[t] = sum over served slots j of w[t][j] * down_e(SiLU(gate_e x[t]) * up_e x[t])
 *     served[t][j] = 1 if e = ids[t][j] is in [0, E) and bit e % 32 of
 *                    resident[e / 32] is set, else 0
 *   resident  device bitmap [ceil(E / 32)] uint32, 4-byte aligned
 *   served    device [T][k] uint8, written
 *   others and the workspace as moe_expert_ffn_int4. A token with no served
 *   slot gets out[t] = 0. The caller adds the unserved slots' terms itself.
 *   A non-resident id is not an error; status bit 0 still flags ids outside
 *   [0, E). Errors: those of moe_expert_ffn_int4, plus QMV_EINVAL for a null
 *   resident or served and QMV_EALIGN for a misaligned resident. */
int moe_expert_ffn_int4_resident(const qmv_moe_int4 *m, const uint32_t *resident, const float *x,
                                 int T, const int32_t *ids, const float *w, int k, float *out,
                                 uint8_t *served, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* The four phases of moe_expert_ffn_int4, for callers that interleave other
 * work or time the phases (the pages split their expert group the same way
 * into issue and take). All four take the same workspace; each phase reads
 * what the previous one left there, so they must run in this order on one
 * stream, with T and k unchanged:
 *   moe_ffn_prepare  clears the status word, groups the pairs (moe_group) and
 *                    converts x into fp16 hi/lo cells with per-group factors;
 *   moe_ffn_gate_up  h = SiLU(gate x) * up x for every served pair, kept in the
 *                    workspace both as fp32 and as cells for the down pass;
 *   moe_ffn_down     y = down h per pair, in the workspace;
 *   moe_ffn_combine  out[t] = sum_j w[t][j] * y[t*k + j], slot order. */
int moe_ffn_prepare(const qmv_moe_int4 *m, const float *x, int T, const int32_t *ids, int k,
                    void *ws, size_t ws_bytes, qmv_stream_t stream);
int moe_ffn_gate_up(const qmv_moe_int4 *m, int T, int k, void *ws, size_t ws_bytes,
                    qmv_stream_t stream);
int moe_ffn_down(const qmv_moe_int4 *m, int T, int k, void *ws, size_t ws_bytes,
                 qmv_stream_t stream);
int moe_ffn_combine(const qmv_moe_int4 *m, const int32_t *ids, const float *w, int T, int k,
                    float *out, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* Which weight stream the decode gate+up and down kernels of this descriptor
 * use (no counterpart on the pages; it names the kernel a profile shows):
 *   1  tensor-map bulk copies (TMA) into an mbarrier-guarded ring, taken when
 *      H/64 and I/64 are multiples of 4 and the four pools are 16-byte aligned;
 *   0  per-warp cp.async rings otherwise.
 * Both compute the same result. Host only, enqueues nothing.
 * Errors: those of the descriptor check shared by every MoE call (QMV_EINVAL,
 * QMV_ESHAPE, QMV_EALIGN). */
int moe_weight_path(const qmv_moe_int4 *m);

/* Whether moe_expert_ffn_int4 with T == 1 and this k runs the single-launch
 * kernel (1) or the grouped phases (0). The single launch is taken when the
 * weight pools suit the tensor-map path (moe_weight_path == 1), H and I are
 * multiples of 256, 1 <= k <= 32, and one CTA's share of the layer's weights
 * fits in its shared memory. No counterpart on the pages; it names the kernel
 * a profile shows. Host only, enqueues nothing.
 * Errors: those of the descriptor check shared by every MoE call. */
int moe_one_token_path(const qmv_moe_int4 *m, int k);

/* Workspace of moe_expert_ffn_int4_prefill, in bytes (0 for unsupported sizes). */
size_t moe_prefill_workspace_bytes(const qmv_moe_int4 *m, int T, int k);

/* Batched MoE prefill on the tcgen05 tensor cores (colibri PR #418 PR summary
 * names cooperative-matrix prefill kernels as the next step for batched
 * prompts; the math is that of moe_expert_ffn_int4):
 *     out[t] = sum_j w[t][j] * down_e(SiLU(gate_e x[t]) * up_e x[t]),  e = ids[t][j]
 * with bf16 operands and fp32 accumulation: the weights are dequantized to
 * bf16 with their group scale folded in, h is rounded to bf16 between the two
 * projections; expected accuracy |out - exact| <= 1e-2 * sum |w * down * h|.
 *   x_bf16 [T][H] bfloat16 bit patterns, 16-byte aligned; ids [T][k] int32;
 *   w [T][k] fp32; out [T][H] fp32.
 *   Each expert's tokens are processed in passes of up to 64, each pass
 *   reading the expert's weights once. I must be a multiple of 128.
 *   ws: at least moe_prefill_workspace_bytes(m, T, k) bytes, 256-byte aligned;
 *   its first int32 is a status word: bit 0 = an id outside [0, E) (pair
 *   skipped), bit 1 = a tensor-core wait timed out (output not valid). */
int moe_expert_ffn_int4_prefill(const qmv_moe_int4 *m, const uint16_t *x_bf16, int T,
                                const int32_t *ids, const float *w, int k, float *out, void *ws,
                                size_t ws_bytes, qmv_stream_t stream);

/* ---------------------------------------------------------------- attention
 *
 * The attention half of a decode or speculative-decoding step next to the
 * expert half above: rotary positions and the append to a paged key/value
 * cache, attention of a tree of drafted tokens (or one token) over it, and
 * eviction from it by accumulated attention weight. */

typedef enum { QMV_F32 = 0, QMV_BF16 = 1, QMV_F16 = 2 } qmv_dtype;

/* A paged cache of one layer. Token `slot` of sequence b is row slot % page of
 * page table[b][slot / page]; a page holds, per head, `page` rows of D values
 * in a row. dtype is QMV_BF16 or QMV_F16; D is 64 or 128; page is 16, 32, 64,
 * 128 or 256; pages * Hkv * page < 2^31. k and v are 16-byte aligned. The
 * running attention weights, where they are kept, are a float array
 * [pages][Hkv][page] of the caller. The descriptor is a HOST struct. */
typedef struct {
    void *k; /* [pages][Hkv][page][D] */
    void *v; /* [pages][Hkv][page][D] */
    int32_t pages, Hkv, page, D, dtype;
} qmv_attn_cache;

/* Shared by the calls below:
 *   table   [B][max_pages] int32 page ids; max_pages * page <= 2^30;
 *           B * Hkv <= 65535.
 *   ctx     [B] int32: the tokens of each sequence already in the cache.
 *   cu      [B + 1] int32: the first new token of each sequence, cu[B] = N;
 *           sequence b's new tokens cu[b] .. cu[b + 1] - 1 have slots
 *           ctx[b], ctx[b] + 1, ... (A descending cu gives a sequence of
 *           negative length, which is left out, and tokens of several: such a
 *           token's keys and values go to the last of these.)
 *   status  [1] int32 or NULL, OR-ed (not cleared) with
 *             1  a page id outside [0, pages): its tokens are left out;
 *             2  a sequence whose lengths are negative, do not fit its row of
 *                the table, or exceed N or max_draft: it is left out (its
 *                output rows are not written);
 *             4  a bounded wait on a copy ran out: outputs are not valid.
 *   B == 0 or N == 0 enqueues nothing. Errors: QMV_EINVAL (null pointer, bad
 *   count or dtype), QMV_ESHAPE (D, page, or a size past its limit),
 *   QMV_EALIGN, QMV_EWORKSPACE, QMV_ECUDA. */

/* Rotary positions of N new tokens and their append to the cache. Token n's
 * query and key heads are turned by the angles pos[n] * inv_freq[i], i < rot/2:
 *     (a, b) -> mscale * (a cos - b sin, b cos + a sin)
 * on elements (i, i + rot/2) of a head, or (2i, 2i + 1) when interleaved != 0;
 * elements rot .. D - 1 pass unchanged. Queries go to q_out, keys and values
 * to the tokens' slots. Angles are formed in 64 bits and
 * the fraction of a turn is rounded to fp32 (off by 3 * 2^-53 of the angle, 7e-7
 * at position 2^31, and 2 pi 2^-25), the rest is fp32, rounded once to the
 * cache's type. Scaled
 * positions for long contexts are a matter of inv_freq and mscale.
 *   q [N] rows of Hq * D, k and v [N] rows of Hkv * D, q_stride, k_stride and
 *     v_stride elements apart (so they may be parts of one projection's rows);
 *     in_dtype QMV_F32 or the cache's. Rows on 16-byte boundaries and rot a
 *     multiple of 16 take the vector path; any other alignment is correct.
 *   pos [N] int32; inv_freq [rot/2] double, 8-byte aligned; 2 <= rot <= D, even
 *   q_out [N][Hq][D] in the cache's type, 16-byte aligned (written)
 *   acc   running attention weights, or NULL: set to 0 for the new tokens
 *   Hq a multiple of Hkv, at most 1024; N <= 2^22. */
int attn_rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                     int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                     const int32_t *pos, const double *inv_freq, int rot, int interleaved,
                     float mscale, const int32_t *table, int max_pages, const int32_t *ctx,
                     const int32_t *cu, int B, int N, void *q_out, float *acc, int32_t *status,
                     qmv_stream_t stream);

/* attn_rope_append with norms: every query and key head x first becomes
 *     x_i * w_i / sqrt(mean(x^2) + eps)
 * (the mean over its D elements, all of them, also where rot < D), then is turned
 * and goes to q_out or the cache as above; values pass unchanged. In fp32 from the
 * inputs to the one rounding at the end, heads of any finite magnitude (where their
 * squares leave fp32's range they are scaled by a power of two first). A head of
 * zeros stays zeros, also with eps = 0.
 *   q_weight, k_weight [D] in w_dtype (QMV_F32 or the cache's), aligned to it, or
 *     NULL: ones; 16-byte aligned ones keep the vector path
 *   eps finite, >= 0; everything else as attn_rope_append. */
int attn_norm_rope_append(const qmv_attn_cache *c, const void *q, int64_t q_stride, const void *k,
                          int64_t k_stride, const void *v, int64_t v_stride, int in_dtype, int Hq,
                          const void *q_weight, const void *k_weight, int w_dtype, float eps,
                          const int32_t *pos, const double *inv_freq, int rot, int interleaved,
                          float mscale, const int32_t *table, int max_pages, const int32_t *ctx,
                          const int32_t *cu, int B, int N, void *q_out, float *acc,
                          int32_t *status, qmv_stream_t stream);

/* Workspace of attn_tree, in bytes (0 for unsupported sizes). weights != 0:
 * with acc_out, which with up to 16 rows a key/value head keeps a score for each
 * of them and every slot of the table, up to 1 GiB. */
size_t attn_tree_workspace_bytes(const qmv_attn_cache *c, int Hq, int B, int N, int max_draft,
                                 int max_pages, int weights);

/* Attention of each sequence's drafted tokens over its cache, drafts included
 * (their keys and values are in their slots: attn_rope_append). Head hq reads
 * key/value head hq / (Hq / Hkv). Token n = cu[b] + t sees every slot below
 * ctx[b], and draft d of its own sequence when bit d % 32 of
 * mask[n][d / 32] is set (mask NULL: when d <= t, a chain; a single token is a
 * tree of one node):
 *     x_j = scale * q[n][hq] . k_j      over the slots j that it sees
 *     lse[n][hq] = log sum_j exp(x_j),  o[n][hq] = sum_j exp(x_j - lse) v_j
 *     acc_out[slot j] = decay * acc_in[slot j] + sum over the tokens of the
 *                       sequence and the query heads of the key/value head of
 *                       exp(x_j - lse)                     (where asked for)
 * A row that sees no key, or only keys of score -inf, gets o = 0 and
 * lse = -inf and adds no weight. What it does not see never reaches a row:
 * not stale slots after the end, nor infinities or NaNs in masked drafts.
 * (Infinities and NaNs among the values of a key that it does see leave these
 * elements of its output infinite or NaN.)
 * Sequences may share pages (a common prefix) as long as acc_out is NULL: with
 * running weights a page belongs to one sequence of the call, since a sum has
 * one decay and one set of rows; the sums of a shared page are not defined.
 * Otherwise results do not depend on the order in which thread blocks finish.
 *   q [N] rows of Hq * D in the cache's type, 16-byte aligned, q_stride
 *     elements apart (a multiple of 8)
 *   max_draft  an upper bound of the drafts of a sequence, 1 .. 256 (a longer
 *     prompt takes several calls, chains over the ones before; each reads all
 *     keys so far)
 *   mask  [N][mask_words] uint32, mask_words * 32 >= max_draft, or NULL
 *   o     [N][Hq][D] in o_dtype (QMV_F32 or the cache's), 16-byte aligned
 *   lse   [N][Hq] fp32
 *   acc_in, acc_out  [pages][Hkv][page] fp32: acc_out NULL: no weights; acc_in
 *     NULL: counts as zeros; both may be the same array. Slots that no
 *     sequence with new tokens holds are not touched: a sequence without any
 *     takes no step, and its sums do not decay.
 *   ws  at least attn_tree_workspace_bytes(...) bytes, 256-byte aligned, not
 *     shared with a concurrent call. */
int attn_tree(const qmv_attn_cache *c, const void *q, int64_t q_stride, int Hq,
              const int32_t *table, int max_pages, const int32_t *ctx, const int32_t *cu, int B,
              int N, int max_draft, const uint32_t *mask, int mask_words, float scale, void *o,
              int o_dtype, float *lse, const float *acc_in, float *acc_out, float decay,
              int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* Workspace of attn_window, in bytes (0 for unsupported sizes). It depends on the
 * heads and on max_new alone. */
size_t attn_window_workspace_bytes(const qmv_attn_cache *c, int Hq, int B, int N, int max_new,
                                   int max_pages);

/* Causal attention of each sequence's new tokens, any number of them (a prompt,
 * a chunk of one, a single token), over its cache, new tokens included (their
 * keys and values are in their slots: attn_rope_append), with a sliding window
 * and first tokens that stay visible. Head hq reads key/value head
 * hq / (Hq / Hkv). Token n = cu[b] + t, at slot p = ctx[b] + t, sees the slots
 *     j <= p with j > p - window or j < sinks
 * (its own among them), and
 *     x_j = scale * q[n][hq] . k_j      over the slots j that it sees
 *     lse[n][hq] = log sum_j exp(x_j),  o[n][hq] = sum_j exp(x_j - lse) v_j
 * A row whose scores are all -inf gets o = 0 and lse = -inf. What a token does
 * not see never reaches its row, infinities and NaNs in stale or hidden slots
 * included. (Infinities and NaNs among the values of a key that it does see
 * leave these elements of its output infinite or NaN.) Pages without a slot that
 * one of the sequence's new tokens sees are not looked at: their table entries
 * may be anything, and they may belong to others by now. Sequences may share
 * pages. Results do not depend on the order in which thread blocks finish.
 * Scores, maxima, sums and outputs are fp32. Where max_new * Hq / Hkv is above 16
 * and o has 16 bits, every exp(x_j - M) is rounded once to the cache's type before it
 * meets its value (half a step of the weight; in all 1.4 times the error of the
 * output's own rounding); otherwise it is carried as two or three 16-bit numbers, and
 * o is off by its own rounding. So the precision of 16-bit outputs, not of fp32 ones,
 * depends on max_new.
 *   q [N] rows of Hq * D in the cache's type, 16-byte aligned, q_stride
 *     elements apart (a multiple of 8); N <= 2^22
 *   max_new  an upper bound of a sequence's new tokens, >= 1, at most 2^22 and
 *     2^30 / (Hq / Hkv); calls of up to 16 / (Hq / Hkv) take a kernel made for few rows
 *   window >= 1 (INT32_MAX: all tokens before), sinks >= 0. The work is counted in
 *     steps of 64 to 128 keys (of min(window + sinks, max_pages * page), plus a few
 *     pieces) by up to 16 rows (the kernel for few) or 128 / (Hq / Hkv) or twice as
 *     many tokens; 2^31 steps a thread block, hours of work, are refused (QMV_ESHAPE)
 *   o     [N][Hq][D] in o_dtype (QMV_F32 or the cache's), 16-byte aligned
 *   lse   [N][Hq] fp32; o and lse are not arrays that the call reads
 *   ws  at least attn_window_workspace_bytes(...) bytes, 256-byte aligned, not
 *     shared with a concurrent call. */
int attn_window(const qmv_attn_cache *c, const void *q, int64_t q_stride, int Hq,
                const int32_t *table, int max_pages, const int32_t *ctx, const int32_t *cu, int B,
                int N, int max_new, int window, int sinks, float scale, void *o, int o_dtype,
                float *lse, int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream);

/* Eviction by accumulated attention weight. Each key/value head of a sequence
 * of lens[b] tokens keeps min(lens[b], budget) of them: all when they fit,
 * else the first `sink`, the last `recent` and, of those between, the
 * budget - sink - recent with the largest acc (equal sums: the lower slot; a
 * NaN sum counts as the lowest). The kept tokens stay in order and are copied,
 * with their sums, to slots 0, 1, ... of the pages of dst_table (pages that
 * hold no token of `table`; dst may be src's pool or another of the same Hkv,
 * D and dtype). Rotations stay those of the tokens' own positions.
 *   acc [src pages][Hkv][page] fp32, 16-byte aligned, dst_acc [dst pages][Hkv][dst page] fp32
 *   dst_table [B][dst_max_pages] int32, with room for the kept tokens
 *   keep [B][Hkv][budget] int32: the kept slots, ascending, then -1 (written)
 *   new_lens [B] int32: min(lens[b], budget) (written)
 *   budget >= 1; sink, recent >= 0, sink + recent <= budget.
 * A sequence whose length does not fit the table keeps nothing (status 2). */
int attn_evict(const qmv_attn_cache *src, const float *acc, const int32_t *table, int max_pages,
               const int32_t *lens, int B, int budget, int sink, int recent,
               const qmv_attn_cache *dst, float *dst_acc, const int32_t *dst_table,
               int dst_max_pages, int32_t *keep, int32_t *new_lens, int32_t *status,
               qmv_stream_t stream);

/* ---------------------------------------------------------------- pages
 *
 * The upkeep of a cache's pages, for page tables as the attention calls take
 * them. refs [pages] int32 counts the table entries that hold a page (0: it is
 * free); a program starts with zeros and tables of -1 and lets the calls below
 * keep both. One pool of pages serves the caches of all layers that use the same
 * table. Everything is on the device and stream-ordered, so a captured step can
 * take and give back pages.
 *   table  [n][max_pages] int32, page of each `page` tokens; below 0: none
 *   page   16, 32, 64, 128 or 256; pages <= 2^30; n <= 65535;
 *          max_pages * page <= 2^30; n * max_pages < 2^31
 *   status [1] int32 or NULL, OR-ed with
 *            1  an id past the pool in an entry, a page given back that nobody held,
 *               or a parent's last, partly filled page that is not there: that entry
 *               is left out (attn_pages_fork: the child ends before it);
 *            2  lengths (or a parent) that are negative or do not fit: that row is
 *               left as it is (attn_pages_fork: the child is empty);
 *            8  no free page was left for some entry.
 *   ws     at least the bytes that the call's workspace function says, 256-byte
 *          aligned, not shared with a concurrent call. */

size_t attn_pages_update_workspace_bytes(int pages, int B, int max_pages);

/* Makes each row of a table hold the pages that its sequence needs, and no others.
 * Sequence b has lens[b] tokens in the cache and is to take more[b] (0 and 0: it is
 * over). With the window and sinks of attn_window, page i is needed when
 *     i * page < lens + more   and
 *     (i * page < sinks  or  (i + 1) * page > lens - window + 1)
 * that is, when it has or will have tokens that a token to come (at slot lens or
 * later) sees. Entries that are not needed give their pages back and become -1;
 * then the needed ones that are below 0 take the lowest free pages, in the order
 * of the sequences and of their entries (a page given back in this call can be
 * taken in it). When the free ones run out the rest stay below 0 (status 8).
 * Tokens are to be appended only to pages that their sequence holds alone:
 * attn_pages_fork leaves it so; a sequence that is cut back into a page it shares
 * is forked (from itself) first.
 *   refs, table  updated in place, and share no bytes with lens, more or one another
 *   window >= 1 (INT32_MAX: none), sinks >= 0 */
int attn_pages_update(int32_t *refs, int pages, int page, int32_t *table, int max_pages,
                      const int32_t *lens, const int32_t *more, int B, int window, int sinks,
                      int32_t *status, void *ws, size_t ws_bytes, qmv_stream_t stream);

size_t attn_pages_fork_workspace_bytes(int pages, int F);

/* F children of sequences: child f begins as parent[f] (0 .. B - 1) is, lens tokens
 * long. Whole pages are shared (their refs grow); a last page that is partly filled
 * is replaced by the lowest free page, and moves[f] says what to copy to it:
 * (page to copy from, page to copy to, tokens), or (-1, -1, 0). attn_pages_copy
 * copies it, in each layer's cache. A child for which no page is left (status 8), or
 * whose parent's partly filled page is not there (status 1), is as long as its whole
 * pages. Parents keep what they hold until attn_pages_update takes it back.
 *   new_table [F][max_pages], new_lens [F], moves [F][3] int32 (written); they
 *   share no bytes with one another or with what the call reads */
int attn_pages_fork(int32_t *refs, int pages, int page, const int32_t *table, int max_pages,
                    const int32_t *lens, int B, const int32_t *parent, int F, int32_t *new_table,
                    int32_t *new_lens, int32_t *moves, int32_t *status, void *ws, size_t ws_bytes,
                    qmv_stream_t stream);

/* Copies the first tokens of pages, keys and values of all heads: moves [n][3]
 * int32, (page of src, page of dst, tokens); a move with a page below 0 or without
 * tokens is none. dst may be src or another cache with the same heads, page and
 * dtype (and any number of pages). No page is the source of one move and the
 * destination of another, or the destination of two. Pages past a pool are left
 * out (status 1), token counts outside 0 .. page too (status 2).
 *   src_acc, dst_acc  running attention weights [pages][Hkv][page] or NULL: with
 *     dst_acc alone the copies' weights are cleared */
int attn_pages_copy(const qmv_attn_cache *src, const qmv_attn_cache *dst, const int32_t *moves, int n,
                    const float *src_acc, float *dst_acc, int32_t *status, qmv_stream_t stream);

/* Keeps some of each sequence's new tokens (the accepted ones of a tree of drafts):
 * token keep[cu[b] + i], counted from the sequence's first new one, moves to slot
 * ctx[b] + i, i < kept[b], in all heads, with its running weights where acc is
 * given; new_ctx[b] = ctx[b] + kept[b]. The kept ones are in strictly ascending
 * order (a path's drafts are). table, ctx, cu as in the attention calls; the pages
 * of new tokens belong to one sequence. A sequence whose lengths do not fit, or
 * whose kept tokens are not ascending or not its own, stays as it is
 * (status 2); moves from or to pages past the pool are left out (status 1).
 *   keep [N] int32, kept [B] int32; acc [pages][Hkv][page] or NULL (in place)
 *   new_ctx [B] int32 (written); it shares no bytes with what the call reads */
int attn_compact(const qmv_attn_cache *c, const int32_t *table, int max_pages, const int32_t *ctx,
                 const int32_t *cu, int B, int N, const int32_t *keep, const int32_t *kept, float *acc,
                 int32_t *new_ctx, int32_t *status, qmv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_H */
