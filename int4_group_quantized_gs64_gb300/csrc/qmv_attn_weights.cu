// qmv_attn_weights.cu - the attention weights of the cached tokens:
//     acc_out[j] = decay * acc_in[j] + sum over the rows of a head of exp(x_j - lse)
//
// A weight needs its row's lse, and so the whole pass over the keys before it.
// What the pass can leave behind, or what has to be done again, depends on
// the rows R of a key/value head:
//   up to 16      k_attn_rows leaves its scores (8 R bytes a key, written and
//                 read); k_weights_stash turns them into weights, a thread a key.
//                 32 sequences of 10,007 keys, 6 rows: 181 us with the attention,
//                 243 with the scores formed again.
//   more, or scores too many to keep
//                 k_weights_tc forms the scores again (2 D bytes a key), keys as
//                 the rows of the tcgen05 product, so that a thread has one key
//                 and sums its own columns: S^T = K Q^T, up to 512 queries resident
//                 in shared memory while the keys stream by once (a launch for
//                 every 512, each adding to the last one's sums).
// What bounds k_weights_tc: 64 sequences of 8191 keys, 128 rows: 195 us, 5.5 TB/s
// of keys. Small trees pay for the start of a block's parts (16 sequences of up to
// 6000 keys of 64 elements, 105 rows: 35 us, a third of which is the first copies
// and queries); the exponentials are not the limit (some of them as polynomials on
// the fp32 pipe: 82.8 -> 84.5 us with the attention).
#include <string.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_plan.cuh"
#include "qmv_attn_tc05.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

// ------------------------------------------------------------------ from kept scores

// A thread takes four keys. vec: the sums lie on 16-byte boundaries.
__global__ void __launch_bounds__(256) k_weights_stash(const TreeArgs a, bool vec) {
    __shared__ float e2[16];
    const int b = blockIdx.z, h = blockIdx.y, slot = (blockIdx.x * 256 + threadIdx.x) * 4;
    bool ok;
    const Seq q = get_seq(a.s, b, ok);  // (a call's inputs are older than its first kernel)
    const int len = q.ctx + q.T, nrows = q.T * a.G;
    const bool any = q.T > 0 && blockIdx.x * 1024 < len;
    int pid = -1;
    if (any && slot < len) pid = a.s.table[(long long)b * a.s.max_pages + (slot >> a.s.lpage)];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!any) return;
    if (threadIdx.x < nrows) {
        const int t = div_g(a, threadIdx.x);
        e2[threadIdx.x] =
            a.lse[(long long)(q.first + t) * a.Hq + h * a.G + threadIdx.x - t * a.G] * kLog2e;
    }
    __syncthreads();
    if ((unsigned)pid >= (unsigned)a.pages) return;
    const long long at = ((long long)pid * a.Hkv + h) * a.s.page + (slot & (a.s.page - 1));
    const float *p = stash_at(a, b, h, slot & ~15) + (slot & 15);
    const int n = min(4, len - slot);
    const bool whole = vec && n == 4;
    float old[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.acc_in) {
        if (whole) {
            const float4 f = *reinterpret_cast<const float4 *>(a.acc_in + at);
            old[0] = f.x; old[1] = f.y; old[2] = f.z; old[3] = f.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) old[e] = a.acc_in[at + e];
        }
    }
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < nrows; r0 += 8) {
        float4 x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            x[r] = r0 + r < nrows ? __ldcs(reinterpret_cast<const float4 *>(p + (r0 + r) * 16))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r0 + r < nrows && e2[r0 + r] != -INFINITY) {
                const float e = e2[r0 + r];
                w[0] += ex2(fmaf(x[r].x, a.sl2, -e));
                w[1] += ex2(fmaf(x[r].y, a.sl2, -e));
                w[2] += ex2(fmaf(x[r].z, a.sl2, -e));
                w[3] += ex2(fmaf(x[r].w, a.sl2, -e));
            }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] += a.decay * old[e];
    if (whole) {
        *reinterpret_cast<float4 *>(a.acc_out + at) = make_float4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) a.acc_out[at + e] = w[e];
    }
}

// ------------------------------------------------------------------ from the keys again

constexpr int kThreads = 352, kKeys = 128, kStages = 12, kSmemMax = 227 * 1024, kMaxRows = 512;

struct alignas(16) Misc {
    ShareScratch<kThreads / 32> share;
    uint64_t full[kStages], empty[kStages], s_full[4], s_free[4], q_full, fin;
    uint32_t tmem, dead;
    int tiles, row_tiles;
    alignas(16) float nlse[kMaxRows];  // -lse in log2 units; -inf where a row has no weights
    uint32_t seen[2][8][128];  // of a tile with drafts: the drafts that see each key
};
constexpr int kMisc = 11264;
static_assert(sizeof(Misc) <= kMisc, "");

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Misc *m, int32_t *status) {
    const uint32_t b = tc05::smem_addr(bar);
    volatile uint32_t *dead = &m->dead;
#pragma unroll 1
    for (uint32_t i = 0; i < kPoll; ++i) {
        if (try_wait(b, parity)) return true;
        if ((i & 255) == 255 && *dead) return false;
    }
    *dead = 1;
    set_status(status, kStTimeout);
    return false;
}

// a.rows is so large that an item is a (sequence, head), and a.unit 128 keys.
// Warps 0-3 and 4-7 take alternate key tiles, 8 and 10 copy them, 9 issues the
// products of a tile with every 128 queries into four score tiles of tensor
// memory: two for each group of warps, by turns. (With all four by turns, a tile
// with four products would lie in the buffers of the other group's last one, whose
// phases this group has not seen: a wait two phases behind passes at once.)
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    k_weights_tc(const __grid_constant__ CUtensorMap kmap, const TreeArgs a, int row0, int q_tiles, int stages) {
    constexpr int kTile = kKeys * D * 2, kHalves = D / 64;
    constexpr uint32_t kIdesc = tc05::idesc_f16kind_f32(kBf16, 128, 128, false);
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *qs = smem, *ring = smem + q_tiles * kTile;
    Misc *m = reinterpret_cast<Misc *>(ring + stages * kTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A call's inputs are older than its first kernel: only lse and the sums
    // have to wait for the kernels before.
    const Share sh = find_share<kThreads>(a, &m->share);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (sh.u0 >= sh.u1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            tc05::mbar_init(m->full + i, 1);
            tc05::mbar_init(m->empty + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc05::mbar_init(m->s_full + i, 1);
            tc05::mbar_init(m->s_free + i, 4);
        }
        tc05::mbar_init(&m->q_full, 256);
        tc05::mbar_init(&m->fin, 1);
        m->dead = 0;
        tc05::fence_mbar_init();
        prefetch_tmap(&kmap);
    }
    if (warp == 9) tc05::tmem_alloc(&m->tmem, 512);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = m->tmem;
    const int units = (int)(sh.u1 - sh.u0);

    if (warp == 8 || warp == 10) {
        // (two warps, a tile each in turn: with small pages one's issue does not keep up)
        const int prow = a.s.page < kKeys ? a.s.page : kKeys;
        Cursor c;
        c.start(a, sh);
        int stage = 0, x = 0;  // the tile that the cursor is at
        uint32_t phase = 1, pending = 0, pending_ph = 0;
        bool ok = true;
        auto step = [&]() {
            ++x;
            if (++stage == stages) {
                stage = 0;
                phase ^= 1;
            }
            if (++c.u == c.nu && x < units) c.next_item(a);
        };
        int slot = 0, pid = -1;
        auto fetch = [&]() {  // this lane's piece of the cursor's tile: its page
            slot = c.u * kKeys + lane * prow;
            pid = lane * prow < kKeys && slot < c.q.ctx + c.q.T
                      ? __ldg(a.s.table + (long long)c.b * a.s.max_pages + (slot >> a.s.lpage))
                      : -1;
        };
        if (warp == 10) step();
        if (x < units) fetch();
        while (x < units) {
            // this tile's, then the next one's page ids are under way
            const bool good = (unsigned)pid < (unsigned)a.pages;
            const int row = (pid * a.Hkv + c.h) * a.s.page + (slot & (a.s.page - 1)), st = stage;
            const uint32_t ph = phase;
            step();
            if (x < units) step();
            if (x < units) fetch();
            const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, good));
            ok = wait(m->empty + st, ph, m, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) {
                if (n)
                    mbar_expect_tx(m->full + st, n * prow * D * 2);
                else
                    mbar_arrive(m->full + st);
            }
            __syncwarp();
            if (good) {
                const uint32_t dst = tc05::smem_addr(ring) + st * kTile + lane * prow * 128;
#pragma unroll
                for (int hf = 0; hf < kHalves; ++hf)
                    tma_load3(dst + hf * (kKeys * 128), &kmap, 0, row, hf, m->full + st);
            }
            pending |= 1u << st;
            pending_ph = (pending_ph & ~(1u << st)) | ((ph ^ 1u) & 1u) << st;
        }
        if (!ok)  // gave up: wait (bounded) for this warp's copies in flight
            for (int i = 0; i < stages; ++i)
                if ((pending >> i) & 1u) tc05::mbar_wait(m->full + i, (pending_ph >> i) & 1u, kPoll / 64);
    } else if (warp == 9) {
        if (lane == 0) {
            const uint64_t kdesc = tc05::sdesc_sw128(tc05::smem_addr(ring));
            const uint64_t qdesc = tc05::sdesc_sw128(tc05::smem_addr(qs));
            int stage = 0, jobs[2] = {0, 0};  // products so far, of each group
            uint32_t phase = 0, qp = 0;
            bool live = true;
            for (int left = units; left > 0 && live;) {
                live = wait(&m->q_full, qp, m, a.status);
                qp ^= 1u;
                const int n = *(volatile int *)&m->tiles, nq = *(volatile int *)&m->row_tiles;
                left -= n;
#pragma unroll 1
                for (int t = 0; t < n && live; ++t) {
                    live = wait(m->full + stage, phase, m, a.status);
                    const uint64_t kd = kdesc + (uint32_t)(stage * (kTile >> 4));
                    const int grp = t & 1;
                    int job = grp ? jobs[1] : jobs[0];
#pragma unroll 1
                    for (int r = 0; r < nq && live; ++r, ++job) {
                        const int buf = 2 * grp + (job & 1);
                        if (job >= 2)
                            live = wait(m->s_free + buf, ((job >> 1) - 1) & 1, m, a.status);
                        if (!live) break;
                        tc05::fence_after_sync();
                        const uint64_t qd = qdesc + (uint32_t)(r * (kTile >> 4));
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const int of = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                            tc05::mma_ss(tmem + buf * 128, kd + of, qd + of, kIdesc, k > 0);
                        }
                        tc05::mma_commit(m->s_full + buf);
                    }
                    if (grp)
                        jobs[1] = job;
                    else
                        jobs[0] = job;
                    tc05::mma_commit(m->empty + stage);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            tc05::mma_commit(&m->fin);
            tc05::mbar_wait(&m->fin, 0, kPoll);
        }
        __syncwarp();
    } else {
        const int s = warp >> 2, tid = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        Cursor c;
        c.start(a, sh);
        int job = 0;  // this group's products so far
        bool waited = false;
        const uint64_t sl2 = pack_f32x2(a.sl2, a.sl2);
        for (int left = units; left > 0;) {
            const Seq q = c.q;
            const int j0 = c.u, n = min(c.nu - c.u, left), nrows = min(q.T * a.G - row0, kMaxRows);
            const int nq = (nrows + 127) / 128;
            // queries, and -lse of each. Past the last row its query again, with no
            // weight: zeros there would make a NaN of a key's infinity, where the
            // last row's score is one that counts anyway.
            constexpr int kChunks = D / 8, kPass = 256 / kChunks;
            const int ch = threadIdx.x % kChunks;
            const uint16_t *p = a.q + (long long)q.first * a.q_stride + (long long)c.h * a.G * D + ch * 8;
            uint8_t *dst = qs + (ch >> 3) * (kKeys * 128);
#pragma unroll 1
            for (int rt = 0; rt < nq; ++rt) {
                uint4 v[128 / kPass];
#pragma unroll
                for (int i = 0; i < 128 / kPass; ++i) {
                    const int rr = row0 + min(rt * 128 + (int)threadIdx.x / kChunks + i * kPass, nrows - 1);
                    const int t = div_g(a, rr);
                    v[i] = __ldg(reinterpret_cast<const uint4 *>(p + t * a.q_stride + (rr - t * a.G) * D));
                }
#pragma unroll
                for (int i = 0; i < 128 / kPass; ++i) {
                    const int r = threadIdx.x / kChunks + i * kPass;
                    *reinterpret_cast<uint4 *>(dst + rt * kTile + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                        make_uint4((v[i].x ^ a.qxor) & a.qand, (v[i].y ^ a.qxor) & a.qand,
                                   (v[i].z ^ a.qxor) & a.qand, (v[i].w ^ a.qxor) & a.qand);
                }
            }
            tc05::fence_proxy_async();
            if (threadIdx.x == 0) {
                m->tiles = n;
                m->row_tiles = nq;
            }
            mbar_arrive(&m->q_full);
            if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
            for (int r = threadIdx.x; r < nq * 128; r += 256) {
                float e = -INFINITY;
                if (r < nrows) {
                    const int t = div_g(a, row0 + r);
                    e = -a.lse[(long long)(q.first + t) * a.Hq + c.h * a.G + row0 + r - t * a.G] * kLog2e;
                    if (e == INFINITY) e = -INFINITY;
                }
                m->nlse[r] = e;
            }
            __syncwarp();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            // a tile's page id is loaded two of this warpgroup's tiles ahead, its
            // old sum one ahead
            auto page_of = [&](int t) {
                const int slot = (j0 + t) * kKeys + tid;
                return t < n && slot < q.ctx + q.T
                           ? __ldg(a.s.table + (long long)c.b * a.s.max_pages + (slot >> a.s.lpage))
                           : -1;
            };
            auto place_of = [&](int t, int pid) {
                const int slot = (j0 + t) * kKeys + tid;
                return (unsigned)pid < (unsigned)a.pages
                           ? ((long long)pid * a.Hkv + c.h) * a.s.page + (slot & (a.s.page - 1))
                           : -1LL;
            };
            int pid1 = page_of(s + 2);
            long long at1 = place_of(s, page_of(s));
            float old1 = at1 >= 0 && a.acc_in ? a.acc_in[at1] : 0.f;
#pragma unroll 1
            for (int t = s; t < n; t += 2) {
                const int slot = (j0 + t) * kKeys + tid;
                const int d = slot - q.ctx;  // this key's draft (negative: seen by all)
                const bool special = (j0 + t + 1) * kKeys > q.ctx;
                const long long at = at1;
                const float old = old1;
                at1 = place_of(t + 2, pid1);
                old1 = at1 >= 0 && a.acc_in ? a.acc_in[at1] : 0.f;
                pid1 = page_of(t + 4);
                if (special) {  // which drafts see this key, as bits
                    const bool all = d < 0 || !a.mask;
#pragma unroll 1
                    for (int w = 0; w < 8; ++w) {
                        uint32_t bits = 0;
                        for (int e = 0; e < 32 && w * 32 + e < q.T; ++e) {
                            const int tt = w * 32 + e;
                            const bool see = all ? d <= tt
                                                 : d < q.T && ((__ldg(a.mask + (long long)(q.first + tt) * a.words +
                                                                      (d >> 5)) >> (d & 31)) & 1u);
                            bits |= (uint32_t)see << e;
                        }
                        m->seen[s][w][tid] = bits;
                    }
                    __syncwarp();
                }
                uint64_t sum[2] = {0, 0};
#pragma unroll 1
                for (int r = 0; r < nq; ++r, ++job) {
                    const int buf = 2 * s + (job & 1);
                    wait(m->s_full + buf, (job >> 1) & 1, m, a.status);
                    __syncwarp();
                    tc05::fence_after_sync();
                    if (special) {  // scores of rows that do not see the key become -inf
                        int tt = div_g(a, row0 + r * 128), gg = row0 + r * 128 - tt * a.G;  // row's draft and head
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t x[32];
                            tc05::tmem_ld32(tmem + lanes + buf * 128 + k * 32, x);
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const uint32_t w = m->seen[s][(tt >> 5) & 7][tid];
                                if (!((w >> (tt & 31)) & 1u)) x[e] = 0xFF800000u;
                                if (++gg == a.G) {
                                    gg = 0;
                                    ++tt;
                                }
                            }
                            tc05::tmem_st32(tmem + lanes + buf * 128 + k * 32, x);
                        }
                        tc05::tmem_wait_st();
                    }
                    uint32_t x[2][32];
                    tc05::tmem_ld32(tmem + lanes + buf * 128, x[0]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        tc05::tmem_wait_ld();
                        if (k < 3) tc05::tmem_ld32(tmem + lanes + buf * 128 + (k + 1) * 32, x[(k + 1) & 1]);
                        const ulonglong2 *nl = reinterpret_cast<const ulonglong2 *>(m->nlse + r * 128 + k * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const ulonglong2 nb = nl[e];
                            float p0, p1, p2, p3;
                            unpack_f32x2(fma_f32x2(pack_u32x2(x[k & 1][4 * e], x[k & 1][4 * e + 1]), sl2, nb.x), p0, p1);
                            unpack_f32x2(fma_f32x2(pack_u32x2(x[k & 1][4 * e + 2], x[k & 1][4 * e + 3]), sl2, nb.y), p2, p3);
                            sum[0] = add_f32x2(sum[0], pack_f32x2(ex2(p0), ex2(p1)));
                            sum[1] = add_f32x2(sum[1], pack_f32x2(ex2(p2), ex2(p3)));
                        }
                    }
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m->s_free + buf);
                }
                if (at >= 0) {
                    float s0, s1, s2, s3;
                    unpack_f32x2(sum[0], s0, s1);
                    unpack_f32x2(sum[1], s2, s3);
                    a.acc_out[at] = a.decay * old + ((s0 + s1) + (s2 + s3));
                }
            }
            __syncwarp();
            asm volatile("bar.sync 1, 256;" ::: "memory");
            left -= n;
            if (left > 0) c.next_item(a);
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    if (warp == 9) tc05::tmem_dealloc(tmem, 512);
}

template <int D, bool kBf16>
cudaError_t run(const AttnCache &c, const TreeArgs &a, int max_rows, cudaStream_t st) {
    const long long most = (long long)a.s.max_pages << a.s.lpage;
    if (a.stash)
        return launch(k_weights_stash, dim3((unsigned)((most + 1023) / 1024), a.Hkv, a.s.B), dim3(256),
                      0, st, true, a,
                      ((reinterpret_cast<uintptr_t>(a.acc_in) | reinterpret_cast<uintptr_t>(a.acc_out)) & 15) == 0);
    constexpr int kTile = kKeys * D * 2;
    TreeArgs w = a;
    w.rows = 1 << 30;
    w.unit = kKeys;
    const long long units = (long long)a.s.B * a.Hkv * ((most + kKeys - 1) / kKeys);
    w.grid = units < sm_count() ? (int)units : sm_count();
    CUtensorMap km;
    if (!encode_pool(&km, c.k, c, c.page < kKeys ? c.page : kKeys, false))
        return cudaErrorNotSupported;
    auto *k = k_weights_tc<D, kBf16>;
    cudaError_t e = set_smem(k, kSmemMax);
    for (int row0 = 0; row0 < max_rows && e == cudaSuccess; row0 += kMaxRows) {
        // Only sequences that have rows from row0 on: in a part without products
        // nothing would hold the softmax warps until its tables have been read.
        w.s.min_draft = row0 / w.G + 1;
        const int rows = max_rows - row0 < kMaxRows ? max_rows - row0 : kMaxRows;
        const int q_tiles = (rows + 127) / 128;
        int stages = (kSmemMax - kMisc - q_tiles * kTile) / kTile;
        if (stages > kStages) stages = kStages;
        e = launch(k, dim3(w.grid), dim3(kThreads), kSmemMax, st, true, km, w, row0, q_tiles, stages);
        w.acc_in = w.acc_out;  // further rows add to what these leave
        w.decay = 1.f;
    }
    return e;
}

}  // namespace

cudaError_t launch_tree_weights(const AttnCache &c, const TreeArgs &a, int max_rows,
                                cudaStream_t st) {
    if (c.D == 64)
        return c.bf16 ? run<64, true>(c, a, max_rows, st) : run<64, false>(c, a, max_rows, st);
    return c.bf16 ? run<128, true>(c, a, max_rows, st) : run<128, false>(c, a, max_rows, st);
}

}  // namespace attn
}  // namespace qmv
