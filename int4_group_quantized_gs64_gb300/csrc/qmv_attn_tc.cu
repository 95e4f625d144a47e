// qmv_attn_tc.cu - tree attention of many rows on the tcgen05 tensor cores.
//
// From some tens of rows on, a key's products cost more than the warp MMA
// gives while the key streams in (128 rows: 128 products a loaded byte; the
// GPU's ratio of tensor rate to bandwidth is near 290), so the scores and the
// output come from tcgen05: S = Q K^T with both operands in shared memory,
// O += P V with P in tensor memory.
//
// A block keeps two streams in flight, each with its own scores S (128
// columns of tensor memory, overwritten by the weights P) and its own O, so
// that one stream's products run under the other's exponentials:
//   rows <= 128: one tile of 128 rows; the streams take alternate key tiles
//                and are joined at the segment's end (in tensor memory, where
//                both have the same row on the same lane);
//   rows  > 128: two tiles of 128 rows against the same key tiles.
// Warps: 0-3 and 4-7 the streams' softmax (a thread a row: maximum and sum
// need no exchange), 8 and 11 the copies of keys and of values, 9 and 10 the
// streams' products. These four need few registers and pass the rest on to the
// softmax warps, whose 128 scores stay in registers (reading them from tensor
// memory twice would cost as much as the products). That is more than 216
// registers hold with everything else: 16-bit outputs spill some 50 bytes a thread
// with more than 128 rows and some 200 with up to 128. For fp32 outputs, whose O
// takes 128 registers at 128 elements, the scores are read 32 at a time twice, and
// 550 bytes are spilled with more than 128 rows, 1.2 to 1.4 KB with up to 128.
//
// A ring of 128-key tiles holds keys and another one values, across segments; a
// copying warp comes to every slot of its ring in turn, and so never waits for a
// phase that is not the next. (In one ring for both it would know of its own entries
// only, and those that other slots imply are the other stream's: a wait two phases
// behind passes at once.) The running maximum moves only when it grows by more than
// 2^8 (a row's weights may then exceed 1, which fp32 sums and 16-bit weights hold),
// since moving it means rescaling O in tensor memory.
//
// What bounds it: a stream's chain of scores, exponentials, weights and product,
// 3,380 cycles for a 128-key tile and 256 rows of 128 elements (the products alone
// are 2,048), and some 15,000 cycles at the start and end of a block's parts.
// 8 trees of 64 nodes, 8 query heads a head, up to 8200 keys: 114 us with the
// join (830 TFLOP/s); 64 sequences of 8191 keys, 32 rows: 244 us, the rate of a copy.
//
// Weights are rounded once to 16 bits for a 16-bit output (half a step of the
// type, like the output's own rounding, and averaged over the keys). For an
// fp32 output they are carried as two fp16 or three bf16 numbers (two bf16 ones:
// 2.3e-6 of the output's norm; fp32 weights and sums: 1.5e-6), and O is summed up
// in registers, tile by tile: a product's own sums cut off what falls below
// their last bit, which over 8191 keys came to 1.1e-5 of the norm. fp16 weights
// are held 2^7 times larger: the small ones would lose bits below fp16's range.
// (256 rows over 16 x 8191 keys: 111 us with a 16-bit output, 205 and 285 with an
// fp32 one from fp16 and bf16.)
#include <string.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_plan.cuh"
#include "qmv_attn_tc05.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

constexpr int kThreads = 384, kKeys = 128, kMaxStages = 12;
constexpr int kMisc = 2880;               // barriers and small tables
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 units the maximum may lag

struct Misc {
    ShareScratch<kThreads / 32> share;
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t s_full[2], p_ready[2], o_full[2], q_full, fin[2], turn[2], s_free[2], pv_done[2];
    uint32_t tmem, dead;
    int tiles;             // of the segment whose queries are ready
    uint32_t nf[8];        // drafts with infinities or NaNs among their values
    float2 ml[2][128];
};
static_assert(sizeof(Misc) <= kMisc, "");

// Waits for a barrier's phase; gives up after a bounded time, or at once when
// another warp has given up. (Not inlined: the softmax loop's code should
// stay small in the instruction cache.)
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Misc *m, int32_t *status) {
    volatile uint32_t *dead = &m->dead;
#pragma unroll 1
    for (uint32_t i = 0; i < kPoll; ++i) {
        if (try_wait(bar, parity)) return true;
        if ((i & 255) == 255 && *dead) return false;
    }
    *dead = 1;
    set_status(status, kStTimeout);
    return false;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Misc *m, int32_t *status) {
    const uint32_t b = tc05::smem_addr(bar);
    return try_wait(b, parity) || wait_slow(b, parity, m, status);
}

__device__ __forceinline__ void pair_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool pair_or(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p)
        : "memory");
    return r != 0;
}

// The upper halves of two floats, which are bf16 numbers, and what they leave.
__device__ __forceinline__ uint32_t cut_bf16x2(float &x, float &y) {
    const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
    x -= __uint_as_float(u & 0xFFFF0000u);
    y -= __uint_as_float(v & 0xFFFF0000u);
    return __byte_perm(u, v, 0x7632);
}

// A block's part of an item: tiles [j0, j0 + n) of the item's keys.
struct Segment {
    int j0, n;
    bool whole;
    __device__ __forceinline__ Segment(const Cursor &c, int left) {
        j0 = c.u;
        n = min(c.nu - c.u, left);
        whole = j0 == 0 && n == c.nu;
    }
};

template <int D, bool kBf16, bool kTwo, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              const TreeArgs a, int stages) {
    constexpr int kTile = kKeys * D * 2, kHalves = D / 64;
    constexpr uint32_t kIdescS = tc05::idesc_f16kind_f32(kBf16, 128, kKeys, false);
    extern __shared__ __align__(1024) uint8_t smem[];
    // Tensor memory columns. Where they suffice (64 elements, one 16-bit number a
    // weight) P lies apart from S, and a stream's next S is formed while its
    // exponentials run (16 sequences of 8191 keys, 320 rows: 124 us, 150 with P
    // over S; 64 sequences, 128 rows: 165 and 182). Otherwise P overwrites S.
    constexpr bool kApart = D == 64 && !kSplit;
    // The third number of a bf16 weight lies in columns that O leaves: with 128
    // elements O comes in two halves, one after the other.
    constexpr bool kThird = kSplit && kBf16, kParted = kThird && D == 128;
    constexpr int kOcols = kParted ? 64 : D;  // columns a product gives
    constexpr uint32_t kIdescO = tc05::idesc_f16kind_f32(kBf16, 128, kOcols, true);
    constexpr int kPcol = kApart ? 256 : 0, kPstep = kApart ? 64 : 128;   // P of stream s at kPcol + s * kPstep
    constexpr int kOcol = kApart ? 384 : 256, kOstep = kApart ? 64 : 128;
    // Slots for keys, then those for values: half of them each. (Of five, three for
    // keys or three for values measured the same.)
    const int kstages = stages / 2, vstages = stages - kstages;
    uint8_t *qs = smem, *ring = smem + (kTwo ? 2 : 1) * kTile;
    Misc *m = reinterpret_cast<Misc *>(ring + stages * kTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            tc05::mbar_init(m->full + i, 1);
            tc05::mbar_init(m->empty + i, kTwo ? 2 : 1);  // both streams read a tile, or one
        }
        for (int s = 0; s < 2; ++s) {
            tc05::mbar_init(m->s_full + s, 1);
            tc05::mbar_init(m->p_ready + s, 4);
            tc05::mbar_init(m->o_full + s, 1);
            tc05::mbar_init(m->fin + s, 1);
            tc05::mbar_init(m->turn + s, 4);
            tc05::mbar_init(m->s_free + s, 4);
            tc05::mbar_init(m->pv_done + s, 1);
        }
        tc05::mbar_init(&m->q_full, 256);
        m->dead = 0;
        tc05::fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && a.status) {
        for (int b = threadIdx.x; b < a.s.B; b += kThreads) {
            bool ok;
            get_seq(a.s, b, ok);
            if (!ok) set_status(a.status, kStLength);
        }
    }
    const Share sh = find_share<kThreads>(a, &m->share);
    if (sh.u0 >= sh.u1) return;
    if (warp == 9) tc05::tmem_alloc(&m->tmem, 512);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = m->tmem;

    const int units = (int)(sh.u1 - sh.u0);  // (the launcher keeps this below 2^31)

    // 168 x 384 registers at launch = 216 x 256 + 72 x 128
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 || warp == 11) {
        // ------------------------------------------------------------ copies
        // warp 8 the keys, 11 the values: a copy is a whole page at most, and
        // with small pages one warp's issue does not keep up (16-token pages, 64
        // elements: a tile's eight copies take some 1,100 cycles)
        const bool keys = warp == 8;
        const CUtensorMap *map = keys ? &kmap : &vmap;
        // read once: first to leave L2 (not by several row blocks, nor keys that
        // the weights' pass reads again)
        const bool once = a.max_rows <= a.rows && !(keys && a.acc_out);
        const uint64_t policy = evict_first_policy();
        const int prow = a.s.page < kKeys ? a.s.page : kKeys;  // rows a copy
        Cursor c;
        c.start(a, sh);
        const int slot0 = keys ? 0 : kstages, slot1 = keys ? kstages : stages;  // this warp's ring
        int stage = slot0;
        uint32_t phase = 1;  // a fresh barrier counts as passed for parity 1
        // this lane's piece of tile j of the sequence at c: its page
        auto page_of = [&](int j, bool &lv) {
            const int slot = j * kKeys + lane * prow;
            lv = lane * prow < kKeys && slot < c.q.ctx + c.q.T;
            return lv ? __ldg(a.s.table + (long long)c.b * a.s.max_pages + (slot >> a.s.lpage)) : 0;
        };
        bool live;
        int pid = page_of(c.u, live);
        bool ok = true;
        uint32_t pending = 0, pending_ph = 0;  // slots this warp copied to, and the phase that ends it
        for (int left = units; left > 0;) {
            const Segment sg(c, left);
#pragma unroll 1
            for (int t = 0; t < sg.n; ++t) {
                const bool good = live && (unsigned)pid < (unsigned)a.pages;
                const int row =
                    (pid * a.Hkv + c.h) * a.s.page + (((sg.j0 + t) * kKeys + lane * prow) & (a.s.page - 1));
                if (live && !good && keys) set_status(a.status, kStPage);
                if (t + 1 < sg.n) pid = page_of(sg.j0 + t + 1, live);
                const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, good));
                ok = ok && wait(m->empty + stage, phase, m, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) continue;
                if (lane == 0) {
                    if (n)
                        mbar_expect_tx(m->full + stage, n * prow * D * 2);
                    else
                        mbar_arrive(m->full + stage);
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = tc05::smem_addr(ring) + stage * kTile + lane * prow * 128;
#pragma unroll
                    for (int hf = 0; hf < kHalves; ++hf)
                        if (once)
                            tma_load3_once(dst + hf * (kKeys * 128), map, 0, row, hf, m->full + stage, policy);
                        else
                            tma_load3(dst + hf * (kKeys * 128), map, 0, row, hf, m->full + stage);
                }
                pending |= 1u << stage;
                pending_ph = (pending_ph & ~(1u << stage)) | ((phase ^ 1u) & 1u) << stage;
                if (++stage == slot1) {
                    stage = slot0;
                    phase ^= 1u;
                }
            }
            left -= sg.n;
            if (left > 0) {
                c.next_item(a);
                pid = page_of(c.u, live);
                if (!keys) {  // the next segment's queries to L2
                    constexpr int kLines = D * 2 / 128;
                    const int r0 = c.rb * a.rows, n = min(a.rows, c.q.T * a.G - r0) * kLines;
                    for (int i = lane; i < n; i += 32) {
                        const int rr = r0 + i / kLines, t = div_g(a, rr);
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            a.q + (long long)(c.q.first + t) * a.q_stride +
                            (long long)(c.h * a.G + rr - t * a.G) * D + (i % kLines) * 64));
                    }
                }
            }
        }
        if (!ok)  // gave up: wait (bounded) for this warp's copies in flight
            for (int i = 0; i < stages; ++i)
                if ((pending >> i) & 1u) tc05::mbar_wait(m->full + i, (pending_ph >> i) & 1u, kPoll / 64);
    } else {
        // ------------------------------------------------------------ products
        // a warp a stream, so that one's waits pass under the other's products
        if (lane == 0) {
            const int s = warp - 9;
            const uint64_t kdesc = tc05::sdesc_sw128(tc05::smem_addr(ring));
            const uint64_t vdesc = tc05::sdesc_sw128_mn(tc05::smem_addr(ring + kstages * kTile), kKeys * 128);
            const uint64_t qdesc =
                tc05::sdesc_sw128(tc05::smem_addr(qs)) + (uint32_t)((kTwo ? s : 0) * (kTile >> 4));
            const uint32_t ts = tmem + s * 128, tp = tmem + kPcol + s * kPstep, to = tmem + kOcol + s * kOstep;
            struct Place {  // in a ring: the slot of the segment's tile `at`, and its phase
                int slot = 0, at = 0;
                uint32_t ph = 0;
                __device__ __forceinline__ void go(int tile, int slots) {
                    slot += tile - at;
                    at = tile;
                    while (slot >= slots) {
                        slot -= slots;
                        ph ^= 1u;
                    }
                }
            } kp, vp;
            uint32_t pp = 0, qp = 0, fp = 0;
            bool live = true;
            auto scores = [&](int t) {  // S = Q K^T
                kp.go(t, kstages);
                live = live && wait(m->full + kp.slot, kp.ph, m, a.status);
                if (!live) return;
                const uint64_t kd = kdesc + (uint32_t)(kp.slot * (kTile >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int of = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                    tc05::mma_ss(ts, qdesc + of, kd + of, kIdescS, k > 0);
                }
                tc05::mma_commit(m->s_full + s);
                tc05::mma_commit(m->empty + kp.slot);
            };
            for (int left = units; left > 0 && live;) {
                live = wait(&m->q_full, qp, m, a.status);
                qp ^= 1u;
                const int n = *(volatile int *)&m->tiles;
                left -= n;
                constexpr int kStep = kTwo ? 1 : 2;
                const int t0 = kTwo ? 0 : s;
                if (t0 < n) scores(t0);
#pragma unroll 1
                for (int t = t0; t < n && live; t += kStep) {
                    // S of the stream's next tile, once its softmax holds this one's
                    if (kApart && t + kStep < n) {
                        live = wait(m->s_free + s, fp, m, a.status);
                        fp ^= 1u;
                        tc05::fence_after_sync();
                        scores(t + kStep);
                    }
                    // O (+)= P V
                    vp.go(t, vstages);
                    // With alternate tiles the weights first: the slot's last
                    // tile may be the other stream's, and a phase that is two
                    // behind looks like the awaited one. Once tile t has its
                    // weights the other stream is past that tile (the turns).
                    uint64_t *vfull = m->full + kstages + vp.slot;
                    if (kTwo) live = live && wait(vfull, vp.ph, m, a.status);
                    live = live && wait(m->p_ready + s, pp, m, a.status);
                    if (!kTwo) live = live && wait(vfull, vp.ph, m, a.status);
                    if (!live) break;
                    pp ^= 1u;
                    tc05::fence_after_sync();
                    const uint64_t v = vdesc + (uint32_t)(vp.slot * (kTile >> 4));
                    if (kSplit) {  // the rests, then the weights: a sum of this tile alone
#pragma unroll
                        for (int hf = 0; hf < D / kOcols; ++hf) {
                            if (hf) {  // (the first half has been taken)
                                tc05::mma_commit(m->pv_done + s);
                                live = wait(m->p_ready + s, pp, m, a.status);
                                if (!live) break;
                                pp ^= 1u;
                                tc05::fence_after_sync();
                            }
#pragma unroll
                            for (int part = kThird ? 2 : 1; part >= 0; --part)
#pragma unroll
                                for (int k = 0; k < kKeys / 16; ++k)
                                    tc05::mma_ts(to, part == 2 ? to + 64 + k * 8 : tp + k * 16 + part * 8,
                                                 v + (hf * (kKeys * 128) + k * 2048 >> 4), kIdescO,
                                                 part < (kThird ? 2 : 1) || k > 0);
                        }
                    } else
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            tc05::mma_ts(to, tp + k * 8, v + k * (2048 >> 4), kIdescO, !(t == t0 && k == 0));
                    tc05::mma_commit(m->empty + kstages + vp.slot);
                    if (kApart || kSplit) tc05::mma_commit(m->pv_done + s);
                    if (t + kStep >= n)
                        tc05::mma_commit(m->o_full + s);
                    else if (!kApart)
                        scores(t + kStep);
                }
                if (kApart && live && t0 < n) {  // (the last tile's hand-over, with nothing to follow)
                    live = wait(m->s_free + s, fp, m, a.status);
                    fp ^= 1u;
                }
                // A stream without tiles here answers too: the segment's table has been
                // read, and its queries' phase was not missed.
                if (t0 >= n) mbar_arrive(m->o_full + s);
                kp.go(n, kstages);
                vp.go(n, vstages);
                kp.at = vp.at = 0;
            }
            // nothing of this thread's is in flight when the block ends
            tc05::mma_commit(m->fin + s);
            tc05::mbar_wait(m->fin + s, 0, kPoll);
        }
        __syncwarp();
    }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int s = warp >> 2, tid = threadIdx.x & 127, wq = warp & 3;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + kOcol;
        const uint32_t tw = tmem + lanes + kPcol + s * kPstep;  // weights
        uint32_t sp = 0, op = 0, tp = 0, vp = 0;
        Cursor c;
        c.start(a, sh);
        // this thread's 16-byte pieces of a segment's queries, loaded a segment ahead
        constexpr int kChunks = D / 8, kPass = 128 / kChunks;  // rows a pass of this warpgroup
        constexpr int kLoads = (kTwo ? 128 : 64) / kPass;
        const int qch = tid % kChunks, qr0 = (kTwo ? 0 : s * 64) + tid / kChunks;
        uint4 qv[kLoads];
        auto load_queries = [&](const Cursor &k) {
            const int rbase = k.rb * a.rows + (kTwo ? s * 128 : 0), last = k.q.T * a.G - 1;
            const uint16_t *p =
                a.q + (long long)k.q.first * a.q_stride + (long long)k.h * a.G * D + qch * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int rr = min(rbase + qr0 + i * kPass, last), t = div_g(a, rr);
                qv[i] = __ldg(reinterpret_cast<const uint4 *>(p + t * a.q_stride + (rr - t * a.G) * D));
            }
        };
        constexpr bool kAhead = kLoads <= 8;  // (16 pieces would push other values to local memory)
        if (kAhead) load_queries(c);
        const float boost = kBf16 ? 0.f : 7.f;
        for (int left = units; left > 0;) {
            const Segment sg(c, left);
            const Seq q = c.q;
            const int len = q.ctx + q.T, nrows = q.T * a.G;
            const int32_t *trow = a.s.table + (long long)c.b * a.s.max_pages;
            const int ns = kTwo ? sg.n : (sg.n + 1 - s) / 2;  // this stream's tiles
            // ---- pages that do not exist, among this segment's
            bool bad = false;
            {
                const int p1 = (min(len, (sg.j0 + sg.n) * kKeys) + a.s.page - 1) >> a.s.lpage;
#pragma unroll 1
                for (int p = ((sg.j0 * kKeys) >> a.s.lpage) + (threadIdx.x & 255); p < p1; p += 256)
                    bad |= (unsigned)trow[p] >= (unsigned)a.pages;
            }
            // ---- queries to shared memory, rows in the products' order
            if (!kAhead) load_queries(c);
            {
                const int rbase = c.rb * a.rows + (kTwo ? s * 128 : 0);
                uint8_t *dst = qs + (kTwo ? s * kTile : 0) + (qch >> 3) * (kKeys * 128);
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int r = qr0 + i * kPass;
                    const uint32_t keep = rbase + r < nrows ? a.qand : 0u;
                    *reinterpret_cast<uint4 *>(dst + r * 128 + (((qch & 7) ^ (r & 7)) << 4)) =
                        make_uint4((qv[i].x ^ a.qxor) & keep, (qv[i].y ^ a.qxor) & keep,
                                   (qv[i].z ^ a.qxor) & keep, (qv[i].w ^ a.qxor) & keep);
                }
            }
            tc05::fence_proxy_async();
            if (threadIdx.x == 0) m->tiles = sg.n;
            mbar_arrive(&m->q_full);
            if (threadIdx.x < 8) m->nf[threadIdx.x] = 0;
            __syncwarp();
            bad = pair_or(bad);

            const int rbase = c.rb * a.rows + (kTwo ? s * 128 : 0);
            const int rr = rbase + tid;
            const bool row_live = rr < nrows, warp_live = rbase + wq * 32 < nrows;
            const int t = row_live ? div_g(a, rr) : 0;
            float mx = -INFINITY, l = 0.f;  // mx: the maximum in use (log2 units)
            uint64_t acc[kSplit ? D / 2 : 1];  // for an fp32 output: O, two columns each
            if (kSplit)
#pragma unroll
                for (int e = 0; e < D / 2; ++e) acc[e] = 0;
#pragma unroll 1
            for (int i = 0; i < ns; ++i) {
                const int tile = kTwo ? i : 2 * i + s, j = sg.j0 + tile;
                const bool special = bad || (j + 1) * kKeys > q.ctx;
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // this tile's keys that the row sees
                if (special && warp_live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        see[k] = row_live ? seen_word(a, q, t, j * kKeys + k * 32) : 0u;
                    if (bad) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int slot = j * kKeys + k * 16;
                            if (slot < len && (unsigned)trow[slot >> a.s.lpage] >= (unsigned)a.pages)
                                see[k >> 1] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                    }
                }
                wait(m->s_full + s, sp, m, a.status);
                __syncwarp();
                sp ^= 1;
                tc05::fence_after_sync();
                // The streams take turns: left alone they fall into step, both
                // at their exponentials and then both waiting for products.
                // (Stream 0 goes first; a pass of the other's is due before
                // each tile but its first.)
                if (i > 0 || s > 0) {
                    wait(m->turn + s, tp ^ (uint32_t)((s ? i : i - 1) & 1), m, a.status);
                    __syncwarp();
                }
                if (special && (!kTwo || s == 0)) {
                    // Values that some row must not see are kept out of the
                    // product where zero times them is not zero: a thread a
                    // key, zeros past the end and where there is no page, and
                    // a draft's infinities and NaNs noted and replaced.
                    // (In its turn, since then the slot's last tile has come.)
                    const int pos = units - left + tile, vst = kstages + pos % vstages;
                    if (wait(m->full + vst, (uint32_t)(pos / vstages) & 1u, m, a.status)) {
                        const int key = j * kKeys + tid;
                        uint8_t *row = ring + vst * kTile + tid * 128;
                        const bool none =
                            key >= len || (bad && (unsigned)trow[key >> a.s.lpage] >= (unsigned)a.pages);
                        if (none || key >= q.ctx) {
                            bool inf = false;
#pragma unroll 4
                            for (int ch = 0; ch < D / 8; ++ch) {
                                uint4 *w = reinterpret_cast<uint4 *>(
                                    row + (ch >> 3) * (kKeys * 128) + (((ch & 7) ^ (tid & 7)) << 4));
                                uint32_t x[4] = {0u, 0u, 0u, 0u};
                                if (!none) {
                                    const uint4 v = *w;
                                    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        if (nonfinite2<kBf16>(x[e] & 0xFFFFu)) { x[e] &= 0xFFFF0000u; inf = true; }
                                        if (nonfinite2<kBf16>(x[e] & 0xFFFF0000u)) { x[e] &= 0xFFFFu; inf = true; }
                                    }
                                }
                                *w = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                            if (inf) atomicOr(&m->nf[(key - q.ctx) >> 5], 1u << ((key - q.ctx) & 31));
                        }
                    }
                    tc05::fence_proxy_async();
                }
                __syncwarp();
                auto hand_over = [&]() {  // the scores are in registers: S is free, and the turn passes
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(m->turn + (s ^ 1));
                        mbar_arrive(m->s_free + s);
                    }
                };
                // P is free again, and O complete so far. Warps without rows wait
                // too: nothing else keeps their next arrival with weights behind
                // the others' last, and it would stand for a slow warp's.
                auto products_done = [&]() {
                    wait(m->pv_done + s, vp, m, a.status);
                    __syncwarp();
                    tc05::fence_after_sync();
                    vp ^= 1u;
                };
                if (warp_live) {
                    if (kSplit && special) {  // scores that a row must not see become -inf
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t x[32];
                            tc05::tmem_ld32(ts + k * 32, x);
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((see[k] >> e) & 1u)) x[e] = 0xFF800000u;
                            tc05::tmem_st32(ts + k * 32, x);
                        }
                        tc05::tmem_wait_st();
                    }
                    // two elements an instruction: weight = 2^(s * sl2 - base)
                    const uint64_t sl2 = pack_f32x2(a.sl2, a.sl2);
                    uint64_t sum[2] = {0, 0};
                    if constexpr (kSplit) {
                        // The scores twice from tensor memory, 32 at a time: O has the registers.
                        float tm = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t x[32];
                            tc05::tmem_ld32(ts + k * 32, x);
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) tm = fmaxf(tm, __uint_as_float(x[e]));
                        }
                        tm *= a.sl2;
                        const bool move = tm > mx + kLazy || (mx == -INFINITY && tm > mx);
                        if (__any_sync(0xFFFFFFFFu, move)) {
                            const float al = move ? ex2(mx - tm) : 1.f;
                            if (move) mx = tm;
                            l *= al;
                            const uint64_t al2 = pack_f32x2(al, al);
#pragma unroll
                            for (int e = 0; e < D / 2; ++e) acc[e] = fma_f32x2(acc[e], al2, 0);
                        }
                        const float base = mx == -INFINITY ? 0.f : mx - boost;
                        const uint64_t nb = pack_f32x2(-base, -base);
#pragma unroll 2
                        for (int h = 0; h < 8; ++h) {  // 16 at a time: one step of the product
                            // (not unrolled whole: fetching that much code took 16,000 cycles
                            // at a block's first tile)
                            uint32_t x[16], hi[8], lo[8], third[8];
                            tc05::tmem_ld16(ts + h * 16, x);
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float p0, p1;
                                unpack_f32x2(fma_f32x2(pack_u32x2(x[2 * e], x[2 * e + 1]), sl2, nb), p0, p1);
                                p0 = ex2(p0);
                                p1 = ex2(p1);
                                sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(p0, p1));
                                if (kThird) {  // cut, not rounded: 3 x 8 bits hold all 24
                                    hi[e] = cut_bf16x2(p0, p1);
                                    lo[e] = cut_bf16x2(p0, p1);
                                    third[e] = cut_bf16x2(p0, p1);
                                } else {
                                    hi[e] = pack2<kBf16>(p0, p1);
                                    const float2 f = unpack2<kBf16>(hi[e]);
                                    lo[e] = pack2<kBf16>(p0 - f.x, p1 - f.y);
                                }
                            }
                            tc05::tmem_st8(tw + h * 16, hi);
                            tc05::tmem_st8(tw + h * 16 + 8, lo);
                            if (kThird) tc05::tmem_st8(to + s * kOstep + 64 + h * 8, third);
                        }
                    } else {
                    uint32_t x[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc05::tmem_ld32(ts + k * 32, x[k]);
                    tc05::tmem_wait_ld();
                    if (kApart) hand_over();
                    if (special)  // scores that a row must not see become -inf
#pragma unroll
                        for (int e = 0; e < 128; ++e)
                            if (!((see[e >> 5] >> (e & 31)) & 1u)) x[e >> 5][e & 31] = 0xFF800000u;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(x[0][e]);
#pragma unroll
                    for (int e = 4; e < 128; ++e)
                        v[e & 3] = fmaxf(v[e & 3], __uint_as_float(x[e >> 5][e & 31]));
                    const float tm = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * a.sl2;
                    if (kApart && i > 0) products_done();
                    const bool move = tm > mx + kLazy || (mx == -INFINITY && tm > mx);
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float al = move ? ex2(mx - tm) : 1.f;
                        if (move) mx = tm;
                        l *= al;
                        if (i > 0) {
                            // all earlier products of this stream are done: they
                            // were issued before this tile's scores
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                uint32_t o[16];
                                tc05::tmem_ld16(to + s * kOstep + k * 16, o);
                                tc05::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                tc05::tmem_st16(to + s * kOstep + k * 16, o);
                            }
                        }
                    }
                    const float base = mx == -INFINITY ? 0.f : mx - boost;
                    const uint64_t nb = pack_f32x2(-base, -base);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t hi[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p0, p1;
                            unpack_f32x2(fma_f32x2(pack_u32x2(x[h][2 * e], x[h][2 * e + 1]), sl2, nb), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(p0, p1));
                            hi[e] = pack2<kBf16>(p0, p1);
                        }
                        tc05::tmem_st16(tw + h * 16, hi);
                    }
                    }
                    float s0, s1, s2, s3;
                    unpack_f32x2(sum[0], s0, s1);
                    unpack_f32x2(sum[1], s2, s3);
                    l += (s0 + s1) + (s2 + s3);
                }
                if (kApart) {
                    if (!warp_live) {
                        hand_over();
                        if (i > 0) products_done();
                    }
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m->turn + (s ^ 1));
                }
                tc05::tmem_wait_st();
                tc05::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(m->p_ready + s);
                if constexpr (kSplit) {  // this tile's share of O
#pragma unroll
                    for (int hf = 0; hf < D / kOcols; ++hf) {
                        products_done();
                        if (warp_live)
#pragma unroll
                            for (int k = 0; k < kOcols / 32; ++k) {
                                uint32_t o[32];
                                tc05::tmem_ld32(to + s * kOstep + k * 32, o);
                                tc05::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    uint64_t &x = acc[hf * 32 + k * 16 + e];
                                    x = add_f32x2(x, pack_u32x2(o[2 * e], o[2 * e + 1]));
                                }
                            }
                        if (hf + 1 < D / kOcols) {  // the other half may come
                            tc05::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(m->p_ready + s);
                        }
                    }
                }
            }
            if constexpr (kSplit) {  // O to where the segment's end takes it from
                if (ns > 0) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
#pragma unroll
                        for (int e = 0; e < 16; ++e) unpack_f32x2(acc[k * 16 + e], o[2 * e], o[2 * e + 1]);
                        tc05::tmem_st32(to + s * kOstep + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
                    }
                    tc05::tmem_wait_st();
                    tc05::fence_before_sync();
                }
            }
            // ---- the segment's end
            Cursor next = c;
            if (left > sg.n) {
                next.next_item(a);
                if (kAhead) load_queries(next);
            }
            wait(m->o_full + s, op, m, a.status);
            op ^= 1;
            if (kApart && ns > 0) vp ^= 1u;  // the last product's, which o_full covers
            __syncwarp();
            if (mx != -INFINITY) mx -= boost;
            m->ml[s][tid] = make_float2(mx, l);
            pair_sync();
            tc05::fence_after_sync();
            if (warp_live) {
                float M = mx, L = l, f0 = 1.f, f1 = 0.f;
                if (!kTwo) {
                    const float2 v0 = m->ml[0][tid], v1 = m->ml[1][tid];
                    M = fmaxf(v0.x, v1.x);
                    f0 = v0.x == -INFINITY ? 1.f : ex2(v0.x - M);
                    f1 = v1.x == -INFINITY ? 1.f : ex2(v1.x - M);
                    L = v0.y * f0 + v1.y * f1;
                }
                const bool has1 = !kTwo && sg.n > 1;
                const float inv = sg.whole ? 1.f / L : 1.f;
                const bool none = sg.whole && L == 0.f;  // no weight: zero, also where a value is infinite
                const long long row =
                    (long long)(q.first + t) * a.Hq + c.h * a.G + (row_live ? rr - t * a.G : 0);
                const int seg_last = left == units ? 0 : 1, prow = (kTwo ? s * 128 : 0) + tid;
                bool odd = false;  // drafts to add by hand
                for (int w = 0; w < 8; ++w) odd |= m->nf[w] != 0;
                const int k0 = kTwo ? 0 : s * (D / 64), k1 = kTwo ? D / 32 : k0 + D / 64;
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {  // 32 columns at a time
                    float o[32];
                    __syncwarp();
                    tc05::tmem_ld32(to + (kTwo ? s * kOstep : 0) + k * 32,
                                    *reinterpret_cast<uint32_t(*)[32]>(o));
                    tc05::tmem_wait_ld();
                    if (!kTwo) {
                        float o1[32];
                        if (has1) {
                            tc05::tmem_ld32(to + kOstep + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o1));
                            tc05::tmem_wait_ld();
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = has1 ? o[e] * f0 + o1[e] * f1 : o[e] * f0;
                    }
                    if (odd && row_live) {
#pragma unroll 1
                        for (int d = 0; d < q.T; ++d) {
                            if (!((m->nf[d >> 5] >> (d & 31)) & 1u) ||
                                !(seen_word(a, q, t, q.ctx + d) & 1u))
                                continue;
                            const int sl = q.ctx + d, pid = trow[sl >> a.s.lpage];
                            if ((unsigned)pid >= (unsigned)a.pages) continue;
                            const uint16_t *v =
                                a.vpool + (((long long)pid * a.Hkv + c.h) * a.s.page +
                                           (sl & (a.s.page - 1))) * D + k * 32;
                            for (int e = 0; e < 32; ++e) {
                                const float y = to_f32<kBf16>(v[e]);
                                if (!isfinite(y)) o[e] += y;
                            }
                        }
                    }
                    if (row_live) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                        if (!sg.whole) {
                            float *p = part_at<D>(a, blockIdx.x, seg_last, prow, k * 32);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<float4 *>(p + e * (a.rows * 4LL)) =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        } else if (a.o_f32) {
                            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.o) + row * D + k * 32);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                p[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        } else {
                            uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + row * D + k * 32);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                p[e] = make_uint4(pack2<kBf16>(o[8 * e], o[8 * e + 1]),
                                                  pack2<kBf16>(o[8 * e + 2], o[8 * e + 3]),
                                                  pack2<kBf16>(o[8 * e + 4], o[8 * e + 5]),
                                                  pack2<kBf16>(o[8 * e + 6], o[8 * e + 7]));
                        }
                    }
                }
                if (row_live && (kTwo || s == 0)) {
                    if (sg.whole)
                        a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
                    else
                        *reinterpret_cast<float2 *>(a.part_ml + (((long long)blockIdx.x * 2 + seg_last) * a.rows + prow) * 2) =
                            make_float2(M, L);
                }
            }
            tc05::fence_before_sync();
            __syncwarp();
            pair_sync();  // O, the queries and the tables may be overwritten
            // the other stream passed the turn once a tile of its own
            tp ^= (uint32_t)(kTwo ? sg.n : (sg.n + s) / 2) & 1u;
            left -= sg.n;
            c = next;
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    if (warp == 9) tc05::tmem_dealloc(tmem, 512);
}

template <int D, bool kBf16>
cudaError_t run_tc(const CUtensorMap &km, const CUtensorMap &vm, const TreeArgs &a, cudaStream_t st) {
    constexpr int kTile = kKeys * D * 2;
    const int q = (a.rows == 256 ? 2 : 1) * kTile;
    int stages = (kSmemMax - kMisc - q) / kTile;
    if (stages > kMaxStages) stages = kMaxStages;
    auto *k = a.rows == 256
                  ? (a.o_f32 ? k_attn_tc<D, kBf16, true, true> : k_attn_tc<D, kBf16, true, false>)
                  : (a.o_f32 ? k_attn_tc<D, kBf16, false, true> : k_attn_tc<D, kBf16, false, false>);
    cudaError_t e = set_smem(k, kSmemMax);
    if (e == cudaSuccess)
        e = launch(k, dim3(a.grid), dim3(kThreads), kSmemMax, st, true, km, vm, a, stages);
    return e;
}

}  // namespace

cudaError_t launch_tree_tc(const AttnCache &c, const TreeArgs &a, cudaStream_t st) {
    CUtensorMap km, vm;
    const int box = c.page < kKeys ? c.page : kKeys;
    if (!encode_pool(&km, c.k, c, box, false) || !encode_pool(&vm, c.v, c, box, false))
        return cudaErrorNotSupported;
    if (c.D == 64)
        return c.bf16 ? run_tc<64, true>(km, vm, a, st) : run_tc<64, false>(km, vm, a, st);
    return c.bf16 ? run_tc<128, true>(km, vm, a, st) : run_tc<128, false>(km, vm, a, st);
}

}  // namespace attn
}  // namespace qmv
