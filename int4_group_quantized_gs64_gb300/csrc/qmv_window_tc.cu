// qmv_window_tc.cu - windowed attention of many rows on the tcgen05 tensor cores.
//
// S = Q K^T from shared memory, O += P V with P in tensor memory, 128 rows a tile
// (whole tokens with their query heads: qmv_attn_plan.cuh), 128 keys a step. A
// block keeps two streams in flight, each with its own scores S and output O:
//   prompts (kTwo): two tiles of rows against the same keys, which are copied once;
//   up to 128 rows a head: one tile; the streams take alternate steps of the keys
//   and are added up at the end of the block's part of an item.
//
// Warps: 0-3 and 4-7 the streams' softmax, a thread a row; 8 copies keys, 11 values
// and queries, 9 and 10 issue the streams' products (9 all of them where the streams
// take alternate steps). Every warp comes to a barrier's phases one by one.
//
// A stream's chain of a step is 1,024 cycles of products (at 128 elements) and its
// softmax; the two streams together need 2,048 of products and, side by side, some
// 1,400 of softmax (exponentials 512 a stream, and as much again for scaling, sums,
// packing and the maximum). For fp32 outputs the softmax is what bounds a step, some
// 3,500 cycles with two or three numbers a weight, and of these more are waits than
// issue (41% of the issue slots taken, loads from tensor memory the top stall: two
// softmax warps a scheduler do not cover each other's). What shortens the chain: the next
// scores are issued right behind the output's products, in turns that hold nothing but
// the issue; products of two or three numbers a weight begin when half of the keys have
// theirs; a step's weights come from the maximum that its rows have, so that no
// exponential waits for the step's own (below); what is looked at or written for the
// edges is kept out of the loop that every step runs through.
//
// The end of an item costs a stream one look at O: queries of the next item come by
// tensor-map copies while the last softmax runs, and its scores are formed while O
// is written out. The streams do not wait for one another there.
//
// Measured (GPU time, from captured graphs; 482 and 101 us through the Python calls):
// 10,746 prompt tokens of 48 heads (8 key/value heads of 128), windows of
// 2048, 16-bit outputs: 467 us, 1,139 TFLOP/s (the kernel of qmv_attn_tc.cu, with
// windows: 678). Of that the steps at the edges cost some 27 us, the look at values
// 24, writing O 28. 16 chunks of up to 301 tokens of 40 heads (8 of 64 elements),
// windows of 513 and 17 first tokens, fp16 to fp32: 99 us, 234 TFLOP/s (with the
// kernel of qmv_attn_tc.cu 178 us).
//
// Masks: a step that all rows of the item see whole is not looked at. In the others
// (at the window's edge, the diagonal, the first tokens' end, with a missing page)
// scores that a row does not see become -inf, and values that some row does not see
// and that are not finite are replaced by zeros, since 0 x inf is not 0; the rows
// that do see them get them added at the end (Misc::odd).
//
// The maximum in use moves when it is found to have grown by more than 2^8; weights
// and sums for 16-bit and fp32 outputs are those of qmv_attn_tc.cu. For 16-bit outputs a
// weight is rounded once, to half a step of itself, as the operand of its product: a
// second number would be half as many products again (1,024 cycles more a step of 2,840),
// and the output is rounded to the same type anyway (prompts against 64 bits: 2.3e-3 of
// the norm, the output's rounding alone 1.7e-3). For fp32 outputs two fp16 or three bf16
// numbers, and sums of each step added up in registers: 5e-7.
#include <cudaTypedefs.h>
#include <string.h>

#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_attn_plan.cuh"
#include "qmv_attn_tc05.cuh"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

constexpr int kThreads = 384, kKeys = 128, kMaxSlots = 6;  // slots a ring
constexpr int kMisc = 2896;               // barriers and small tables
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 units the maximum may lag

struct Misc {
    ShareScratch<kThreads / 32> share;
    uint64_t kfull[kMaxSlots], kempty[kMaxSlots], vfull[kMaxSlots], vempty[kMaxSlots];
    uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2], o_full[2];
    uint64_t p_half[2];  // kSplit: the weights of the step's first 64 keys are there
    uint64_t vready[kMaxSlots];  // values have been looked at
    uint64_t turn[2], fin[2];
    uint32_t kflag[kMaxSlots];  // of the step whose keys lie there: 1 first of its segment, 2 last
    uint32_t tmem, dead;
    uint32_t odd;          // some value that not all rows saw was not finite
    float2 ml[2][128];     // !kTwo: the streams' maxima and sums
};
static_assert(sizeof(Misc) <= kMisc, "");

// Waits for a barrier's phase; gives up after a bounded time, or at once when
// another warp has given up.
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

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                          int c3, uint64_t *mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(tc05::smem_addr(mbar))
        : "memory");
}

// 32 bytes (a whole sector) where `wide`, which wants p on a 32-byte boundary; else 16 twice.
__device__ __forceinline__ void store32(void *p, bool wide, const uint32_t (&x)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
                     "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        uint4 *q = static_cast<uint4 *>(p);
        q[0] = make_uint4(x[0], x[1], x[2], x[3]);
        q[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// The upper halves of two floats, which are bf16 numbers, and what they leave.
__device__ __forceinline__ uint32_t cut_bf16x2(float &x, float &y) {
    const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
    x -= __uint_as_float(u & 0xFFFF0000u);
    y -= __uint_as_float(v & 0xFFFF0000u);
    return __byte_perm(u, v, 0x7632);
}

// A block's part of an item: steps [j0, j0 + n) of the item's keys.
struct Segment {
    int j0, n;
    bool whole;
    __device__ __forceinline__ Segment(const CursorOf<true> &c, int left) {
        j0 = c.u;
        n = min(c.nu - c.u, left);
        whole = j0 == 0 && n == c.nu;
    }
};

template <int D, bool kBf16, bool kTwo, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ CUtensorMap qmap, const TreeArgs a, int stages) {
    constexpr int kTile = kKeys * D * 2, kHalves = D / 64, kQ = kTwo ? 2 : 1;
    constexpr uint32_t kIdescS = tc05::idesc_f16kind_f32(kBf16, 128, kKeys, false);
    extern __shared__ __align__(1024) uint8_t smem[];
    // Tensor memory columns. Where they suffice (64 elements, one 16-bit number a
    // weight) P lies apart from S, and a stream's next S is formed while its
    // exponentials run. Otherwise P overwrites S.
    constexpr bool kApart = D == 64 && !kSplit;
    // The third number of a bf16 weight lies in columns that O leaves: with 128
    // elements O comes in two halves, one after the other.
    constexpr bool kThird = kSplit && kBf16, kParted = kThird && D == 128;
    constexpr int kOcols = kParted ? 64 : D;  // columns a product gives
    constexpr uint32_t kIdescO = tc05::idesc_f16kind_f32(kBf16, 128, kOcols, true);
    // The two streams' products are issued in turn where they are what bounds a step:
    // side by side both streams' scores would come at once, and the pipe would wait
    // for both softmaxes.
    constexpr bool kTurns = kTwo && !kSplit && !kApart;
    constexpr int kPcol = kApart ? 256 : 0, kPstep = kApart ? 64 : 128;   // P of stream s at kPcol + s * kPstep
    constexpr int kOcol = kApart ? 384 : 256, kOstep = kApart ? 64 : 128;
    const int kslots = stages / 2, vslots = stages - kslots;
    uint8_t *qs = smem, *kring = smem + kQ * kTile, *vring = kring + kslots * kTile;
    Misc *m = reinterpret_cast<Misc *>(vring + vslots * kTile);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            tc05::mbar_init(m->kfull + i, 1);
            tc05::mbar_init(m->kempty + i, kQ);
            tc05::mbar_init(m->vfull + i, 1);
            tc05::mbar_init(m->vempty + i, kQ);
            tc05::mbar_init(m->vready + i, 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc05::mbar_init(m->q_full + s, 1);
            tc05::mbar_init(m->q_empty + s, 1);
            tc05::mbar_init(m->s_full + s, 1);
            tc05::mbar_init(m->s_free + s, 4);
            tc05::mbar_init(m->p_full + s, 4);
            tc05::mbar_init(m->p_half + s, 4);
            tc05::mbar_init(m->pv_done + s, 1);
            tc05::mbar_init(m->o_full + s, 1);
            tc05::mbar_init(m->turn + s, 1);
            tc05::mbar_init(m->fin + s, 1);
        }
        m->dead = 0;
        m->odd = 0;
        tc05::fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        prefetch_tmap(&qmap);
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
    const Share sh = find_share<kThreads, true>(a, &m->share);
    if (threadIdx.x == 0) a.info[blockIdx.x * 2].n = a.info[blockIdx.x * 2 + 1].n = 0;
    if (too_long(a, sh) || sh.u0 >= sh.u1) return;
    if (warp == 9) tc05::tmem_alloc(&m->tmem, 512);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, m->tmem, 0);
    const int units = (int)(sh.u1 - sh.u0);  // (the launcher keeps this below 2^31)

    // 168 x 384 registers at launch = 216 x 256 + 72 x 128 = 208 x 256 + 88 x 128. With 64
    // elements the softmax has some to spare, and the warps that copy and issue keep
    // theirs out of memory (16 chunks to fp32 105 -> 101 us; with 128 elements long
    // contexts to fp32 go from 2,190 to 2,270, prompts differ by less than a percent).
    constexpr int kSoftRegs = D == 64 ? 208 : 216, kIssueRegs = D == 64 ? 88 : 72;
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 8 || warp == 11) {
        // ------------------------------------------------------------ copies
        const bool keys = warp == 8;
        const CUtensorMap *map = keys ? &kmap : &vmap;
        // read once: first to leave L2 (not by several items)
        const bool once = a.max_rows <= a.tb * a.hb * kQ;
        const uint64_t policy = evict_first_policy();
        const int prow = a.s.page < kKeys ? a.s.page : kKeys;  // rows a copy
        CursorOf<true> c;
        c.start(a, sh);
        uint64_t *full = keys ? m->kfull : m->vfull, *empty = keys ? m->kempty : m->vempty;
        const uint32_t ring = tc05::smem_addr(keys ? kring : vring);
        const int slots = keys ? kslots : vslots;
        int stage = 0;
        uint32_t phase = 1, qphase = 1;  // a fresh barrier counts as passed for parity 1
        // this lane's piece of the item's step u at c: its page
        auto page_of = [&](int u, bool &lv) {
            const int slot = c.slot(u * kKeys + lane * prow);
            lv = lane * prow < kKeys && c.some(a, slot, slot + prow);
            return lv ? __ldg(a.s.table + (long long)c.b * a.s.max_pages + (slot >> a.s.lpage)) : 0;
        };
        // Values that some row must not see are kept out of the product where zero times
        // them is not zero: a step behind its copies the values' warp looks at them, in the
        // steps that not all rows see whole; keys that no row of the item sees, or without
        // a page, get zeros, and of those that some rows see infinities and NaNs are
        // replaced (the rows that see them get them added when O is written).
        struct {
            int at, stage;         // its first place; the slot of the ring
            uint32_t gone, phase;  // pieces without a page
            Reach r;
        } was;
        was.stage = -1;
        auto look = [&]() {
            if (was.stage < 0) return;
            const Reach &r = was.r;
            if (wait(m->vfull + was.stage, was.phase, m, a.status) &&
                (was.gone || !r.all_at(a, was.at, kKeys))) {
                __syncwarp();
#pragma unroll 1
                for (int x = lane; x < kKeys; x += 32) {
                    const int key = r.slot(was.at + x);
                    uint8_t *row = vring + was.stage * kTile + x * 128;
                    auto at_chunk = [&](int ch) {
                        return reinterpret_cast<uint4 *>(row + (ch >> 3) * (kKeys * 128) +
                                                         (((ch & 7) ^ (x & 7)) << 4));
                    };
                    if (!r.some(a, key, key + 1) || ((was.gone >> (x / prow)) & 1u)) {
#pragma unroll
                        for (int ch = 0; ch < D / 8; ++ch) *at_chunk(ch) = make_uint4(0u, 0u, 0u, 0u);
                    } else if (!r.all(a, key, key + 1)) {
                        uint32_t top = 0;  // the largest magnitudes of even and odd elements
#pragma unroll
                        for (int ch = 0; ch < D / 8; ++ch) {
                            const uint4 v = *at_chunk(ch);
                            top = __vimax3_u16x2(top, v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
                            top = __vimax3_u16x2(top, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
                        }
                        if (nonfinite2<kBf16>(top)) {
                            atomicOr(&m->odd, 1u);
#pragma unroll 1
                            for (int ch = 0; ch < D / 8; ++ch) {
                                uint4 v = *at_chunk(ch);
                                uint32_t *y = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if (nonfinite2<kBf16>(y[e] & 0xFFFFu)) y[e] &= 0xFFFF0000u;
                                    if (nonfinite2<kBf16>(y[e] & 0xFFFF0000u)) y[e] &= 0xFFFFu;
                                }
                                *at_chunk(ch) = v;
                            }
                        }
                    }
                }
                tc05::fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(m->vready + was.stage);
        };
        bool live;
        int pid = page_of(c.u, live);
        bool ok = true;
        uint32_t pending = 0, pending_ph = 0;  // slots this warp copied to, and the phase that ends it
        uint32_t q_pending = 0, q_phase = 0;  // streams whose queries were copied last, and the phase that ends it
        for (int left = units; left > 0;) {
            const Segment sg(c, left);
            if (!keys) {  // the item's queries, once the last item's scores are done
                if (ok) {
                    q_pending = 0;
                    q_phase = qphase ^ 1u;
                }
#pragma unroll
                for (int s = 0; s < kQ; ++s) {
                    ok = ok && wait(m->q_empty + s, qphase, m, a.status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (ok && lane == 0) {
                        const int x = c.rb * a.tpi + s, k = x / a.hs;
                        const int head = c.h * a.G + (x - k * a.hs) * a.hb;
                        mbar_expect_tx(m->q_full + s, kHalves * 128 * a.hb * a.tb);
#pragma unroll
                        for (int hf = 0; hf < kHalves; ++hf)
                            tma_load4(tc05::smem_addr(qs) + s * kTile + hf * (128 * 128), &qmap, 0, head,
                                      c.q.first + k * a.tb, hf, m->q_full + s);
                    }
                    if (ok) q_pending |= 1u << s;
                }
                qphase ^= 1u;
            }
#pragma unroll 1
            for (int t = 0; t < sg.n; ++t) {
                const bool good = live && (unsigned)pid < (unsigned)a.pages;
                const int row =
                    (pid * a.Hkv + c.h) * a.s.page + (c.slot((sg.j0 + t) * kKeys + lane * prow) & (a.s.page - 1));
                if (live && !good && keys) set_status(a.status, kStPage);
                const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, good));
                const uint32_t gone = __ballot_sync(0xFFFFFFFFu, live && !good);
                if (t + 1 < sg.n) pid = page_of(sg.j0 + t + 1, live);
                ok = ok && wait(empty + stage, phase, m, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) continue;
                if (lane == 0) {
                    if (keys) m->kflag[stage] = (t == 0 ? 1u : 0u) | (t == sg.n - 1 ? 2u : 0u);
                    if (n)
                        mbar_expect_tx(full + stage, n * prow * D * 2);
                    else
                        mbar_arrive(full + stage);
                }
                __syncwarp();
                if (good) {
                    const uint32_t dst = ring + stage * kTile + lane * prow * 128;
#pragma unroll
                    for (int hf = 0; hf < kHalves; ++hf)
                        if (once)
                            tma_load3_once(dst + hf * (kKeys * 128), map, 0, row, hf, full + stage, policy);
                        else
                            tma_load3(dst + hf * (kKeys * 128), map, 0, row, hf, full + stage);
                }
                if (!keys) {
                    look();
                    was.at = (sg.j0 + t) * kKeys;
                    was.r = c.r;
                    was.stage = stage;
                    was.gone = gone;
                    was.phase = phase ^ 1u;
                }
                pending |= 1u << stage;
                pending_ph = (pending_ph & ~(1u << stage)) | ((phase ^ 1u) & 1u) << stage;
                if (++stage == slots) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            left -= sg.n;
            if (left > 0) {
                c.next_item(a);
                pid = page_of(c.u, live);
            }
        }
        if (!keys) look();
        if (!ok) {  // gave up: wait (bounded) for this warp's copies in flight
            for (int i = 0; i < slots; ++i)
                if ((pending >> i) & 1u) tc05::mbar_wait(full + i, (pending_ph >> i) & 1u, kPoll / 64);
            for (int s = 0; s < kQ; ++s)
                if ((q_pending >> s) & 1u) tc05::mbar_wait(m->q_full + s, q_phase, kPoll / 64);
        }
    } else if (kTwo || warp == 9) {
        // ------------------------------------------------------------ products
        // kTwo: a warp a stream. The warp walks its steps as a whole and one elected lane
        // issues: operands that the compiler sees to be uniform go to a product in some 10
        // cycles, where a lone thread's took 48 of the 64 that the product runs for.
        {
            const int me = warp - 9;  // kTwo: the stream
            const uint64_t kdesc = tc05::sdesc_sw128(tc05::smem_addr(kring));
            const uint64_t vdesc = tc05::sdesc_sw128_mn(tc05::smem_addr(vring), kKeys * 128);
            const uint64_t qdesc = tc05::sdesc_sw128(tc05::smem_addr(qs)) + (uint32_t)(me * (kTile >> 4));
            // the next scores' step: whether its keys have been waited for, its flags, and
            // its place in its segment
            bool seen = false;
            uint32_t flag = 0;
            int place = 0;
            // the outputs' steps lag at most two behind: bits 2 x and 2 x + 1 say of the
            // x-th whether its stream's O begins anew and whether the segment ends
            uint32_t ahead_bits = 0;
            int ahead_n = 0, kslot = 0, vslot = 0;
            uint32_t kph = 0, vph = 0, qph = 0, tph = 0;
            uint32_t fph = 0, hph = 0, frph = 0;  // bit s: p_full, p_half, s_free of stream s
            bool live = true;
            auto await = [&](uint64_t *bar, uint32_t parity) {
                live = __all_sync(0xFFFFFFFFu, live && wait(bar, parity, m, a.status));
            };
            // The scores of a step: what they wait for, the products, and what they tell.
            auto peek = [&]() {
                if (seen) return;
                await(m->kfull + kslot, kph);
                flag = *(volatile uint32_t *)(m->kflag + kslot);
                seen = true;
                place = flag & 1u ? 0 : place + 1;
            };
            auto scores_wait = [&](int s, bool again) {  // again: not the stream's first
                peek();
                if (flag & 1u) {
                    await(m->q_full + me, qph);
                    qph ^= 1u;
                }
                if (kApart && again) {
                    await(m->s_free + s, (frph >> s) & 1u);
                    frph ^= 1u << s;
                }
            };
            auto scores_issue = [&](int s) {  // S = Q K^T
                const uint64_t kd = kdesc + (uint32_t)(kslot * (kTile >> 4));
                if (elected()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int of = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                        tc05::mma_ss(tmem + s * 128, qdesc + of, kd + of, kIdescS, k > 0);
                    }
                    tc05::mma_commit(m->s_full + s);
                }
                __syncwarp();
            };
            auto scores_done = [&]() {
                if (elected()) {
                    tc05::mma_commit(m->kempty + kslot);
                    if (flag & 2u) tc05::mma_commit(m->q_empty + me);
                }
                __syncwarp();
                ahead_bits |= ((place < (kTwo ? 1 : 2) ? 1u : 0u) | (flag & 2u)) << (2 * ahead_n++);
                seen = false;
                if (++kslot == kslots) {
                    kslot = 0;
                    kph ^= 1u;
                }
            };
            auto scores = [&](int s, bool again) {
                scores_wait(s, again);
                if (!live) return;
                tc05::fence_after_sync();
                scores_issue(s);
                scores_done();
            };
            // The output of the oldest step: O (+)= P V.
            auto weights_wait = [&](int s) {
                await(m->p_full + s, (fph >> s) & 1u);
                fph ^= 1u << s;
            };
            auto output_wait = [&](int s) {
                await(m->vready + vslot, vph);
                if (kSplit) {
                    await(m->p_half + s, (hph >> s) & 1u);
                    hph ^= 1u << s;
                } else {
                    weights_wait(s);
                }
            };
            // kSplit: k0 .. k1 - 1 of the eight sixteenths of the keys; hf: kParted, which
            // half of the columns.
            auto output_issue = [&](int s, int hf, int k0, int k1) {
                const uint32_t tp = tmem + kPcol + s * kPstep, to = tmem + kOcol + s * kOstep;
                const uint64_t v = vdesc + (uint32_t)(vslot * (kTile >> 4));
                if (elected()) {
                    if constexpr (kSplit) {  // the rests, then the weights: a sum of this step alone
#pragma unroll
                        for (int part = kThird ? 2 : 1; part >= 0; --part)
#pragma unroll
                            for (int k = k0; k < k1; ++k)
                                tc05::mma_ts(to, part == 2 ? to + 64 + k * 8 : tp + k * 16 + part * 8,
                                             v + (hf * (kKeys * 128) + k * 2048 >> 4), kIdescO,
                                             part < (kThird ? 2 : 1) || k > 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            tc05::mma_ts(to, tp + k * 8, v + k * (2048 >> 4), kIdescO, k ? 1u : ~ahead_bits & 1u);
                    }
                    if (kSplit ? k1 == kKeys / 16 : kApart) tc05::mma_commit(m->pv_done + s);
                }
                __syncwarp();
            };
            auto output_rest = [&](int s) {
                if (!kParted) return;
                weights_wait(s);  // (the first half has been taken)
                if (!live) return;
                tc05::fence_after_sync();
                output_issue(s, 1, 0, kKeys / 16);
            };
            auto output_done = [&](int s) {
                if (elected()) {
                    tc05::mma_commit(m->vempty + vslot);
                    if (ahead_bits & 2u) {
                        tc05::mma_commit(m->o_full + s);
                        if (!kTwo) tc05::mma_commit(m->o_full + (s ^ 1));
                    }
                }
                __syncwarp();
                if (++vslot == vslots) {
                    vslot = 0;
                    vph ^= 1u;
                }
                ahead_bits >>= 2;
                --ahead_n;
            };
            auto output = [&](int s) {
                output_wait(s);
                if (!live) return;
                tc05::fence_after_sync();
                if (kSplit) {  // as the weights come
                    output_issue(s, 0, 0, kKeys / 32);
                    weights_wait(s);
                    if (!live) return;
                    tc05::fence_after_sync();
                    output_issue(s, 0, kKeys / 32, kKeys / 16);
                } else {
                    output_issue(s, 0, 0, kKeys / 16);
                }
                output_rest(s);
                if (live) output_done(s);
            };
            auto pass = [&]() {
                if (elected()) mbar_arrive(m->turn + (me ^ 1));
                __syncwarp();
            };
            if constexpr (kTurns) {
                // Stream 0's step n, stream 1's, stream 0's next: each the output of the
                // step and the scores of the one after, with the waits before the turn and
                // what can be told later after it (600 cycles of it in the turn, and the
                // two threads' turns added up to 4,600 cycles a step).
                scores(me, false);
#pragma unroll 1
                for (int n = 0; n < units && live; ++n) {
                    // (the next item's queries may be on their way: then the turn passes first)
                    const bool more = n + 1 < units;
                    if (more) peek();
                    const bool held = more && (flag & 1u), now = more && !held;
                    if (now) scores_wait(me, true);
                    output_wait(me);
                    if (me || n) {
                        await(m->turn + me, tph);
                        tph ^= 1u;
                    }
                    if (!live) break;
                    tc05::fence_after_sync();
                    output_issue(me, 0, 0, kKeys / 16);
                    if (now) scores_issue(me);
                    pass();
                    output_done(me);
                    if (now) scores_done();
                    if (held) scores(me, true);
                }
            } else if constexpr (kTwo) {
                scores(me, false);
#pragma unroll 1
                for (int n = 0; n < units && live; ++n) {
                    const bool more = n + 1 < units;
                    if (kApart && more) scores(me, true);
                    output(me);
                    if (!kApart && more) scores(me, true);
                }
            } else {
                // step n is stream n % 2's; at most two steps' scores ahead
                int qn = 0;
                auto ahead = [&](int upto) {
                    while (qn < units && qn < upto && live) {
                        scores(qn & 1, qn >= 2);
                        ++qn;
                    }
                };
                auto starts = [&]() {  // whether the next step begins a segment
                    peek();
                    return (flag & 1u) != 0;
                };
                ahead(1);
                if (units > 1 && !starts()) ahead(2);
#pragma unroll 1
                for (int n = 0; n < units && live; ++n) {
                    // S of step n + 2, and before it those that an item's start held
                    // back: they wait for its queries, so the outputs before go first
                    if (kApart && qn == n + 2 && qn < units && !starts()) ahead(n + 3);
                    ahead(n + 1);
                    output(n & 1);
                    ahead(n + 2);
                    if (qn < units && !starts()) ahead(n + 3);
                }
            }
            // nothing of this warp's is in flight when the block ends
            if (elected()) tc05::mma_commit(m->fin + me);
            __syncwarp();
            tc05::mbar_wait(m->fin + me, 0, kPoll);
        }
        __syncwarp();
    }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int s = warp >> 2, tid = threadIdx.x & 127, wq = warp & 3;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + kOcol;
        const uint32_t tw = tmem + lanes + kPcol + s * kPstep;  // weights
        uint32_t sp = 0, op = 0, vp = 0;  // phases of s_full, o_full, pv_done
        bool again = false;               // a step of this stream came before
        CursorOf<true> c, next;
        c.start(a, sh);
        const float boost = kBf16 ? 0.f : 7.f;
        constexpr float kMost = kBf16 ? 1048576.f : 32768.f;
        const int piece = min(a.s.page, kKeys);
        // The page of this lane's piece of step i of a segment (it is loaded a step ahead, and
        // over the end of a segment).
        auto page_of = [&](const CursorOf<true> &x, const Segment &g, int i) {
            const int slot = x.slot((g.j0 + i) * kKeys + lane * piece);
            const bool need = lane * piece < kKeys && i < g.n && x.some(a, slot, slot + piece);
            return need ? __ldg(a.s.table + (long long)x.b * a.s.max_pages + (slot >> a.s.lpage)) : 0;
        };
        int pid = page_of(c, Segment(c, units), kTwo ? 0 : s);
        for (int left = units; left > 0;) {
            const Segment sg(c, left);
            const Seq q = c.q;
            const int32_t *trow = a.s.table + (long long)c.b * a.s.max_pages;
            // this stream's steps: i0, i0 + kStep, ...
            constexpr int kStep = kTwo ? 1 : 2;
            const int i0 = kTwo ? 0 : (s ^ (units - left)) & 1;
            int t, g;
            const bool row_live = tile_row(a, q, c.rb * a.tpi + (kTwo ? s : 0), tid, t, g);
            const bool warp_live = __any_sync(0xFFFFFFFFu, row_live);
            const int pos = q.ctx + t;  // the row's slot
            float mx = -INFINITY, l = 0.f;  // mx: the maximum in use (log2 units)
            uint64_t acc[kSplit ? D / 2 : 1];  // for an fp32 output: O, two columns each
            if (kSplit)
#pragma unroll
                for (int e = 0; e < D / 2; ++e) acc[e] = 0;
            // P is free again, and O complete so far. Warps without rows wait
            // too: nothing else keeps their next arrival with weights behind
            // the others' last, and it would stand for a slow warp's.
            auto products_done = [&]() {
                wait(m->pv_done + s, vp, m, a.status);
                __syncwarp();
                tc05::fence_after_sync();
                vp ^= 1u;
            };
            auto scores_free = [&]() {  // S may be overwritten
                tc05::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(m->s_free + s);
            };
            auto give = [&](uint64_t *bar) {  // weights are in tensor memory
                tc05::tmem_wait_st();
                tc05::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + s);
            };
#pragma unroll 1
            for (int i = i0; i < sg.n; i += kStep) {
                const int at = (sg.j0 + i) * kKeys;
                const uint32_t gone = __ballot_sync(0xFFFFFFFFu, (unsigned)pid >= (unsigned)a.pages);
                pid = page_of(c, sg, i + kStep);
                const bool special = gone || !c.r.all_at(a, at, kKeys);
                uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};  // this step's keys that the row sees
                if (special && warp_live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        see[k] = row_live ? c.r.word(a, pos, at + k * 32) : 0u;
                    if (gone) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if ((gone >> (k * 16 / piece)) & 1u)
                                see[k >> 1] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
                }
                wait(m->s_full + s, sp, m, a.status);
                __syncwarp();
                sp ^= 1;
                tc05::fence_after_sync();
                if (warp_live) {
                    // two elements an instruction: weight = 2^(s * sl2 - base)
                    const uint64_t sl2 = pack_f32x2(a.sl2, a.sl2);
                    uint64_t sum[2] = {0, 0};
                    if (special || a.flip != 1.f) {
                        // Scores that a row must not see become -inf, and those of a negative
                        // scale turn, in tensor memory, 32 at a time: nothing to do where all
                        // rows of the warp see all, no look at them where none sees any.
                        // (As selects among the registers' 128 scores the code that every step
                        // jumps over cost all steps.)
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t w = k < 2 ? (k ? see[1] : see[0]) : (k == 2 ? see[2] : see[3]);
                            uint32_t x[32];
                            if (__any_sync(0xFFFFFFFFu, w != 0u)) {
                                if (__all_sync(0xFFFFFFFFu, w == ~0u) && a.flip == 1.f) continue;
                                tc05::tmem_ld32(ts + k * 32, x);
                                tc05::tmem_wait_ld();
                                if (a.flip != 1.f)
#pragma unroll
                                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * a.flip);
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = w & (1u << e) ? x[e] : 0xFF800000u;
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = 0xFF800000u;
                            }
                            tc05::tmem_st32(ts + k * 32, x);
                        }
                        tc05::tmem_wait_st();
                    }
                    if constexpr (kSplit) {
                        // The scores twice from tensor memory, 32 at a time: O has the registers.
                        constexpr int kUnroll = D == 64 ? 1 : 2;
                        float tm = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t x[32];
                            tc05::tmem_ld32(ts + k * 32, x);
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                tm = max3(tm, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
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
#pragma unroll kUnroll
                        for (int h = 0; h < 8; ++h) {  // 16 at a time: one step of the product
                            if (h == 4) give(m->p_half);
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
                        // P over S: weights from the maximum that the row has, which need not
                        // be this step's. Only if they get too large for fp16, or for sums of
                        // them (kMost), is the maximum looked for and the step begun again;
                        // nothing has left the registers by then. (Maxima of every step: 553
                        // us where this took 521.) P apart: the maximum first, since S is
                        // wanted free soon.
                        uint32_t hi[4][16];
                        bool look = kApart || __any_sync(0xFFFFFFFFu, row_live && mx == -INFINITY);
#pragma unroll 1
                        for (;;) {
                            uint32_t x[4][32];
#pragma unroll
                            for (int k = 0; k < 4; ++k) tc05::tmem_ld32(ts + k * 32, x[k]);
                            tc05::tmem_wait_ld();
                            if (kApart) scores_free();
                            if (look) {
                                float v[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(x[0][e]);
#pragma unroll
                                for (int e = 4; e < 128; ++e)
                                    v[e & 3] = fmaxf(v[e & 3], __uint_as_float(x[e >> 5][e & 31]));
                                const float tm = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * a.sl2;
                                if (kApart && again) products_done();
                                const bool move = tm > mx + kLazy || (mx == -INFINITY && tm > mx);
                                if (__any_sync(0xFFFFFFFFu, move)) {
                                    const float al = move ? ex2(mx - tm) : 1.f;
                                    if (move) mx = tm;
                                    l *= al;
                                    if (i > i0) {
                                        // all earlier products of this stream are done: they
                                        // were issued before this step's scores
#pragma unroll 1
                                        for (int k = 0; k < D / 32; ++k) {
                                            uint32_t o[32];
                                            tc05::tmem_ld32(to + s * kOstep + k * 32, o);
                                            tc05::tmem_wait_ld();
#pragma unroll
                                            for (int e = 0; e < 32; ++e)
                                                o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                            tc05::tmem_st32(to + s * kOstep + k * 32, o);
                                        }
                                    }
                                }
                            }
                            const float base = mx == -INFINITY ? 0.f : mx - boost;
                            const uint64_t nb = pack_f32x2(-base, -base);
                            sum[0] = sum[1] = 0;
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float p0, p1;
                                    unpack_f32x2(fma_f32x2(pack_u32x2(x[h][2 * e], x[h][2 * e + 1]), sl2, nb), p0, p1);
                                    p0 = ex2(p0);
                                    p1 = ex2(p1);
                                    sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(p0, p1));
                                    hi[h][e] = pack2<kBf16>(p0, p1);
                                }
                                if (kApart) tc05::tmem_st16(tw + h * 16, hi[h]);
                            }
                            if (kApart) break;
                            float s0, s1, s2, s3;
                            unpack_f32x2(sum[0], s0, s1);
                            unpack_f32x2(sum[1], s2, s3);
                            const bool large = row_live && !((s0 + s1) + (s2 + s3) <= kMost);
                            if (look || !__any_sync(0xFFFFFFFFu, large)) break;
                            look = true;
                        }
                        if (!kApart)
#pragma unroll
                            for (int h = 0; h < 4; ++h) tc05::tmem_st16(tw + h * 16, hi[h]);
                        give(m->p_full);
                    }
                    float s0, s1, s2, s3;
                    unpack_f32x2(sum[0], s0, s1);
                    unpack_f32x2(sum[1], s2, s3);
                    l += (s0 + s1) + (s2 + s3);
                } else if (!kSplit) {  // a warp without rows: the arrivals alone
                    if (kApart) {
                        scores_free();
                        if (again) products_done();
                    }
                    give(m->p_full);
                }
                if (kSplit && !warp_live) give(m->p_half);
                if constexpr (kSplit) {  // this step's share of O
#pragma unroll
                    for (int hf = 0; hf < D / kOcols; ++hf) {
                        give(m->p_full);
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
                    }
                }
                again = true;
            }
            // ---- the segment's end
            const bool mine = i0 < sg.n;  // this stream had steps
            if (kSplit && mine) {  // O to where the segment's end takes it from
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 16; ++e) unpack_f32x2(acc[k * 16 + e], o[2 * e], o[2 * e + 1]);
                    tc05::tmem_st32(to + s * kOstep + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
                }
                tc05::tmem_wait_st();
            }
            next = c;
            if (left > sg.n) {
                next.next_item(a);
                pid = page_of(next, Segment(next, left - sg.n), kTwo ? 0 : (s ^ (units - left + sg.n)) & 1);
            }
            wait(m->o_full + s, op, m, a.status);
            op ^= 1;
            __syncwarp();
            tc05::fence_after_sync();
            if (mx != -INFINITY) mx -= boost;
            float M = mx, L = l, f0 = 1.f, f1 = 0.f;
            bool has0 = true, has1 = false;
            // the two warps that have the same rows
            auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + wq) : "memory"); };
            if (!kTwo) {
                m->ml[s][tid] = make_float2(mx, l);
                tc05::fence_before_sync();
                pair_sync();
                tc05::fence_after_sync();
                const float2 v0 = m->ml[0][tid], v1 = m->ml[1][tid];
                M = fmaxf(v0.x, v1.x);
                f0 = v0.x == -INFINITY ? 1.f : ex2(v0.x - M);
                f1 = v1.x == -INFINITY ? 1.f : ex2(v1.x - M);
                L = v0.y * f0 + v1.y * f1;
                const int e0 = (units - left) & 1;  // the stream of the segment's first step
                has0 = sg.n > 1 || e0 == 0;
                has1 = sg.n > 1 || e0 == 1;
            }
            if (!sg.whole && threadIdx.x == 0)
                a.info[blockIdx.x * 2 + (left == units ? 0 : 1)] =
                    PartInfo{c.b, c.h, c.rb, sg.j0, sg.n, c.nu, (int)sh.quota, 0};
            if (warp_live) {
                const float inv = sg.whole ? 1.f / L : 1.f;
                const bool none = sg.whole && L == 0.f;  // no weight: zero, also where a value is infinite
                const long long row = (long long)(q.first + t) * a.Hq + c.h * a.G + g;
                const int seg_last = left == units ? 0 : 1, prow = (kTwo ? s * 128 : 0) + tid;
                const bool wide = reinterpret_cast<uintptr_t>(a.o) % 32 == 0;
                const bool odd = *(volatile uint32_t *)&m->odd != 0;  // values to add by hand
                const int k0 = kTwo ? 0 : s * (D / 64), k1 = kTwo ? D / 32 : k0 + D / 64;
                auto columns = [&](int k, float (&o)[32]) {  // columns 32 k .. 32 k + 31 of O, out
                    if (odd && row_live) {
#pragma unroll 1
                        for (int d = 0; d < 512; ++d) {  // (Reach: at most 255 keys an edge)
                            const int key = d < 256 ? c.r.p0 + d : c.r.lo + d - 256;
                            const int u = c.r.place(key) / kKeys;
                            if (key > c.r.p1 || u < sg.j0 || u >= sg.j0 + sg.n || c.r.all(a, key, key + 1) ||
                                (d >= 256 && key > c.r.p0) || !(window_word(a, pos, key) & 1u))
                                continue;
                            const int pg = trow[key >> a.s.lpage];
                            if ((unsigned)pg >= (unsigned)a.pages) continue;
                            const uint16_t *v =
                                a.vpool + (((long long)pg * a.Hkv + c.h) * a.s.page +
                                           (key & (a.s.page - 1))) * D + k * 32;
                            for (int e = 0; e < 32; ++e) {
                                const float y = to_f32<kBf16>(v[e]);
                                if (!isfinite(y)) o[e] += y;
                            }
                        }
                    }
                    if (!row_live) return;
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                    if (!sg.whole) {
                        float *p = part_at<D>(a, blockIdx.x, seg_last, prow, k * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(p + e * (a.rows * 4LL)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else if (kSplit) {  // (an fp32 output)
                        float *p = static_cast<float *>(a.o) + row * D + k * 32;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) x[z] = __float_as_uint(o[8 * e + z]);
                            store32(p + 8 * e, wide, x);
                        }
                    } else {
                        uint16_t *p = static_cast<uint16_t *>(a.o) + row * D + k * 32;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t x[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) x[z] = pack2<kBf16>(o[16 * e + 2 * z], o[16 * e + 2 * z + 1]);
                            store32(p + 16 * e, wide, x);
                        }
                    }
                };
#pragma unroll 1
                    for (int k = k0; k < k1; ++k) {
                        float o[32];
                        __syncwarp();
                        if (kTwo) {
                            tc05::tmem_ld32(to + s * kOstep + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
                            tc05::tmem_wait_ld();
                        } else {
                            float o1[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = o1[e] = 0.f;
                            if (has0) tc05::tmem_ld32(to + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
                            if (has1) tc05::tmem_ld32(to + kOstep + k * 32, *reinterpret_cast<uint32_t(*)[32]>(o1));
                            tc05::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
                        }
                        columns(k, o);
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
            if (!kTwo) pair_sync();  // O and the maxima may be overwritten
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
cudaError_t run_tc(const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm, const TreeArgs &a,
                   cudaStream_t st) {
    constexpr int kTile = kKeys * D * 2;
    const bool two = a.tpi == 2;
    int stages = (kSmemMax - kMisc - (two ? 2 : 1) * kTile) / kTile;
    if (stages > 2 * kMaxSlots) stages = 2 * kMaxSlots;
    auto *k = two ? (a.o_f32 ? k_window_tc<D, kBf16, true, true> : k_window_tc<D, kBf16, true, false>)
                  : (a.o_f32 ? k_window_tc<D, kBf16, false, true> : k_window_tc<D, kBf16, false, false>);
    cudaError_t e = set_smem(k, kSmemMax);
    if (e == cudaSuccess)
        e = launch(k, dim3(a.grid), dim3(kThreads), kSmemMax, st, true, km, vm, qm, a, stages);
    return e;
}

}  // namespace

cudaError_t launch_window_tc(const AttnCache &c, const TreeArgs &a, cudaStream_t st) {
    CUtensorMap km, vm, qm;
    const int box = c.page < kKeys ? c.page : kKeys;
    if (!encode_pool(&km, c.k, c, box, false) || !encode_pool(&vm, c.v, c, box, false) ||
        !encode_heads(&qm, a.q, a.s.N, a.Hq, c.D, a.q_stride, a.hb, a.tb))
        return cudaErrorNotSupported;
    if (c.D == 64)
        return c.bf16 ? run_tc<64, true>(km, vm, qm, a, st) : run_tc<64, false>(km, vm, qm, a, st);
    return c.bf16 ? run_tc<128, true>(km, vm, qm, a, st) : run_tc<128, false>(km, vm, qm, a, st);
}

}  // namespace attn
}  // namespace qmv
