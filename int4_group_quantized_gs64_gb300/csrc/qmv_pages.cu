// qmv_pages.cu - the pages of a cache: who holds them, which are free, forks of
// sequences, and the moves of their tokens.
//
// refs[p] counts the table entries that hold page p; a page with none is free.
// There is no list of free pages: what a call needs is found in refs from page 0
// on, so the lowest free pages go out in the order of the entries that miss one
// (sequence by sequence), whatever the order in which thread blocks run. All of it
// is integer work on a few hundred KB at most: launches and dependent loads are
// what it costs, so a call is few kernels, each with many loads in flight.
#include "qmv_attn.cuh"
#include "qmv_attn.h"
#include "qmv_launch.cuh"

namespace qmv {
namespace attn {
namespace {

constexpr int kStNone = 8;  // no free page left

constexpr int kChunk = 512;   // table entries a block
constexpr int kSmall = 128;   // its threads: four warps of four 32-entry pieces
constexpr int kOne = 1024;    // threads of the one block that hands pages out

struct PagesArgs {
    int32_t *refs;
    int pages, lpage;  // page = 1 << lpage
    int32_t *table;
    int max_pages, B, chunks;
    const int32_t *lens, *more;
    int window, sinks;
    int32_t *status;
    // fork
    const int32_t *parent;
    int F;
    int32_t *new_table, *new_lens, *moves;
    // workspace: entries that miss a page in each chunk, how many do in the chunks
    // before, and the pages handed out, in order
    int32_t *miss, *before, *found, *list;
};

// A sequence's length and what it is to take; false: it does not fit its table.
__device__ __forceinline__ bool length_ok(const PagesArgs &a, int len, int more) {
    return len >= 0 && more >= 0 && (long long)len + more <= ((long long)a.max_pages << a.lpage);
}
// Page i of a sequence of len tokens that takes `more`: a coming token at slot p >= len
// sees the slots > p - window and those < sinks.
__device__ __forceinline__ bool needed(const PagesArgs &a, int i, int len, int more) {
    const long long s0 = (long long)i << a.lpage, s1 = s0 + (1 << a.lpage);
    return s0 < (long long)len + more && (s0 < a.sinks || s1 > (long long)len - a.window + 1);
}

// ------------------------------------------------------------------ update

// Entries that are not needed give their pages back; those that miss one are counted.
__global__ void __launch_bounds__(kSmall) k_pages_release(const PagesArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / a.chunks, c = blockIdx.x - b * a.chunks;
    int32_t *row = a.table + (long long)b * a.max_pages;
    const int i0 = c * kChunk + threadIdx.x;
    int id[kChunk / kSmall];
#pragma unroll
    for (int k = 0; k < kChunk / kSmall; ++k)
        id[k] = i0 + k * kSmall < a.max_pages ? row[i0 + k * kSmall] : -1;
    const int len = a.lens[b], more = a.more[b];
    const bool ok = length_ok(a, len, more);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kChunk / kSmall; ++k) {
        const int i = i0 + k * kSmall;
        if (i >= a.max_pages) continue;
        if (id[k] >= a.pages) {
            set_status(a.status, kStPage);
        } else if (ok) {
            const bool need = needed(a, i, len, more);
            n += need && id[k] < 0;
            if (!need && id[k] >= 0) {
                if (atomicSub(a.refs + id[k], 1) <= 0) {  // nobody held it
                    atomicAdd(a.refs + id[k], 1);
                    set_status(a.status, kStPage);
                }
                row[i] = -1;
            }
        }
    }
    if (!ok && threadIdx.x == 0) set_status(a.status, kStLength);
    __shared__ int sums[kSmall / 32];
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) a.miss[blockIdx.x] = sums[0] + sums[1] + sums[2] + sums[3];
}

// Inclusive sums over the block's threads (kOne of them) and the total; sh: 32 ints.
__device__ __forceinline__ int block_scan(int v, int *sh, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();  // sh may still be read from the call before
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += x;
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const int base = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
    return v + (warp > 0 ? base : 0);
}

// before[i] = miss[0] + .. + miss[i - 1] for i <= n; returns the sum of all.
__device__ __forceinline__ int scan_misses(const PagesArgs &a, int n, int *sh) {
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += kOne) {
        const int i = i0 + threadIdx.x, v = i < n ? a.miss[i] : 0;
        int total;
        const int inc = block_scan(v, sh, total);
        if (i < n) a.before[i] = carry + inc - v;
        carry += total;
    }
    return carry;
}

// The `want` lowest free pages, or as many as there are, to the list, each held
// once from here on; returns how many. A warp looks at 256 pages a pass, and loads
// the next pass's meanwhile: what bounds it is the latency of a pass. (An update of
// 1,024 sequences that takes 34,345 pages, the last of them number 94,590 of 650,492,
// looks at 12 passes: GPU time with the two copies around it 42 us in passes of 128
// pages a warp without loading ahead, 30 so. By themselves and from cold the three
// kernels take 7, 20 and 7 us.)
__device__ __forceinline__ int take_free(const PagesArgs &a, int want, int *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = 8, kPass = kOne * kPer;
    const int p0 = warp * (32 * kPer) + lane;
    int next[kPer];
    auto load = [&](int pass) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int p = pass + p0 + k * 32;
            next[k] = p < a.pages ? a.refs[p] : 1;
        }
    };
    if (want > 0) load(0);
    int got = 0;
    for (int pass = 0; pass < a.pages && got < want; pass += kPass) {
        uint32_t free[kPer];
        int n = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            free[k] = __ballot_sync(0xFFFFFFFFu, next[k] == 0);
            n += __popc(free[k]);
        }
        load(pass + kPass);
        int total;
        int at = got + block_scan(lane == 31 ? n : 0, sh, total);
        at = __shfl_sync(0xFFFFFFFFu, at, 31) - n;  // free pages before this warp's
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int rank = at + __popc(free[k] & ((1u << lane) - 1u));
            if (((free[k] >> lane) & 1u) && rank < want) {
                a.list[rank] = pass + p0 + k * 32;
                a.refs[pass + p0 + k * 32] = 1;
            }
            at += __popc(free[k]);
        }
        got += total;
    }
    return min(got, want);
}

__global__ void __launch_bounds__(kOne) k_pages_find(const PagesArgs a) {
    __shared__ int sh[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int want = scan_misses(a, a.B * a.chunks, sh);
    const int got = take_free(a, want, sh);
    if (threadIdx.x == 0) {
        *a.found = got;
        if (got < want) set_status(a.status, kStNone);
    }
}

// The entries of this block's chunk that miss a page get theirs.
__global__ void __launch_bounds__(kSmall) k_pages_give(const PagesArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.miss[blockIdx.x] == 0) return;
    const int b = blockIdx.x / a.chunks, c = blockIdx.x - b * a.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *row = a.table + (long long)b * a.max_pages;
    constexpr int kPer = kChunk / kSmall;
    const int i0 = c * kChunk + warp * (32 * kPer) + lane;
    const int len = a.lens[b], more = a.more[b], got = *a.found;
    uint32_t miss[kPer];
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = i0 + k * 32;
        miss[k] = __ballot_sync(0xFFFFFFFFu, i < a.max_pages && row[i] < 0 && needed(a, i, len, more));
        n += __popc(miss[k]);
    }
    __shared__ int sums[kSmall / 32];
    if (lane == 0) sums[warp] = n;
    __syncthreads();
    int at = a.before[blockIdx.x];
    for (int w = 0; w < warp; ++w) at += sums[w];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int rank = at + __popc(miss[k] & ((1u << lane) - 1u));
        if (((miss[k] >> lane) & 1u) && rank < got) row[i0 + k * 32] = a.list[rank];
        at += __popc(miss[k]);
    }
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(kSmall) k_pages_share(const PagesArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int f = blockIdx.x / a.chunks, c = blockIdx.x - f * a.chunks;
    const int p = a.parent[f];
    const int len = (unsigned)p < (unsigned)a.B ? a.lens[p] : -1;
    const bool ok = length_ok(a, len, 0);
    const int32_t *from = a.table + (long long)p * a.max_pages;
    int32_t *to = a.new_table + (long long)f * a.max_pages;
    const int whole = ok ? len >> a.lpage : 0, rows = ok ? len & ((1 << a.lpage) - 1) : 0;
#pragma unroll
    for (int k = 0; k < kChunk / kSmall; ++k) {
        const int i = c * kChunk + threadIdx.x + k * kSmall;
        if (i >= a.max_pages) continue;
        int id = -1;
        if (i < whole) {
            id = from[i];
            if (id >= a.pages) set_status(a.status, kStPage);
            if ((unsigned)id < (unsigned)a.pages)
                atomicAdd(a.refs + id, 1);
            else
                id = -1;
        }
        to[i] = id;
    }
    if (c == 0 && threadIdx.x == 0) {
        int id = -1;
        if (rows) {
            id = from[whole];
            if ((unsigned)id >= (unsigned)a.pages) {
                id = -1;
                set_status(a.status, kStPage);
            }
        }
        // (without it the child ends with its whole pages: a hole there would be filled
        // by the next update, with a page that its tokens were never written to)
        a.miss[f] = id >= 0;
        a.moves[f * 3LL] = id;
        a.moves[f * 3LL + 1] = -1;
        a.moves[f * 3LL + 2] = id >= 0 ? rows : 0;
        a.new_lens[f] = ok ? (id >= 0 ? len : whole << a.lpage) : 0;
        if (!ok) set_status(a.status, kStLength);
    }
}

__global__ void __launch_bounds__(kOne) k_pages_fork(const PagesArgs a) {
    __shared__ int sh[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int want = scan_misses(a, a.F, sh);
    const int got = take_free(a, want, sh);
    if (threadIdx.x == 0 && got < want) set_status(a.status, kStNone);
    __syncthreads();  // the list
    for (int f = threadIdx.x; f < a.F; f += kOne) {
        if (!a.miss[f]) continue;
        const int rank = a.before[f], len = a.new_lens[f];
        if (rank < got) {
            const int id = a.list[rank];
            a.new_table[(long long)f * a.max_pages + (len >> a.lpage)] = id;
            a.moves[f * 3LL + 1] = id;
        } else {  // as long as its whole pages
            a.new_lens[f] = len >> a.lpage << a.lpage;
            a.moves[f * 3LL] = -1;
            a.moves[f * 3LL + 2] = 0;
        }
    }
}

// ------------------------------------------------------------------ copy

struct CopyArgs {
    const uint16_t *sk, *sv;
    uint16_t *dk, *dv;
    int spages, dpages, Hkv, page, D;
    const int32_t *moves;
    const float *sacc;
    float *dacc;
    int32_t *status;
};

// A block a move and head: the first rows of a page, one stretch of each pool.
// What bounds it is the copy.
__global__ void __launch_bounds__(256) k_pages_copy(const CopyArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int m = blockIdx.x / a.Hkv, h = blockIdx.x - m * a.Hkv;
    const int32_t *mv = a.moves + m * 3LL;
    const int from = mv[0], to = mv[1], rows = mv[2];
    if (from < 0 || to < 0 || rows == 0) return;
    if (from >= a.spages || to >= a.dpages || rows < 0 || rows > a.page) {
        if (h == 0 && threadIdx.x == 0)
            set_status(a.status, rows < 0 || rows > a.page ? kStLength : kStPage);
        return;
    }
    const long long s = ((long long)from * a.Hkv + h) * a.page, d = ((long long)to * a.Hkv + h) * a.page;
    const bool v = blockIdx.y;
    const uint4 *src = reinterpret_cast<const uint4 *>((v ? a.sv : a.sk) + s * a.D);
    uint4 *dst = reinterpret_cast<uint4 *>((v ? a.dv : a.dk) + d * a.D);
    const int n = rows * a.D / 8;
    for (int i = threadIdx.x; i < n; i += 256 * 4) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * 256 < n) x[k] = src[i + k * 256];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * 256 < n) dst[i + k * 256] = x[k];
    }
    if (a.dacc && !v)
        for (int i = threadIdx.x; i < rows; i += 256) a.dacc[d + i] = a.sacc ? a.sacc[s + i] : 0.f;
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
    Seqs s;
    uint16_t *k, *v;
    int pages, Hkv, D;
    const int32_t *keep, *kept;
    float *acc;
    int32_t *new_ctx, *status;
};

// A block a sequence and head. Rows go to lower slots in ascending order: a pass
// reads its rows, and when all are read writes them; what it overwrites are rows of
// this pass or of passes before, since keep[i] >= i. What bounds it is the chain of
// loads: lengths, kept tokens, page, row.
__global__ void __launch_bounds__(128) k_compact(const CompactArgs a) {
    constexpr int kAhead = 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / a.Hkv, h = blockIdx.x - b * a.Hkv;
    bool ok;
    const int n = a.kept[b];
    const Seq q = get_seq(a.s, b, ok);
    ok = ok && n >= 0 && n <= q.T;
    const int32_t *keep = a.keep + q.first;
    bool bad = false;
    if (ok)
        for (int i = threadIdx.x; i < n; i += 128) {
            const int x = keep[i];
            bad |= x < i || x >= q.T || (i > 0 && x <= keep[i - 1]);
        }
    ok = !__syncthreads_or(bad || !ok);
    if (h == 0 && threadIdx.x == 0) {
        a.new_ctx[b] = ok ? q.ctx + n : a.s.ctx[b];
        if (!ok) set_status(a.status, kStLength);
    }
    if (!ok || n == 0 || keep[n - 1] == n - 1) return;  // (all in their places)
    const int32_t *row = a.s.table + (long long)b * a.s.max_pages;
    // offset of slot x's row in a pool of one element a token, -1: no page
    auto place = [&](int x) -> long long {
        const int slot = q.ctx + x, pid = row[slot >> a.s.lpage];
        if ((unsigned)pid >= (unsigned)a.pages) {
            set_status(a.status, kStPage);
            return -1;
        }
        return ((long long)pid * a.Hkv + h) * a.s.page + (slot & (a.s.page - 1));
    };
    const int lanes = a.D / 8, per = 128 / lanes;  // threads a row, rows at a time
    const int l = threadIdx.x % lanes, r = threadIdx.x / lanes;
    for (int i0 = 0; i0 < n; i0 += per * kAhead) {
        uint4 x[kAhead], y[kAhead];
        float w[kAhead];
        long long to[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * per + r;
            to[j] = -1;
            if (i >= n || keep[i] == i) continue;
            const long long from = place(keep[i]);
            to[j] = place(i);
            if (from < 0) to[j] = -1;
            if (to[j] < 0) continue;
            x[j] = *reinterpret_cast<const uint4 *>(a.k + from * a.D + l * 8);
            y[j] = *reinterpret_cast<const uint4 *>(a.v + from * a.D + l * 8);
            if (a.acc && l == 0) w[j] = a.acc[from];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (to[j] < 0) continue;
            *reinterpret_cast<uint4 *>(a.k + to[j] * a.D + l * 8) = x[j];
            *reinterpret_cast<uint4 *>(a.v + to[j] * a.D + l * 8) = y[j];
            if (a.acc && l == 0) a.acc[to[j]] = w[j];
        }
        __syncthreads();
    }
}

int log2_of(int page) {
    int l = 0;
    while ((1 << l) < page) ++l;
    return l;
}

// The workspace's parts: n counts, n sums before, how many were found, the list.
size_t carve(PagesArgs &a, long long n, long long most, void *ws) {
    a.miss = static_cast<int32_t *>(ws);
    a.before = a.miss + n;
    a.found = a.before + n;
    a.list = a.found + 1;
    return (size_t)(2 * n + 1 + (most < a.pages ? most : a.pages)) * 4;
}

}  // namespace
}  // namespace attn

size_t pages_update_ws_bytes(int pages, int B, int max_pages) {
    attn::PagesArgs a;
    a.pages = pages;
    const int chunks = (max_pages + attn::kChunk - 1) / attn::kChunk;
    return (attn::carve(a, (long long)B * chunks, (long long)B * max_pages, nullptr) + 255) / 256 * 256;
}

size_t pages_fork_ws_bytes(int pages, int F) {
    attn::PagesArgs a;
    a.pages = pages;
    return (attn::carve(a, F, F, nullptr) + 255) / 256 * 256;
}

cudaError_t launch_pages_update(int32_t *refs, int pages, int page, int32_t *table, int max_pages,
                                const int32_t *lens, const int32_t *more, int B, int window, int sinks,
                                int32_t *status, void *ws, cudaStream_t st) {
    using namespace attn;
    PagesArgs a = {};
    a.refs = refs; a.pages = pages; a.lpage = log2_of(page);
    a.table = table; a.max_pages = max_pages; a.B = B;
    a.chunks = (max_pages + kChunk - 1) / kChunk;
    a.lens = lens; a.more = more; a.window = window; a.sinks = sinks; a.status = status;
    carve(a, (long long)B * a.chunks, (long long)B * max_pages, ws);
    const dim3 grid((unsigned)(B * a.chunks));
    cudaError_t e = launch(k_pages_release, grid, dim3(kSmall), 0, st, true, a);
    if (e == cudaSuccess) e = launch(k_pages_find, dim3(1), dim3(kOne), 0, st, true, a);
    if (e == cudaSuccess) e = launch(k_pages_give, grid, dim3(kSmall), 0, st, true, a);
    return e;
}

cudaError_t launch_pages_fork(int32_t *refs, int pages, int page, const int32_t *table, int max_pages,
                              const int32_t *lens, int B, const int32_t *parent, int F,
                              int32_t *new_table, int32_t *new_lens, int32_t *moves, int32_t *status,
                              void *ws, cudaStream_t st) {
    using namespace attn;
    PagesArgs a = {};
    a.refs = refs; a.pages = pages; a.lpage = log2_of(page);
    a.table = const_cast<int32_t *>(table); a.max_pages = max_pages; a.B = B;
    a.chunks = (max_pages + kChunk - 1) / kChunk;
    a.lens = lens; a.parent = parent; a.F = F;
    a.new_table = new_table; a.new_lens = new_lens; a.moves = moves; a.status = status;
    carve(a, F, F, ws);
    cudaError_t e = launch(k_pages_share, dim3((unsigned)(F * a.chunks)), dim3(kSmall), 0, st, true, a);
    if (e == cudaSuccess) e = launch(k_pages_fork, dim3(1), dim3(kOne), 0, st, true, a);
    return e;
}

cudaError_t launch_pages_copy(const AttnCache &src, const AttnCache &dst, const int32_t *moves, int n,
                              const float *src_acc, float *dst_acc, int32_t *status, cudaStream_t st) {
    using namespace attn;
    const CopyArgs a{static_cast<const uint16_t *>(src.k), static_cast<const uint16_t *>(src.v),
                     static_cast<uint16_t *>(dst.k), static_cast<uint16_t *>(dst.v), src.pages,
                     dst.pages, src.Hkv, src.page, src.D, moves, src_acc, dst_acc, status};
    return launch(k_pages_copy, dim3((unsigned)(n * src.Hkv), 2), dim3(256), 0, st, true, a);
}

cudaError_t launch_attn_compact(const AttnCache &c, const AttnSeqs &s, const int32_t *keep,
                                const int32_t *kept, float *acc, int32_t *new_ctx, int32_t *status,
                                cudaStream_t st) {
    using namespace attn;
    CompactArgs a;
    a.s = Seqs{s.table, s.ctx, s.cu, s.B, s.N, 0, s.max_pages, c.page, log2_of(c.page), 0};
    a.k = static_cast<uint16_t *>(c.k);
    a.v = static_cast<uint16_t *>(c.v);
    a.pages = c.pages; a.Hkv = c.Hkv; a.D = c.D;
    a.keep = keep; a.kept = kept; a.acc = acc; a.new_ctx = new_ctx; a.status = status;
    return launch(k_compact, dim3((unsigned)(s.B * c.Hkv)), dim3(128), 0, st, true, a);
}

}  // namespace qmv
