// pages.cu -- the pages of a paged cache: copying, forking, reserving, freeing
// and compacting them on the device.
//
// A pool is a set of caches (K and V codes, scales, ... of every layer) that
// share one page numbering, a block table [B, max_blocks] whose negative
// entries hold no page, the rows' context lengths, and a reference count per
// page (0 or less = free). Page numbers are handed out lowest first and in the
// order of the request lists, so a call's result is a function of its inputs.
//
// The data moves are bound by HBM (each byte read and written once); the
// bookkeeping is a few passes over the counts and tables, latency alone. fork
// and compact run a one-CTA plan that decides every move (the decisions are
// ordered: ranks among the free pages), then one kernel that carries the moves
// out over all SMs. The plan starts the second kernel early by programmatic
// dependent launch, so that only its wait remains between them. A grid can so
// be there while the kernel before it writes the lists, tables and counts that
// it takes: they are read by plain loads or from L2 after the wait, never by
// the read-only path (no `const ... __restrict__` here), which asks for data
// that nothing writes as long as the grid is there.
// Measured over the 160 caches of a 40-layer 4-bit pool (5.57 MB a page), each
// launch by itself with cold caches: 96 copies 164 us (6.5 TB/s read and
// written, 0.98 of the copy rate); 64 forks of 16 parents, half a page each, 45
// us (their 214 MB take 32 at the copy rate) between a plan of 9 and a reserve
// of 10; 57 for the three in a row.
#include <algorithm>

#include "kernels.cuh"

namespace a8w8 {

namespace {

constexpr int kCopyThreads = 256;
constexpr unsigned kUnitBytes = 16384;   // a copy unit: 4 vectors of 16 bytes per thread
// CTAs per SM: 4 for whole pages (copy of 1.07 GB 170 us as a replayed graph,
// 181 at 6 or 8; compaction 278, 290, 294); 8, all that fit, for forks, whose
// partial pages leave some of a CTA's items empty (fork of 64 children and
// reserve 57.7 us, 58.3 at 6, 65.9 at 4). Units of 8 KB: 198 and 69.8 us; of
// 32 KB: 172 and 58.9.
constexpr int kCopyCtasPerSm = 4, kForkCtasPerSm = 8;
constexpr int kPlanThreads = 1024;
constexpr unsigned kErrBlock = 0x2u, kErrCtx = 0x4u, kErrRow = 0x40u, kErrPages = 0x80u,
                   kErrAlias = 0x100u;

// Copies n bytes (a multiple of 4) with the CTA's threads: 16-byte vectors,
// four per thread in flight, where both addresses allow it, and 4-byte words
// for the rest.
__device__ __forceinline__ void copy_unit(unsigned char* dst, const unsigned char* src,
                                          unsigned n) {
    unsigned done = 0;
    if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src)) & 15) == 0) {
        const unsigned nv = n / 16;
        const int4* s = reinterpret_cast<const int4*>(src);
        int4* d = reinterpret_cast<int4*>(dst);
        for (unsigned i = threadIdx.x; i < nv; i += 4 * kCopyThreads) {
            int4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kCopyThreads < nv) v[k] = __ldcs(s + i + k * kCopyThreads);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kCopyThreads < nv) __stcs(d + i + k * kCopyThreads, v[k]);
        }
        done = nv * 16;
    }
    for (unsigned i = done / 4 + threadIdx.x; i < n / 4; i += kCopyThreads)
        reinterpret_cast<unsigned*>(dst)[i] = __ldcs(reinterpret_cast<const unsigned*>(src) + i);
}

// The cache that unit u of a page belongs to (units of one page are numbered
// through all caches).
__device__ __forceinline__ int unit_cache(const CacheList& c, unsigned u) {
    int lo = 0, hi = c.num_caches - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c.first_unit[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Copies unit u of page `from` to page `to`.
__device__ __forceinline__ void copy_page_unit(const CacheList& c, unsigned u, int from, int to) {
    const int k = unit_cache(c, u);
    const unsigned pb = c.page_bytes[k], off = (u - c.first_unit[k]) * kUnitBytes;
    copy_unit(c.base[k] + (size_t)to * pb + off, c.base[k] + (size_t)from * pb + off,
              min(kUnitBytes, pb - off));
}

// Exclusive prefix sum of v over the CTA's kPlanThreads threads; the total in
// `total`. `s` is 32 ints of shared memory. All threads call it.
__device__ __forceinline__ int block_exclusive(int v, int* s, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = s[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s[lane] = w;
    }
    __syncthreads();
    const int before = warp ? s[warp - 1] : 0;
    total = s[31];
    __syncthreads();   // s may be written again
    return before + x - v;
}

// Which of pages [4 i, 4 i + 4) are free, as four bits (pages at or past n are
// not).
__device__ __forceinline__ unsigned free_mask(const int32_t* refcount, int i, int n) {
    unsigned f = 0;
    if (4 * i + 3 < n) {
        const int4 r = ld_cg_v4(refcount + 4 * (size_t)i);
        f = (r.x <= 0) | (r.y <= 0) << 1 | (r.z <= 0) << 2 | (r.w <= 0) << 3;
    } else {
        for (int k = 0; k < 4; ++k)
            if (4 * i + k < n && __ldcg(refcount + 4 * (size_t)i + k) <= 0) f |= 1u << k;
    }
    return f;
}

// put(rank, page) for the lowest `want` free pages, rank counted from 0;
// returns how many there are (at most `want`). All threads call it, with the
// mask of their first four pages (quad threadIdx.x), loaded well before.
__device__ __forceinline__ int quads_of(int n) { return n / 4 + (n % 4 != 0); }
__device__ __forceinline__ unsigned first_mask(const int32_t* refcount, int n) {
    return (int)threadIdx.x < quads_of(n) ? free_mask(refcount, threadIdx.x, n) : 0u;
}
template <typename Put>
__device__ __forceinline__ int lowest_free(const int32_t* refcount, int n, unsigned mask, int want,
                                           int* s, Put put) {
    int found = 0;
    const int quads = quads_of(n);
    for (int q0 = 0; q0 < quads && found < want; q0 += kPlanThreads) {
        const int q = q0 + (int)threadIdx.x;
        const unsigned f = q0 == 0 ? mask : q < quads ? free_mask(refcount, q, n) : 0u;
        int total;
        int rank = found + block_exclusive(__popc(f), s, total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (f >> k & 1u) {
                if (rank < want) put(rank, 4 * q + k);
                ++rank;
            }
        found += total;
    }
    return min(found, want);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

constexpr int kPairBatch = 64;

// Each CTA takes a contiguous range of (pair, unit), so that it checks few
// pairs. A pair is carried out unless its destination is the destination of an
// earlier pair or the source of another one; a pair counts if both pages are
// in range and differ.
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const __grid_constant__ CacheList c, const int32_t* src, const int32_t* dst,
                      int n, unsigned* err) {
    __shared__ int sfrom[kPairBatch], sto[kPairBatch], sbad[kPairBatch];
    pdl_wait();
    pdl_trigger();
    const unsigned U = c.first_unit[c.num_caches];
    const long total = (long)n * U;
    const long share = total / gridDim.x, rest = total - share * gridDim.x;
    const long u0 = share * blockIdx.x + min((long)blockIdx.x, rest);
    const long u1 = u0 + share + (blockIdx.x < rest ? 1 : 0);
    if (u0 >= u1) return;
    const int p1 = (int)((u1 - 1) / U) + 1;
    for (int p0 = (int)(u0 / U); p0 < p1; p0 += kPairBatch) {
        const int np = min(kPairBatch, p1 - p0);
        if ((int)threadIdx.x < np) {
            const int f = src[p0 + threadIdx.x], t = dst[p0 + threadIdx.x];
            const bool ok = f >= 0 && t >= 0 && f < c.num_blocks && t < c.num_blocks;
            if (!ok && f >= 0 && t >= 0) set_error(err, kErrBlock);
            sfrom[threadIdx.x] = f;
            sto[threadIdx.x] = t;
            sbad[threadIdx.x] = !ok || f == t;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kCopyThreads) {
            const int f = src[j], t = dst[j];
            if (f < 0 || t < 0 || f >= c.num_blocks || t >= c.num_blocks || f == t) continue;
            for (int i = 0; i < np; ++i) {
                if (sbad[i] == 1) continue;
                if (f == sto[i] || (t == sto[i] && j < p0 + i)) sbad[i] = 2;
            }
        }
        __syncthreads();
        if ((int)threadIdx.x < np && sbad[threadIdx.x] == 2) set_error(err, kErrAlias);
        const long a = max(u0, (long)p0 * U), b = min(u1, (long)(p0 + np) * U);
        for (long u = a; u < b; ++u) {
            const int i = (int)(u / U) - p0;
            if (sbad[i]) continue;
            copy_page_unit(c, (unsigned)(u - (long)(p0 + i) * U), sfrom[i], sto[i]);
        }
        __syncthreads();   // the batch is read until here
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

struct __align__(16) ForkPlan {
    int src;        // the parent's page in part, -1: none
    int fresh;      // the page that takes its copy
    int full;       // shared pages, -1: the fork is not carried out
    int part;       // tokens of the page in part
};

// The plan's lists stand in the workspace, whatever their length. In shared
// memory (28 KB) each step is a round trip to L2 shorter, yet 64 forks with
// their reserve took 58.9 us instead of 56.9.
// The lowest entry of the list that names each row, for the rows named by
// valid entries. All threads call it.
template <typename Row>
__device__ __forceinline__ void first_entries(int* first, int B, int n, Row row) {
    for (int r = threadIdx.x; r < B; r += kPlanThreads) first[r] = 0x7fffffff;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int r = row(i);
        if (r >= 0) atomicMin(first + r, i);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const PageTables t, int num_blocks, const int32_t* parents,
                     const int32_t* children, int n, ForkPlan* plan, int* need, int* first,
                     unsigned* err) {
    __shared__ int s[32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned mask = first_mask(t.refcount, num_blocks);
    first_entries(first, t.B, n, [&](int i) {
        const int p = parents[i], c = children[i];
        return p >= 0 && p < t.B && c >= 0 && c < t.B ? c : -1;
    });
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int p = parents[i], c = children[i];
        ForkPlan f = {-1, -1, -1, 0};
        if (p >= 0 && c >= 0) {
            unsigned bad = 0u;
            int ctx = 0;
            if (p >= t.B || c >= t.B) {
                bad = kErrRow;
            } else {
                const int32_t* row = t.block_table + (size_t)p * t.max_blocks;
                ctx = __ldcg(t.ctx_lens + p);
                const int busy = __ldcg(t.ctx_lens + c);
                const int held = __ldcg(t.block_table + (size_t)c * t.max_blocks);
                int e = lane < t.max_blocks ? __ldcg(row + lane) : -1;   // before ctx is known
                if (first[c] != i || busy != 0 || held >= 0) bad |= kErrAlias;
                if (ctx < 0 || ctx > t.max_blocks * t.page) bad |= kErrCtx;
                if (!bad) {
                    f.full = ctx / t.page;
                    f.part = ctx % t.page;
                    const int used = f.full + (f.part > 0);
                    bool out = false;
                    int src = -1;
                    for (int j = lane; j < used; j += 32) {
                        if (j >= 32) e = __ldcg(row + j);
                        out |= e < 0 || e >= num_blocks;
                        if (j == f.full) src = e;
                    }
                    if (__any_sync(0xffffffffu, out)) bad |= kErrBlock;
                    f.src = __shfl_sync(0xffffffffu, src, f.full & 31);
                }
            }
            if (bad && lane == 0) set_error(err, bad);
            if (bad || ctx == 0) f = {-1, -1, -1, 0};
        }
        if (lane == 0) plan[i] = f;
    }
    __syncthreads();
    // ranks of the pages in part in list order, then the lowest free pages
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + (int)threadIdx.x;
        const bool w = i < n && plan[i].src >= 0;
        int total;
        const int rank = want + block_exclusive(w, s, total);
        if (w) need[rank] = i;
        want += total;
    }
    __syncthreads();
    const int found = lowest_free(t.refcount, num_blocks, mask, want, s,
                                  [&](int rank, int page) { plan[need[rank]].fresh = page; });
    __syncthreads();
    for (int k = found + (int)threadIdx.x; k < want; k += kPlanThreads) {
        plan[need[k]] = {-1, -1, -1, 0};
        if (k == found) set_error(err, kErrPages);
    }
}

// Items (cache, chunk of its page, fork) dealt out in turn, forks fastest:
// children of one parent read its page from L2 together, and forks that use
// little of their page leave no CTA idle. Every cache counts as many chunks as
// the largest page has (a power of two, 1 << shift): an empty item costs a few
// instructions, where finding the cache of a unit costs every thread a search
// through the list (159 warp instructions per unit: 64 forks of a 40-layer pool
// took 7 us longer). The tables and counts of fork i by CTA i mod grid.
__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(const __grid_constant__ CacheList c, const PageTables t,
                      const int32_t* parents, const int32_t* children, int n,
                      const ForkPlan* plan, int shift) {
    __shared__ unsigned char* s_base[kMaxCaches];
    __shared__ unsigned s_token[kMaxCaches];    // bytes of a token
    for (int k = threadIdx.x; k < c.num_caches; k += kCopyThreads) {
        s_base[k] = c.base[k];
        s_token[k] = c.page_bytes[k] / (unsigned)t.page;
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const ForkPlan f = plan[i];
        if (f.full < 0) continue;
        const int32_t* from = t.block_table + (size_t)parents[i] * t.max_blocks;
        const int child = children[i];
        int32_t* to = t.block_table + (size_t)child * t.max_blocks;
        for (int j = threadIdx.x; j < t.max_blocks; j += kCopyThreads) {
            int e = -1;
            if (j < f.full) {
                // from L2: a line of the table may hold rows that other SMs write
                e = __ldcg(from + j);
                atomicAdd(t.refcount + e, 1);
            } else if (j == f.full && f.part > 0) {
                e = f.fresh;
                t.refcount[e] = 1;
            }
            to[j] = e;
        }
        if (threadIdx.x == 0) t.ctx_lens[child] = f.full * t.page + f.part;
    }
    const unsigned items = (unsigned)c.num_caches << shift;
    const int du = gridDim.x / n, di = gridDim.x % n;
    unsigned u = blockIdx.x / n;
    int i = blockIdx.x % n;
    while (u < items) {
        const ForkPlan f = plan[i];
        const unsigned tb = s_token[u >> shift], off = (u & ((1u << shift) - 1u)) * kUnitBytes;
        const unsigned used = f.src >= 0 ? tb * (unsigned)f.part : 0u;
        if (off < used) {
            const unsigned pb = tb * (unsigned)t.page;
            unsigned char* base = s_base[u >> shift] + off;
            copy_unit(base + (size_t)f.fresh * pb, base + (size_t)f.src * pb,
                      min(kUnitBytes, used - off));
        }
        u += du;
        i += di;
        if (i >= n) {
            i -= n;
            ++u;
        }
    }
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------

// Lists of up to this many entries, and tables of up to this many rows, are
// planned in shared memory, a round trip to L2 less at each step (0.2 us of 59
// for a fork of 64 and its reserve); longer ones in the workspace.
constexpr int kSharedList = 1024, kSharedRows = 2048;

__global__ void __launch_bounds__(kPlanThreads)
    reserve_kernel(const PageTables t, int num_blocks, const int32_t* rows, const int32_t* tokens,
                   int n, int2* need_ws, int* first_ws, int* fresh, unsigned* err) {
    __shared__ int s[32];
    __shared__ int2 s_need[kSharedList];      // pages needed, first rank
    __shared__ int s_first[kSharedRows];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int2* need = n <= kSharedList ? s_need : need_ws;
    int* first = t.B <= kSharedRows ? s_first : first_ws;
    const unsigned mask = first_mask(t.refcount, num_blocks);
    first_entries(first, t.B, n, [&](int i) { return rows[i] < t.B ? rows[i] : -1; });
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int r = rows[i], tok = tokens[i];
        int count = 0;
        if (r >= 0) {
            unsigned bad = 0u;
            if (r >= t.B) bad = kErrRow;
            else if (first[r] != i) bad = kErrAlias;
            else if (tok < 0 || tok > t.max_blocks * t.page) bad = kErrCtx;
            if (!bad) {
                const int32_t* row = t.block_table + (size_t)r * t.max_blocks;
                for (int j = lane; j < ceil_div(tok, t.page); j += 32) count += __ldcg(row + j) < 0;
                count = warp_sum_i(count);
            } else if (lane == 0) {
                set_error(err, bad);
            }
        }
        if (lane == 0) need[i].x = count;
    }
    __syncthreads();
    // A row is served if its last rank is below the number of free pages; a
    // rank past the pool is held at its size, and one row's need too (1024
    // needs below 2^21 add up in 32 bits).
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + (int)threadIdx.x;
        const int v = i < n ? min(need[i].x, num_blocks) : 0;
        int total;
        const int rank = min(want + block_exclusive(v, s, total), num_blocks);
        if (i < n) need[i].y = rank;
        want = min(want + min(total, num_blocks), num_blocks);
    }
    __syncthreads();
    const int found = lowest_free(t.refcount, num_blocks, mask, want, s,
                                  [&](int rank, int page) { fresh[rank] = page; });
    __syncthreads();
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const int2 want_at = need[i];
        if (want_at.x == 0) continue;
        if (want_at.x > found - want_at.y) {
            if (lane == 0) set_error(err, kErrPages);
            continue;
        }
        int32_t* row = t.block_table + (size_t)rows[i] * t.max_blocks;
        const int entries = ceil_div(tokens[i], t.page);
        int at = want_at.y;
        for (int j0 = 0; j0 < entries; j0 += 32) {
            const int j = j0 + lane;
            const bool empty = j < entries && __ldcg(row + j) < 0;
            const unsigned m = __ballot_sync(0xffffffffu, empty);
            if (empty) {
                const int page = fresh[at + __popc(m & ((1u << lane) - 1u))];
                row[j] = page;
                t.refcount[page] = 1;
            }
            at += __popc(m);
        }
    }
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------

// One warp per listed row. Each entry is taken by an atomic exchange, so a row
// named twice gives its pages back once.
__global__ void __launch_bounds__(kCopyThreads)
    free_kernel(const PageTables t, int num_blocks, const int32_t* rows, int n, unsigned* err) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= n) return;
    const int r = rows[i];
    if (r < 0) return;
    if (r >= t.B) {
        if (lane == 0) set_error(err, kErrRow);
        return;
    }
    int32_t* row = t.block_table + (size_t)r * t.max_blocks;
    for (int j = lane; j < t.max_blocks; j += 32) {
        if (__ldcg(row + j) < 0) continue;
        const int e = atomicExch(row + j, -1);
        if (e < 0) continue;
        if (e >= num_blocks) {
            set_error(err, kErrBlock);
        } else if (atomicSub(t.refcount + e, 1) <= 0) {
            atomicAdd(t.refcount + e, 1);   // the page was free already
            set_error(err, kErrBlock);
        }
    }
    if (lane == 0) t.ctx_lens[r] = 0;
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

// head[0] = live pages, head[1] = moves; move k takes page from[k] (the k-th
// live page at or past head[0]) to page to[k] (the k-th free page below it);
// remap[p - head[0]] for p >= head[0]: the page's new number, -1 if free.
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const int32_t* refcount, int num_blocks, int* head, int* from,
                        int* to, int* remap, int32_t* num_live) {
    __shared__ int s[32];
    pdl_wait();
    pdl_trigger();
    const int quads = num_blocks / 4 + (num_blocks % 4 != 0);
    int free_pages = 0;
    for (int q = threadIdx.x; q < quads; q += kPlanThreads)
        free_pages += __popc(free_mask(refcount, q, num_blocks));
    int total;
    block_exclusive(free_pages, s, total);
    const int live = num_blocks - total;
    const int holes = lowest_free(refcount, live, first_mask(refcount, live), num_blocks, s,
                                  [&](int rank, int page) { to[rank] = page; });
    __syncthreads();
    int moved = 0;
    for (int q0 = live / 4; q0 < quads; q0 += kPlanThreads) {
        const int q = q0 + (int)threadIdx.x;
        unsigned used = 0;
        if (q < quads) {
            used = ~free_mask(refcount, q, num_blocks) & 15u;
            for (int k = 0; k < 4; ++k)
                if (4 * q + k < live || 4 * q + k >= num_blocks) used &= ~(1u << k);
        }
        int rank = moved + block_exclusive(__popc(used), s, total);
        for (int k = 0; k < 4; ++k) {
            const int p = 4 * q + k;
            if (q >= quads || p < live || p >= num_blocks) continue;
            int r = -1;
            if (used >> k & 1u) {
                r = to[rank];
                from[rank++] = p;
            }
            remap[p - live] = r;
        }
        moved += total;
    }
    if (threadIdx.x == 0) {
        head[0] = live;
        head[1] = holes;
        if (num_live) *num_live = live;
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(const __grid_constant__ CacheList c, const PageTables t, const int* head,
                         const int* from, const int* to, const int* remap, unsigned* err) {
    pdl_wait();
    pdl_trigger();
    const int live = head[0], moves = head[1];
    const long tid = (long)blockIdx.x * kCopyThreads + threadIdx.x;
    const long stride = (long)gridDim.x * kCopyThreads;
    for (long i = tid; i < (long)t.B * t.max_blocks; i += stride) {
        const int e = t.block_table[i];
        if (e < live) continue;
        const int r = e < c.num_blocks ? remap[e - live] : -1;
        if (r < 0) set_error(err, kErrBlock);   // left as it is
        else t.block_table[i] = r;
    }
    for (long k = tid; k < moves; k += stride) {
        t.refcount[to[k]] = t.refcount[from[k]];
        t.refcount[from[k]] = 0;
    }
    const unsigned U = c.first_unit[c.num_caches];
    const long total = (long)moves * U;
    for (long u = blockIdx.x; u < total; u += gridDim.x) {
        const int k = (int)(u / U);
        copy_page_unit(c, (unsigned)(u - (long)k * U), from[k], to[k]);
    }
}

// ---------------------------------------------------------------------------

template <typename Kern, typename... Args>
cudaError_t launch_pages(Kern kern, int grid, int block, const Launch& L, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// CTAs for `units` copy units of kUnitBytes at most.
int copy_grid(long units, int per_sm, const Launch& L) {
    return (int)std::max(1L, std::min(units, (long)L.num_sms * per_sm));
}

constexpr size_t kPart = 256;
size_t up(size_t x) { return (x + kPart - 1) / kPart * kPart; }

// The workspace: plans [n], needs [n], first [B], then three lists of
// num_blocks page numbers, and a head.
struct PageWs {
    size_t plan, need, first, list, total;
};
PageWs page_ws(int num_blocks, int B, int n) {
    PageWs w;
    w.plan = kPart;
    w.need = w.plan + up((size_t)n * sizeof(ForkPlan));
    w.first = w.need + up((size_t)n * 8);
    w.list = w.first + up((size_t)B * 4);
    w.total = w.list + 3 * up((size_t)num_blocks * 4);
    return w;
}

}  // namespace

void page_units(CacheList& c) {
    unsigned u = 0;
    for (int k = 0; k < c.num_caches; ++k) {
        c.first_unit[k] = u;
        u += (c.page_bytes[k] + kUnitBytes - 1) / kUnitBytes;
    }
    c.first_unit[c.num_caches] = u;
}

size_t pages_workspace_bytes(int num_blocks, int B, int n) {
    return page_ws(num_blocks, B, n).total;
}

cudaError_t launch_copy_pages(const CacheList& c, const int32_t* src, const int32_t* dst, int n,
                              unsigned* err, const Launch& L) {
    const long units = (long)n * c.first_unit[c.num_caches];
    return launch_pages(copy_pages_kernel, copy_grid(units, kCopyCtasPerSm, L), kCopyThreads, L, c,
                        src, dst, n, err);
}

cudaError_t launch_fork(const CacheList& c, const PageTables& t, const int32_t* parents,
                        const int32_t* children, int n, void* ws, unsigned* err, const Launch& L) {
    const PageWs w = page_ws(c.num_blocks, t.B, n);
    unsigned char* p = static_cast<unsigned char*>(ws);
    ForkPlan* plan = reinterpret_cast<ForkPlan*>(p + w.plan);
    cudaError_t e = launch_pages(fork_plan_kernel, 1, kPlanThreads, L, t, c.num_blocks, parents,
                                 children, n, plan, reinterpret_cast<int*>(p + w.need),
                                 reinterpret_cast<int*>(p + w.first), err);
    if (e != cudaSuccess) return e;
    unsigned largest = 0;
    for (int k = 0; k < c.num_caches; ++k) largest = std::max(largest, c.page_bytes[k]);
    int shift = 0;
    while (((size_t)kUnitBytes << shift) < largest) ++shift;
    const long items = ((long)n * c.num_caches) << shift;
    return launch_pages(fork_apply_kernel, copy_grid(items, kForkCtasPerSm, L), kCopyThreads, L, c,
                        t, parents, children, n, (const ForkPlan*)plan, shift);
}

cudaError_t launch_reserve(const PageTables& t, int num_blocks, const int32_t* rows,
                           const int32_t* tokens, int n, void* ws, unsigned* err, const Launch& L) {
    const PageWs w = page_ws(num_blocks, t.B, n);
    unsigned char* p = static_cast<unsigned char*>(ws);
    return launch_pages(reserve_kernel, 1, kPlanThreads, L, t, num_blocks, rows, tokens, n,
                        reinterpret_cast<int2*>(p + w.need), reinterpret_cast<int*>(p + w.first),
                        reinterpret_cast<int*>(p + w.list), err);
}

cudaError_t launch_free(const PageTables& t, int num_blocks, const int32_t* rows, int n,
                        unsigned* err, const Launch& L) {
    const int warps = kCopyThreads / 32;
    return launch_pages(free_kernel, n / warps + (n % warps != 0), kCopyThreads, L, t, num_blocks,
                        rows, n, err);
}

cudaError_t launch_compact(const CacheList& c, const PageTables& t, int32_t* num_live, void* ws,
                           unsigned* err, const Launch& L) {
    const PageWs w = page_ws(c.num_blocks, t.B, 0);
    unsigned char* p = static_cast<unsigned char*>(ws);
    const size_t list = up((size_t)c.num_blocks * 4);
    int* head = reinterpret_cast<int*>(p);
    int* from = reinterpret_cast<int*>(p + w.list);
    int* to = reinterpret_cast<int*>(p + w.list + list);
    int* remap = reinterpret_cast<int*>(p + w.list + 2 * list);
    cudaError_t e = launch_pages(compact_plan_kernel, 1, kPlanThreads, L,
                                 (const int32_t*)t.refcount, c.num_blocks, head, from, to, remap,
                                 num_live);
    if (e != cudaSuccess) return e;
    return launch_pages(compact_apply_kernel, L.num_sms * kCopyCtasPerSm, kCopyThreads, L, c, t,
                        (const int*)head, (const int*)from, (const int*)to, (const int*)remap, err);
}

}  // namespace a8w8
