// attn_chunk.cu -- attention of a chunk of new tokens over a paged KV cache.
//
// Request b's n new tokens are the last of its ctx cached ones; row i of them sees
// keys t <= ctx - n + i. Per row and query head, over BF16, INT8 or 4-bit rows:
//   s_t = scale q.k_t,  o = sum_t e^{s_t} v_t / sum_t e^{s_t}.
//
// What bounds it: the matrix units where a tile of rows is full (4 D operations a
// row and key: a prompt), HBM where it is not (single tokens and drafts over long
// contexts). One kernel covers both, since a batch mixes them:
//   - A tile is 256 rows, the G query heads of one KV head times 256 / G tokens: a
//     key read serves them all, and G = 1 to 8 fill the MMA's 128 lanes.
//   - The tiles' blocks of 128 keys laid end to end are cut into equal parts, one
//     a CTA (chunk_plan.cuh), wherever that falls. A tile in several parts leaves
//     partials (O, maximum, sum, in float32), which a second kernel joins.
//   - S = Q K^T and O = P V are tcgen05 products of 128 x 128 x 16 with the
//     accumulators in tensor memory, P written back there over S as 16-bit. Two
//     streams of 128 rows each take turns: one's softmax runs beside the other's
//     products. A tile of 128 rows or fewer gives the streams every other block of
//     keys instead, joined at its end.
//   - Softmax: a thread a row, no shuffles. Exponentials are taken against the
//     row's last reference first and its maximum beside them; only where that
//     grew by more than 2^8 are O and the sum rescaled and they are taken again.
//   - P is rounded to BF16 (a BF16 cache) or FP16 (2^-8 or 2^-11 of a weight): what the
//     products take; over INT8 and 4-bit rows the finer one, as K and V are FP16 there.
//     Sums, maxima and O are float32.
//   - Sixteen warps: two warpgroups of softmax, one that brings K and V (asynchronous
//     copies of rows by the block table; a page may end anywhere) or makes FP16 of their
//     codes, one thread that issues products, three warps for queries and codes.
// The order of the sums depends on the sizes and the grid alone: the same call gives
// the same bits.
//
// Measured (GB300, a graph's launch; 40 heads on 8 of 128 where not said):
//   a prompt of 16384 tokens, BF16        1.93 ms, 1420 TFLOP/s of 1920
//   the same, INT8 and 4-bit              2.75 and 2.59 ms, 1000 and 1060 TFLOP/s
//   512 tokens at 16384, BF16             152 us, 1110 TFLOP/s
//   4 prompts of 512, BF16                34 us
//   16 single tokens past 63 to 4095      39 us, 3.5 TB/s of 6.8
//   64 x 4 drafts past 64 to 4096, 4-bit  146 us, 1.0 TB/s
//   16 requests of 1 to 512 tokens, INT8  214 us, 620 TFLOP/s
// Long ones are bound by a stream's chain S -> softmax -> P -> O of a block (2900 clocks
// for both streams' blocks, 2048 of them products); INT8 and 4-bit ones by the
// conversion (3500 to 4400 a block); short ones by the start: 7000 clocks to find the
// part, 8000 more to the first S (table, keys, code that no cache holds yet).
#include <algorithm>

#include <cuda_fp16.h>

#include "chunk_plan.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace a8w8 {

namespace {

using namespace tc;
using namespace chunk;

constexpr unsigned kErrBlock = 0x2u, kErrCtx = 0x4u, kErrTimeout = 0x20u, kErrRow = 0x40u;

constexpr int kStreamRows = 128;      // rows of a stream: the MMA's M, the tensor memory's lanes
constexpr int kHalf = kKeys / 2;      // keys whose scores and weights go round at a time
constexpr int kThreads = 512;         // warps 0-7 softmax, 8-11 keys and values, 12 MMA, 13-15 queries
constexpr int kMaxParts = 152;
constexpr uint32_t kTmemCols = 512;   // S of stream s at 128 s, O of stream s at 256 + D s
constexpr uint32_t kColO = 256;
constexpr float kLazy = 8.0f;         // a row's reference may lag behind its maximum by 2^8

template <int D>
__host__ __device__ constexpr int tile_bytes() { return kKeys * D * 2; }
template <int D, int KV>
__host__ __device__ constexpr int num_stages() {
    return (KV == kKvBf16 ? 5 : 3) * 128 / D;
}
// Tiles of codes on their way, INT8 and 4-bit caches: 48 KB of the shared memory.
template <int D, int KV>
__host__ __device__ constexpr int raw_tiles() {
    return KV == kKvBf16 ? 0 : (KV == kKvI8 ? 3 : 6) * 128 / D;
}

struct Ctl {
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_first, q_full[2], q_free[2];                     // by the segment's parity
    uint64_t q_ready[2];                                        // INT8, 4-bit: made FP16
    uint64_t s_full[2], p_full[2][2], pv_half[2], pv_done[2];   // of stream (and half block)
    uint64_t o_free, merge, done;
    long u0, u1;                   // this part's units
    int b, h, i;                   // its first unit's request, KV head, tile
    long first;                    // and that tile's first unit
    int v_unit[2];                 // narrow tiles: a stream's O is in units of 2^this
    int bad_tile;                  // the segment that bad[] is about, -1 for none
    uint32_t tmem;
    volatile int abort, never;     // never: always 0
};

constexpr int kFeeders = 3;            // warps 13-15
// INT8 and 4-bit caches: the ring of codes, a block's largest pairs by the warps that convert.
struct CodesCtl {
    uint64_t full[12], empty[12], tops;
    uint2 top[2][4];
};
constexpr int kFacRing = 8, kPairRing = 8;     // blocks

template <int D, int KV>
struct Lay {
    static constexpr int kSt = num_stages<D, KV>();
    static constexpr size_t q = 0;                                   // two tiles of 128 rows
    static constexpr size_t kv = 2 * (size_t)tile_bytes<D>();
    static constexpr size_t stat = kv + (size_t)kSt * tile_bytes<D>();   // (ref, sum) [2][128]
    static constexpr size_t bad = stat + 2 * kStreamRows * 8;        // see BadValues
    static constexpr size_t ctl = bad + D * 4;
    static constexpr size_t fac = ctl + (sizeof(Ctl) + 15) / 16 * 16;    // see convert_codes, q_to_f16
    static constexpr size_t raw = fac + (KV == kKvBf16 ? 0 : kFacRing * 8 + 4 * kTileRows * 4);
    static constexpr size_t pairs = raw + (KV == kKvBf16 ? 0 : 48 * 1024);
    static constexpr size_t codes = pairs + (KV == kKvBf16 ? 0 : kPairRing * kKeys * 8);
    static constexpr size_t total = codes + (KV == kKvBf16 ? 0 : sizeof(CodesCtl));
};

// tc::mbar_wait with the limit (about two seconds) by the SM's clock: a third of
// the code, which counts here, as the roles' loops have to share the
// instruction cache.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (*abort || clock64() - t0 > 4000000000ll) return false;
    } while (!mbar_try_wait(bar, parity));
    return true;
}

// Whether that phase is over, without a wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same after a wait of half a microsecond at most.
__device__ __forceinline__ bool mbar_wait_shortly(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(500u)
        : "memory");
    return ok != 0;
}

// ex2 of the special function unit: 2^-22 relative, 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {   // a in the low half
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// Sixteen bytes to shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void cp16z(uint32_t s, const void* g, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(g), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t s, const void* g, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(g), "r"(bytes) : "memory");
}
// An arrival on the barrier once this thread's copies so far have landed (one of
// the barrier's count). The copies write through the generic proxy: who waits
// orders them before the tensor cores' reads by fence_async_shared().
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
template <int R>
__device__ __forceinline__ void set_max_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_max_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

#define A8W8_R8(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), \
                   "=r"(r[b + 5]), "=r"(r[b + 6]), "=r"(r[b + 7])
// 64 consecutive columns of the warp's lanes, loaded and waited for in one statement.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, "
        "%45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : A8W8_R8(0), A8W8_R8(8), A8W8_R8(16), A8W8_R8(24), A8W8_R8(32), A8W8_R8(40), A8W8_R8(48),
          A8W8_R8(56)
        : "r"(taddr)
        : "memory");
}
#undef A8W8_R8

// Shared-memory descriptor of an operand whose rows are contiguous along M or
// N (the values' rows: 64 dimensions of a token are 128 bytes), in the layout
// of sw128_kmajor_desc: groups of 8 tokens 1024 bytes apart (stride offset),
// the next 64 dimensions a whole sub-tile of 128 tokens further (leading
// offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t next64) {
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(next64 >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// idesc_f16_f32 with the operands' type (BF16: format 1) and, for B contiguous
// along N, the transpose bit 16. Bit 13 negates A.
constexpr uint32_t kNegateA = 1u << 13;
__host__ __device__ constexpr uint32_t idesc_chunk(bool bf, int N, bool b_mn) {
    return idesc_f16_f32(kStreamRows, N) | (bf ? (1u << 7) | (1u << 10) : 0u) |
           (b_mn ? 1u << 16 : 0u);
}

// Byte offset of 16-byte chunk c of row r in a tile of 128 rows: sub-tiles of
// 64 elements, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// A request as the tables give it: rows clamped to [0, T), no context where it
// is out of range (flagged, if `check`).
__device__ __forceinline__ Req load_req(const ChunkParams& p, int b, bool check = false) {
    Req r;
    const int a = p.q_starts[b], e = p.q_starts[b + 1], c = p.ctx_lens[b];
    r.row0 = min(max(a, 0), p.T);
    r.n = max(min(max(e, 0), p.T) - r.row0, 0);      // (each end clamped: any int is safe)
    const bool out = c < 0 || c > p.max_blocks * p.page;
    r.ctx = out ? 0 : c;
    if (check) {
        if (out) set_error(p.err, kErrCtx);
        if (a < 0 || e < a || e > p.T) set_error(p.err, kErrRow);
    }
    return r;
}

// A tile's blocks within the part.
struct Seg {
    int k;                // which segment of the part
    int b, h, i;
    int row0, ntok;       // the tile's first row of q and its tokens
    int pos0;             // position of its first token
    int kend;             // keys that its last token sees (0 or more)
    int j0, j1;           // key blocks
    bool head, tail;      // the tile begins, ends in this part
    __device__ __forceinline__ int blocks() const { return j1 - j0; }
};

// Walks the part's tiles; every role of the CTA does, on its own.
struct Walk {
    const ChunkParams& p;
    long u, u1, tile;      // next unit, end, first unit of the current tile
    int b, h, i, tpt, nt, k;
    Req r;
    __device__ __forceinline__ Walk(const ChunkParams& p_, const Ctl& c)
        : p(p_), u(c.u0), u1(c.u1), tile(c.first), b(c.b), h(c.h), i(c.i), k(0) {
        tpt = tile_tokens(p.G);
        if (u < u1) {
            r = load_req(p, b);
            nt = tiles_of(r, tpt);
        }
    }
    __device__ __forceinline__ bool next(Seg& s) {
        if (u >= u1) return false;
        if (i == nt) {
            i = 0;
            if (++h == p.Hkv) {
                h = 0;
                do r = load_req(p, ++b);
                while (r.n == 0);
                nt = tiles_of(r, tpt);
            }
        }
        const long keys = keys_of(r, tpt, i);
        const int nb = blocks_of(keys);
        s.k = k++;
        s.b = b;
        s.h = h;
        s.i = i;
        s.row0 = r.row0 + i * tpt;
        s.ntok = tokens_in(r, tpt, i);
        s.kend = keys > 0 ? (int)keys : 0;
        s.pos0 = (int)(keys - s.ntok);
        const int cost = cost_of(is_narrow(s.ntok, tpt));
        s.head = u == tile;
        s.j0 = s.head ? 0 : (int)(u - tile) - cost;
        s.j1 = (int)min((long)nb, u1 - tile - cost);
        s.tail = s.j1 == nb;
        if (s.tail) {
            u = tile += tile_units(r, tpt, i);
            ++i;
        } else {
            u = u1;
        }
        return true;
    }
};

// What the second kernel needs of the tile that a part begins in.
struct alignas(32) PlanEntry {
    int inside;           // whether it begins inside one
    int kf, kl;           // the parts that do in this tile; part kf - 1 holds the tile's begin
    int row0, ntok;       // as Seg
    int pos0, h, pad;
};
__host__ __device__ constexpr size_t plan_bytes() {
    return (kMaxParts * sizeof(PlanEntry) + 255) / 256 * 256;
}

// Workspace: the plan, then per part two slots (0: the tile that it begins
// inside, 1: the one whose begin it holds and whose end it does not): of `rows`
// rows each (ref, sum), then o in groups of four columns, the rows of a group side by
// side, as the threads that hold a row each write them.
struct PartView {
    float* base;
    int D, rows;
    __host__ __device__ static size_t floats(int D, int rows) { return (size_t)(rows + 3) / 4 * 4 * (D + 2); }
    __device__ __forceinline__ int pad() const { return (rows + 3) / 4 * 4; }
    __device__ __forceinline__ float* slot(int part, int which) const {
        return base + (size_t)(part * 2 + which) * floats(D, rows);
    }
    __device__ __forceinline__ float2* stat(float* slot, int row) const {
        return reinterpret_cast<float2*>(slot) + row;
    }
    __device__ __forceinline__ float4* o(float* slot, int row, int c) const {   // columns 4 c ..
        return reinterpret_cast<float4*>(slot + 2 * pad()) + (size_t)c * pad() + row;
    }
};

__device__ __forceinline__ void set_timeout(unsigned* err, volatile int* abort) {
    *abort = 1;
    set_error(err, kErrTimeout);
}

// ---------------------------------------------------------------------------
// The part's units
// ---------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_l2(const void* g) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(g));
}

// Exclusive sum of v over the CTA's threads; `s` is one long per warp.
__device__ __forceinline__ long cta_exclusive(long v, long* s, long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    long before = 0;
    total = 0;
#pragma unroll 4
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s[w];
        total += s[w];
    }
    return before + x - v;
}

// Finds this CTA's part: the requests' units added up, each thread a few; the
// thread that holds the part's first unit (and the next part's) names the
// request and the head; half of the threads each then look for the tile, one tile a
// thread. `scratch` is shared memory that nothing else uses yet.
__device__ __forceinline__ void find_part(const ChunkParams& p, Ctl& ctl, void* scratch) {
    struct Hit {
        long raw, head, tile;   // the unit, and the first one of its head, then of its tile
        Req r;
        int b, h, i;
    };
    long* sums = static_cast<long*>(scratch);
    Hit* hits = reinterpret_cast<Hit*>(sums + kThreads / 32);
    const int tpt = tile_tokens(p.G);
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    long mine = 0, head = 0;
    Req r = {};
    for (int b = b0; b < b1; ++b) {
        r = load_req(p, b, blockIdx.x == 0);
        head = head_units(r, tpt);
        mine += head * p.Hkv;
    }
    long W;
    const long before = cta_exclusive(mine, sums, W);
    const Shares sh(W, gridDim.x);
    const int c = blockIdx.x;
    if (c < sh.parts && mine > 0) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const long raw = sh.raw(c + k);
            if (c + k == sh.parts || raw < before || raw - before >= mine) continue;
            long at = before;
            int b = b0;
            if (per > 1) {
                for (;; ++b) {
                    r = load_req(p, b);
                    head = head_units(r, tpt);
                    if (raw - at < head * p.Hkv) break;
                    at += head * p.Hkv;
                }
            }
            const int h = (int)div_long(raw - at, head);
            hits[k].raw = raw;
            hits[k].head = at + h * head;
            hits[k].r = r;
            hits[k].b = b;
            hits[k].h = h;
        }
    }
    __syncthreads();
    const int k = threadIdx.x / (kThreads / 2);
    if (c + k < sh.parts) {
        Hit& x = hits[k];
        const Req rk = x.r;
        const long at = x.raw - x.head;
        const int nt = tiles_of(rk, tpt);
        for (int i = threadIdx.x % (kThreads / 2); i < nt; i += kThreads / 2) {
            const long u = units_before(rk, tpt, i);
            if (u <= at && at < u + tile_units(rk, tpt, i)) {
                x.i = i;
                x.tile = x.head + u;
                if (k == 0) {        // where the first keys' block id is, about
                    const long at_key = max(at - u - cost_of(is_narrow(tokens_in(rk, tpt, i), tpt)), 0l) * kKeys;
                    prefetch_l2(p.block_table + (size_t)x.b * p.max_blocks +
                                min((int)((unsigned)min(at_key, 0x7FFFFFFFl) / (unsigned)p.page), p.max_blocks - 1));
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        PlanEntry e = {};
        ctl.u0 = ctl.u1 = 0;
        if (c < sh.parts) {
            Hit x = hits[0];
            const long end = x.tile + tile_units(x.r, tpt, x.i), slack = sh.slack(x.r, tpt, x.i);
            ctl.u0 = sh.snap(x.raw, x.tile, end, slack);
            ctl.u1 = W;
            if (c + 1 < sh.parts) {
                const Hit& y = hits[1];
                ctl.u1 = sh.snap(y.raw, y.tile, y.tile + tile_units(y.r, tpt, y.i), sh.slack(y.r, tpt, y.i));
            }
            if (ctl.u0 > x.tile && ctl.u0 < end) {
                const long keys = keys_of(x.r, tpt, x.i);
                sh.inside(x.tile, end, slack, c, e.kf, e.kl);
                e.inside = 1;
                e.row0 = x.r.row0 + x.i * tpt;
                e.ntok = tokens_in(x.r, tpt, x.i);
                e.pos0 = (int)(keys - e.ntok);
                e.h = x.h;
            } else if (ctl.u0 == end) {      // the next tile's begin
                x.tile = end;
                if (++x.i == tiles_of(x.r, tpt)) {
                    x.i = 0;
                    if (++x.h == p.Hkv) {
                        x.h = 0;
                        do ++x.b;
                        while (x.b < p.B && load_req(p, x.b).n == 0);
                    }
                }
            }
            ctl.b = x.b;
            ctl.h = x.h;
            ctl.i = x.i;
            ctl.first = x.tile;
        }
        reinterpret_cast<PlanEntry*>(p.ws)[c] = e;
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Infinities and NaN among the values
// ---------------------------------------------------------------------------

// A product with V multiplies a weight of zero with the values of tokens that a
// row does not see; that is nothing for finite values only. So the values of the
// tokens that some rows of a tile see and others do not (those behind its first
// token) are looked over as they are loaded: an infinity or NaN becomes zero and
// is noted by its dimension as the first token that has a NaN, plus or minus
// infinity there (ten bits each, counted from `base`); the rows that see it get
// it back at the end. One segment at a time holds the notes, in their order: a segment ends
// only when all of its values have come, so an earlier one must never find the notes
// held by a later one.
constexpr uint32_t kNoBad = 0x3FFFFFFFu;
struct BadValues {
    uint32_t* words;      // [D]
    Ctl& ctl;
    unsigned* err;
    __device__ __forceinline__ static int base(const Seg& s) { return (s.pos0 + 1) & ~(kKeys - 1); }
    // kind 0: NaN, 1: infinity, 2: minus infinity. `before`: the barrier (and the phase) by
    // which all have looked over the segments before, null where that is known.
    __device__ __noinline__ void note(int seg, int token, int d, int kind, uint64_t* before = nullptr,
                                      unsigned parity = 0) {
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (!before || mbar_test(before, parity)) {
                const int owner = atomicCAS(&ctl.bad_tile, -1, seg);
                if (owner == -1 || owner == seg) break;
            }
            if (ctl.abort) return;
            if (globaltimer_ns() - t0 > 2000000000ull) {
                set_timeout(err, &ctl.abort);
                return;
            }
        }
        uint32_t old = words[d], was;
        do {
            was = old;
            const uint32_t field = (was >> (10 * kind)) & 1023u;
            if (field <= (uint32_t)token) return;
            const uint32_t now = (was & ~(1023u << (10 * kind))) | ((uint32_t)token << (10 * kind));
            old = atomicCAS(&words[d], was, now);
        } while (old != was);
    }
    __device__ __forceinline__ bool any(int seg) const {
        return *reinterpret_cast<volatile int*>(&ctl.bad_tile) == seg;
    }
    // Adds what the notes hold for a row that sees the tokens up to `last` (from base) to its
    // dimensions [d0, d1): in `out`, or in `part` (groups of four, `step` floats apart).
    template <int D>
    __device__ __noinline__ void add(int last, int d0, int d1, bf16* out, float* part, int step) const {
        for (int d = d0; d < d1; ++d) {
            const uint32_t w = *reinterpret_cast<volatile uint32_t*>(&words[d]);
            float x = 0.0f;
            if ((int)(w & 1023u) <= last) x = __int_as_float(0x7FC00000);
            if ((int)((w >> 10) & 1023u) <= last) x += INFINITY;
            if ((int)((w >> 20) & 1023u) <= last) x -= INFINITY;
            if (x == 0.0f) continue;
            if (out) out[d] = f2bf(__bfloat162float(out[d]) + x);
            else part[(size_t)(d >> 2) * step + (d & 3)] += x;
        }
    }
    // By one warp, when all have read segment seg's notes.
    __device__ __forceinline__ void clear(int seg, int D) {
        if (!any(seg)) return;
        for (int d = threadIdx.x & 31; d < D; d += 32) words[d] = kNoBad;
        __threadfence_block();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) atomicExch(&ctl.bad_tile, -1);
        __syncwarp();
    }
};

// ---------------------------------------------------------------------------
// Keys and values: four warps, a warp the tokens 32 w .. 32 w + 31 of a block
// ---------------------------------------------------------------------------

// Where token t of request b lies, in two steps: its block id is read (no token
// beyond kend, the tile's last key), and some work later made a slot, -1 for no
// token and for a bad block id. Read and used at once, each costs its latency.
struct Look {
    int blk, off;         // blk -2: no token
};
__device__ __forceinline__ Look look_up(const ChunkParams& p, int b, int kend, int t) {
    const unsigned k = (unsigned)t / (unsigned)p.page;
    Look l = {-2, t - (int)k * p.page};
    if (t < kend) l.blk = p.block_table[(size_t)b * p.max_blocks + k];
    return l;
}
__device__ __forceinline__ int slot_of(const ChunkParams& p, const Look& l) {
    if ((unsigned)l.blk < (unsigned)p.num_blocks) return l.blk * p.page + l.off;
    if (l.blk != -2) set_error(p.err, kErrBlock);
    return -1;
}

template <int D>
__device__ void load_bf16(const ChunkParams& p, Ctl& ctl, uint32_t kv, unsigned char* kvp,
                          BadValues bad) {
    constexpr int kSt = num_stages<D, kKvBf16>();
    constexpr int CPR = D / 8;            // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;         // rows that one copy instruction covers
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
    const int c = lane % CPR, rl = lane / CPR;
    unsigned cnt = 0;
    Walk walk(p, ctl);
    Seg s;
    bool ok = true;
    // a tile of values that is still to be looked over: its ring tile, segment, rows
    // [lo, hi), the first row's token from BadValues::base, its number and that of its
    // segment's first tile
    struct { int st, seg, lo, hi, tok; unsigned at, first; } look = {-1, 0, 0, 0, 0, 0, 0};
    // The warps do not wait for one another here. All have looked over the segments before
    // when the tile before this segment has come. From kSt tiles behind it on that is so,
    // as its place in the ring was free again; up to there its barrier cannot be past the
    // phase behind it, which needs this warp.
    auto look_over = [&]() {
        unsigned char* tile = kvp + look.st * tile_bytes<D>();
#pragma unroll 1
        for (int i = 0; i < 32 / RPI; ++i) {
            const int row = 32 * w + i * RPI + rl;
            if (row < look.lo || row >= look.hi) continue;
            uint4& v = *reinterpret_cast<uint4*>(tile + tile_off(row, c));
            const uint4 x = v;
            auto odd = [](uint32_t u) { return (u & 0x7F80u) == 0x7F80u || (u & 0x7F800000u) == 0x7F800000u; };
            if (!(odd(x.x) || odd(x.y) || odd(x.z) || odd(x.w))) continue;
            uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const uint32_t h = (u[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                if ((h & 0x7F80u) != 0x7F80u) continue;
                const unsigned prev = look.first - 1;
                const bool ask = look.first && look.at - prev < kSt;
                bad.note(look.seg, look.tok + row, 8 * c + e, h & 0x7Fu ? 0 : h & 0x8000u ? 2 : 1,
                         ask ? &ctl.kv_full[prev % kSt] : nullptr, (prev / kSt) & 1);
                u[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            }
            v = make_uint4(u[0], u[1], u[2], u[3]);
        }
        fence_async_shared();
        mbar_arrive(&ctl.kv_full[look.st]);
        look.st = -1;
    };
    while (ok && walk.next(s)) {
        const unsigned first = cnt;
        Look next = look_up(p, s.b, s.kend, s.j0 * kKeys + 32 * w + lane);
        for (int j = s.j0; ok && j < s.j1; ++j) {
            const int slot = slot_of(p, next);
            if (j + 1 < s.j1) next = look_up(p, s.b, s.kend, (j + 1) * kKeys + 32 * w + lane);
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                const int st = cnt % kSt;
                if (cnt >= kSt && !mbar_try_wait(&ctl.kv_empty[st], (cnt / kSt - 1) & 1)) {
                    if (look.st >= 0) {
                        cp_async_wait_all();
                        look_over();
                    }
                    if (!wait_bar(&ctl.kv_empty[st], (cnt / kSt - 1) & 1, &ctl.abort)) {
                        ok = false;
                        break;
                    }
                }
                const bf16* src = static_cast<const bf16*>(v ? p.v : p.k);
                const uint32_t dst = kv + st * tile_bytes<D>();
#pragma unroll
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int rr = i * RPI + rl, row = 32 * w + rr;
                    const int sl = __shfl_sync(0xffffffffu, slot, rr);
                    const bf16* g = src + ((size_t)max(sl, 0) * p.Hkv + s.h) * D + 8 * c;
                    cp16z(dst + tile_off(row, c), g, sl >= 0 ? 16u : 0u);
                }
                cp_async_commit();
                if (look.st >= 0) {              // behind this tile's copies, which go on
                    cp_async_wait_group<1>();
                    look_over();
                }
                const int lo = s.pos0 + 1 - j * kKeys, hi = s.kend - j * kKeys;
                if (v == 1 && lo < kKeys && hi > max(lo, 0)) {
                    look.st = st;
                    look.seg = s.k;
                    look.lo = lo;
                    look.hi = hi;
                    look.tok = j * kKeys - BadValues::base(s);
                    look.at = cnt;
                    look.first = first;
                } else {
                    cp_async_arrive(&ctl.kv_full[st]);
                }
                ++cnt;
            }
        }
    }
    if (!ok && !ctl.abort) set_timeout(p.err, &ctl.abort);
    cp_async_wait_all();
    if (look.st >= 0) look_over();
}

// INT8 and 4-bit rows become FP16 on the way into the ring: value 2^-E, E a
// whole number per block for keys (the softmax takes the power of two back with
// the scale) and for values one that only grows through a segment (O is in units
// of it). A block's largest |value| comes to between 8 and 16, and of later blocks of
// values to 2^15. A rounding to FP16 is off by 2^-11 of what it rounds, or by 2^-25
// below the normal numbers, which is 2^-28 of the largest value. An INT8 value has two,
// its row's scale (taken as 128 s, times code / 128) and the product: 2^-10 of
// itself, and 2^-27 of the largest. A 4-bit value has one, the sum's: pairs are BF16 and
// exact but below FP16's normal numbers (8 s and m; 15 codes / 8 of the one): 2^-11 of
// itself, and 2^-26 of the largest. (With s and code as they are, small rows' scales were
// off by 2^-21 of the block's largest value. As BF16 rows, scores
// would be off by 2^-8 of |q| |k|, several times what the weights' rounding
// does.)
//
// The codes and the pairs come by asynchronous copies into rings of their own
// (feed_codes). The four converting warps wait for one another once a block, for
// the largest pair of their quarters (each reading all pairs instead took 3000
// clocks of a block's 7900), so that all have looked over the blocks before.
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// The power of two 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The dimensions of value rows with an infinity or NaN, row r's in the mask of
// `odd` (its slot's first code and pair in lane r), go to the notes; tok0 is row
// 0's token from BadValues::base.
template <int D, int KV>
__device__ __noinline__ void note_rows(const void* codes, size_t row, uint32_t meta, unsigned odd, int tok0,
                                       int seg, BadValues bad) {
    const int lane = threadIdx.x & 31;
    for (; odd; odd &= odd - 1) {
        const int r = __ffs(odd) - 1;
        const size_t at = __shfl_sync(0xffffffffu, row, r);
        const uint32_t m = __shfl_sync(0xffffffffu, meta, r);
        const float sc = KV == kKvI8 ? __uint_as_float(m) : __uint_as_float(m << 16);
        const float mn = KV == kKvI8 ? 0.0f : __uint_as_float(m & 0xFFFF0000u);
        for (int d = lane; d < D; d += 32) {
            const size_t i = at * D + d;
            const float code = KV == kKvI8 ? (float)static_cast<const int8_t*>(codes)[i]
                                           : (float)(static_cast<const uint8_t*>(codes)[i / 2] >> (4 * (d & 1)) & 15);
            const float val = __fmaf_rn(code, sc, mn);
            bad.note(seg, tok0 + r, d, isnan(val) ? 0 : val < 0.0f ? 2 : 1);
        }
        __syncwarp();
    }
}

// The part's blocks one after the other.
struct Blocks {
    Walk walk;
    Seg s;
    int j;
    bool live, first;
    __device__ __forceinline__ Blocks(const ChunkParams& p, const Ctl& ctl) : walk(p, ctl) {
        j = -1;
        s.j1 = 0;
        next();
    }
    __device__ __forceinline__ void next() {
        first = false;
        if (++j >= s.j1) {
            live = walk.next(s);
            j = s.j0;
            first = true;
        }
    }
};

// A ring tile's codes: thread t of the four converting warps finds its 16-byte
// pieces, rows 32 (t / 32) + i RPI + (t % 32) / LPR, at 16 t + 2048 i.
template <int D, int KV>
struct Raw {
    static constexpr int kTiles = raw_tiles<D, KV>();
    static constexpr int RB = KV == kKvI8 ? D : D / 2;      // bytes of a row's codes
    static constexpr int LPR = RB / 16, RPI = 32 / LPR, NI = LPR;
    static_assert(kTiles * kKeys * RB == 48 * 1024 && kTiles <= 12, "the ring of codes");
    static_assert(kTiles / 2 + 1 < kPairRing, "copies are ahead by kTiles tiles, two a block");
};

template <int D, int KV>
__device__ void convert_codes(const ChunkParams& p, Ctl& ctl, CodesCtl& cc, unsigned char* kvp, const unsigned char* raw,
                              const uint2* pairs, float2* fac, BadValues bad) {
    using R = Raw<D, KV>;
    constexpr int kSt = num_stages<D, KV>(), kRaw = R::kTiles;
    constexpr int RB = R::RB, LPR = R::LPR, RPI = R::RPI, NI = R::NI;
    constexpr int CPC = KV == kKvI8 ? 2 : 4;         // 16-byte chunks of FP16 per 16 bytes of codes
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
    const int c = lane % LPR, rl = lane / LPR;
    const unsigned char* mine = raw + 16 * (threadIdx.x & 127);
    const uint2* my_pairs = pairs + (threadIdx.x & 127);

    // whether a row holds an infinity or NaN
    auto odd_row = [](uint32_t m) {
        if (KV == kKvI8) return (m & 0x7F800000u) == 0x7F800000u;
        return (m & 0x7F80u) == 0x7F80u || (m & 0x7F800000u) == 0x7F800000u;
    };
    // the largest |value| of a finite row by its pair, as a float's bits: 128 s (2^7 times what
    // this gives), or the larger of |m| and |m + 15 s|
    auto size_of = [&](uint32_t m) {
        if (odd_row(m)) return 0u;
        if (KV == kKvI8) return m & 0x7FFFFFFFu;
        const float least = __uint_as_float(m & 0xFFFF0000u);
        return max(m & 0x7FFF0000u,
                   __float_as_uint(__fmaf_rn(15.0f, __uint_as_float(m << 16), least)) & 0x7FFFFFFFu);
    };
    // e with |value| <= 2^e: -100 at least, -1000 for rows of zeros alone
    auto exponent_of = [](unsigned top) {
        return top == 0 ? -1000 : min(max((int)(top >> 23) - 126 + (KV == kKvI8 ? 7 : 0), -100), 131);
    };
    // Ring tile cnt from the thread's pieces of codes (pairs `meta` of the lanes' tokens) times `up`.
    // Where piece 0's chunks go. Lanes of one store in different banks: the second half of a
    // row's lanes takes its words' halves in the other order (the sub-tiles lie a multiple of
    // all banks apart).
    const bool turn = D == 128 && (KV == kKvI8 ? c >> 2 : c >> 1);
    uint32_t to[CPC];
#pragma unroll
    for (int e = 0; e < CPC; ++e)
        to[e] = tile_off(32 * w + rl, CPC * c + (turn ? e ^ (CPC / 2) : e));
    unsigned cnt = 0;
    auto convert = [&](uint32_t meta, float up) {
        const unsigned char* src = mine + (cnt % kRaw) * (kKeys * RB);
        unsigned char* tile = kvp + (cnt % kSt) * tile_bytes<D>();
        // (not unrolled further: the instruction cache is what these warps wait for most)
#pragma unroll 2
        for (int i = 0; i < NI; ++i) {
            const uint32_t m = __shfl_sync(0xffffffffu, meta, i * RPI + rl);
            const uint4 r = *reinterpret_cast<const uint4*>(src + 2048 * i);
            const uint32_t word[4] = {turn ? r.z : r.x, turn ? r.w : r.y, turn ? r.x : r.z, turn ? r.y : r.w};
            unsigned char* const row = tile + i * RPI * 128;
            const uint32_t flip = RPI == 4 && (i & 1) ? 64u : 0u;      // bit 2 of the row
            if (KV == kKvI8) {
                // 128 s and code / 128 (exact): s alone would leave FP16's normal numbers 2^7 earlier
                const __half2 sc = __float2half2_rn(__uint_as_float(m) * (up * 128.0f));
                const __half2 by = as_half2(0x20002000u), off = as_half2(0xC880C880u);   // 2^-7, -1152 2^-7
#pragma unroll
                for (int e = 0; e < CPC; ++e) {
                    uint32_t o[4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint32_t u = word[2 * e + g] ^ 0x80808080u;        // 1024 + 128 + code
                        o[2 * g] = as_u32(__hmul2(__hfma2(as_half2(__byte_perm(u, 0x64646464u, 0x4140)), by, off), sc));
                        o[2 * g + 1] = as_u32(__hmul2(__hfma2(as_half2(__byte_perm(u, 0x64646464u, 0x4342)), by, off), sc));
                    }
                    *reinterpret_cast<uint4*>(row + (to[e] ^ flip)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            } else {
                // 8 s and code / 8 (exact), as above; 8 s is 1.07 times the largest |value| at most
                const __half2 sc = __float2half2_rn(__uint_as_float(m << 16) * (up * 8.0f));
                const __half2 mn = __float2half2_rn(__uint_as_float(m & 0xFFFF0000u) * up);
                const __half2 by = as_half2(0x20003000u), off = as_half2(0xC800D800u);   // (2^-3, 2^-7), -1024 of them
#pragma unroll
                for (int e = 0; e < CPC; ++e) {
                    uint32_t o[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        // 1024 + low nibble, 1024 + 16 times the high one
                        const uint32_t u = __byte_perm(word[e], 0x64646464u, 0x4040 + 0x0101 * g) & 0x64F0640Fu;
                        o[g] = as_u32(__hfma2(__hfma2(as_half2(u), by, off), sc, mn));
                    }
                    *reinterpret_cast<uint4*>(row + (to[e] ^ flip)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
        fence_async_shared();
        mbar_arrive(&ctl.kv_full[cnt % kSt]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&cc.empty[cnt % kRaw]);
        ++cnt;
    };
    auto landed = [&]() { return wait_bar(&cc.full[cnt % kRaw], (cnt / kRaw) & 1, &ctl.abort); };
    auto room = [&]() {
        return cnt < kSt || wait_bar(&ctl.kv_empty[cnt % kSt], (cnt / kSt - 1) & 1, &ctl.abort);
    };

    Blocks x(p, ctl);
    unsigned blk = 0;
    int ev = -1000;
    bool ok = true;
    while (x.live) {
        if (!(ok = landed())) break;
        const uint2 m = my_pairs[(blk % kPairRing) * kKeys];
        const unsigned tk = __reduce_max_sync(0xffffffffu, size_of(m.x));
        const unsigned tv = __reduce_max_sync(0xffffffffu, size_of(m.y));
        if (lane == 0) {
            cc.top[blk & 1][w] = make_uint2(tk, tv);
            mbar_arrive(&cc.tops);
        }
        __syncwarp();
        if (!(ok = wait_bar(&cc.tops, blk & 1, &ctl.abort))) break;
        uint2 top = cc.top[blk & 1][0];
#pragma unroll
        for (int q = 1; q < 4; ++q) {
            const uint2 t = cc.top[blk & 1][q];
            top = make_uint2(max(top.x, t.x), max(top.y, t.y));
        }
        // the exponents, before the keys are handed over: the softmax reads them behind those
        int ek = exponent_of(top.x);
        ek = ek == -1000 ? 0 : ek;
        const int e = exponent_of(top.y);
        if (x.first) ev = e == -1000 ? -100 : e;
        else if (e > ev + 11) ev = e;
        if (threadIdx.x % 128 == 0)
            fac[blk % kFacRing] = make_float2(pow2(min(ek - 4, 127)), __int_as_float(min(ev - 4, 127)));
        uint32_t pair_of = m.x, vmine = m.y;
        float up = pow2(max(4 - ek, -126));
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
            if (!(ok = (v == 0 || landed()) && room())) break;
            convert(pair_of, up);
            // the values: rows that are not finite, of tokens that some rows of the tile do not see
            const int t = x.j * kKeys + 32 * w + lane;
            const unsigned odd = __ballot_sync(0xffffffffu, t > x.s.pos0 && t < x.s.kend && odd_row(vmine));
            if (v == 0 && odd) {
                const int slot = slot_of(p, look_up(p, x.s.b, x.s.kend, t));
                note_rows<D, KV>(p.v, (size_t)max(slot, 0) * p.Hkv + x.s.h, vmine, odd,
                                 x.j * kKeys + 32 * w - BadValues::base(x.s), x.s.k, bad);
                if (odd >> lane & 1) vmine = 0u;       // zeros
            }
            pair_of = vmine;
            up = pow2(max(4 - ev, -126));
        }
        if (!ok) break;
        ++blk;
        x.next();
    }
    if (!ok && !ctl.abort) set_timeout(p.err, &ctl.abort);
}

// ---------------------------------------------------------------------------
// Queries: three warps
//
// A wide tile's rows take both of the query tiles, the rows of narrow ones in turn
// the first and the second, so that the next is loaded beside a narrow segment.
// Only warps' rows (32) that hold some are filled. The first segment's come by the
// softmax's eight warps, which have nothing else to do then.
// ---------------------------------------------------------------------------

// Segment k's half of the queries, and whether it may be loaded: the last segment but
// one, where both are narrow, or the last one has no products to come. Both barriers
// are one phase ahead of what is asked for at most: the next segment of their parity
// is loaded only after this one.
__device__ __forceinline__ int q_half(int k, bool narrow) { return narrow ? k & 1 : 0; }
struct QueryTurn {
    int k;
    bool narrow, was;        // segment k, segment k - 1
    __device__ __forceinline__ bool free_at_start() const { return k < (narrow && was ? 2 : 1); }
    __device__ __forceinline__ uint64_t* bar(Ctl& ctl) const { return &ctl.q_free[narrow && was ? k & 1 : (k - 1) & 1]; }
    __device__ __forceinline__ unsigned parity() const { return (narrow && was ? (k >> 1) - 1 : (k - 1) >> 1) & 1; }
};
__device__ __forceinline__ int rows_filled(int rows) { return (rows + 31) & ~31; }

// A segment's queries into tile `to` (and the next) by asynchronous copies, warp w's
// share of kWarps.
template <int D, int kWarps>
__device__ __forceinline__ void copy_q(const ChunkParams& p, const Seg& s, uint32_t to, int w, uint64_t* full) {
    constexpr int CPR = D / 8, RPI = 32 / CPR;
    const int lane = threadIdx.x & 31;
    const int c = lane % CPR, rl = lane / CPR;
    const int inv = (65536 + p.G - 1) / p.G;      // r / G = r inv >> 16 for r < 256
    const int rows = s.ntok * p.G;
#pragma unroll 2
    for (int r0 = RPI * w; r0 < rows_filled(rows); r0 += kWarps * RPI) {
        const int r = r0 + rl;
        const int t = (r * inv) >> 16;
        const bool live = r < rows;
        const bf16* g = p.q + (size_t)(s.row0 + (live ? t : 0)) * p.q_stride +
                        (s.h * p.G + (live ? r - t * p.G : 0)) * D + 8 * c;
        cp16z(to + (r >> 7) * tile_bytes<D>() + tile_off(r & 127, c), g, live ? 16u : 0u);
    }
    cp_async_arrive(full);
}

// The segments after the first.
struct QueryTurns {
    Walk walk;
    Seg s;
    QueryTurn turn;
    bool more;
    __device__ __forceinline__ QueryTurns(const ChunkParams& p, const Ctl& ctl) : walk(p, ctl) {
        turn = {-1, false, false};
        next();
        if (more) next();
    }
    __device__ __forceinline__ void next() {
        more = walk.next(s);
        ++turn.k;
        turn.was = turn.narrow;
        turn.narrow = s.ntok * walk.p.G <= kStreamRows;
    }
    template <int D>
    __device__ __forceinline__ void copy(const ChunkParams& p, Ctl& ctl, uint32_t q) {
        copy_q<D, kFeeders>(p, s, q + q_half(turn.k, turn.narrow) * tile_bytes<D>(), (threadIdx.x >> 5) - 13,
                            &ctl.q_full[turn.k & 1]);
        next();
    }
};
// Waits for segment k's queries.
__device__ __forceinline__ bool wait_q(Ctl& ctl, int k) {
    return k == 0 ? wait_bar(&ctl.q_first, 0, &ctl.abort) : wait_bar(&ctl.q_full[k & 1], ((k - 1) >> 1) & 1, &ctl.abort);
}

template <int D>
__device__ void load_q(const ChunkParams& p, Ctl& ctl, uint32_t q) {
    QueryTurns next(p, ctl);
    while (next.more) {
        const QueryTurn& turn = next.turn;
        if (!turn.free_at_start() && !wait_bar(turn.bar(ctl), turn.parity(), &ctl.abort)) {
            if (!ctl.abort) set_timeout(p.err, &ctl.abort);
            break;
        }
        next.copy<D>(p, ctl, q);
    }
    cp_async_wait_all();
}

// INT8 and 4-bit caches: the thread's row r of a query tile in place as FP16 times a
// power of two that brings its largest |q| to 16 at most; returns what the row is in
// units of. The softmax does this, a row per thread, before it writes the last
// segment's results: the warps that load queries took 16000 clocks for a wide tile's.
template <int D>
__device__ __noinline__ float q_to_f16(unsigned char* tile, int r) {
    uint4 v[D / 8];
    unsigned top = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        v[c] = *reinterpret_cast<const uint4*>(tile + tile_off(r, c));
        const unsigned m = __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                                    __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu));
        top = __vmaxu2(top, m);
    }
    top = max(top >> 16, top & 0xFFFFu);
    if (top >= 0x7F80u) {                // infinities and NaN do not count
        top = 0;
#pragma unroll 1
        for (int i = 0; i < D; ++i) {
            const unsigned h = *reinterpret_cast<const uint16_t*>(tile + tile_off(r, i >> 3) + 2 * (i & 7)) & 0x7FFFu;
            if (h < 0x7F80u) top = max(top, h);
        }
    }
    const int e = top ? max((int)(top >> 7) - 126, -100) : 0;
    const float up = pow2(min(4 - e, 127));
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        float x[8];
        unpack8(make_int4(v[c].x, v[c].y, v[c].z, v[c].w), x);
        *reinterpret_cast<uint4*>(tile + tile_off(r, c)) =
            make_uint4(f16x2_of(x[0] * up, x[1] * up), f16x2_of(x[2] * up, x[3] * up),
                       f16x2_of(x[4] * up, x[5] * up), f16x2_of(x[6] * up, x[7] * up));
    }
    return pow2(e - 4);
}

// What comes from outside, INT8 and 4-bit caches: codes and pairs by asynchronous
// copies into their rings, keys then values of block after block, and a tile's
// queries as soon as the last tile's are used, whichever can go on (a wait for one
// of them alone could wait for itself). Each of the three warps takes a third of a
// block's rows. By the warps that convert, the copies took 1400 clocks of a block's
// 5000 there.
template <int D, int KV>
__device__ void feed_codes(const ChunkParams& p, Ctl& ctl, CodesCtl& cc, uint32_t q, unsigned char* raw,
                           uint2* pairs) {
    using R = Raw<D, KV>;
    constexpr int RPI = R::RPI, NG = kKeys / RPI;         // groups of rows of one copy instruction
    constexpr int N = (NG + kFeeders - 1) / kFeeders;
    static_assert(N * RPI <= 64, "a lane holds two slots");
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 13;
    const int rl = lane / R::LPR, g0 = NG * w / kFeeders, n = NG * (w + 1) / kFeeders - g0;
    const int row0 = g0 * RPI, rows = n * RPI;
    const unsigned slot_bytes = (unsigned)p.Hkv * R::RB;

    Blocks in(p, ctl);
    Look look[2];
    auto look_ahead = [&]() {            // the next block's tokens
#pragma unroll
        for (int i = 0; i < 2; ++i)
            look[i] = look_up(p, in.s.b, in.live && lane + 32 * i < rows ? in.s.kend : 0,
                              in.j * kKeys + row0 + 32 * i + lane);
    };
    int slot[2] = {-1, -1}, h = 0;
    bool live = in.live;
    auto step = [&]() {                  // its slots
        live = in.live;
        if (!live) return;
        slot[0] = slot_of(p, look[0]);
        slot[1] = slot_of(p, look[1]);
        h = in.s.h;
        in.next();
    };
    if (live) {
        look_ahead();
        step();
    }
    QueryTurns queries(p, ctl);
    const QueryTurn& turn = queries.turn;
    unsigned cnt = 0;
    long long t0 = clock64();
    while (live || queries.more) {
        bool moved = false;
        if (live && (cnt < R::kTiles ||
                     __all_sync(0xffffffffu, mbar_wait_shortly(&cc.empty[cnt % R::kTiles], (cnt / R::kTiles - 1) & 1)))) {
            const bool values = cnt & 1;
            const unsigned char* codes = static_cast<const unsigned char*>(values ? p.v : p.k) + h * R::RB +
                                         16 * (lane % R::LPR);
            const uint32_t dst = smem_u32(raw) + (cnt % R::kTiles) * (kKeys * R::RB) + 16 * lane;
            if (!values) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (lane + 32 * i >= rows) continue;
                    const uint32_t to = smem_u32(pairs + (cnt / 2 % kPairRing) * kKeys + row0 + 32 * i + lane);
                    const size_t at = (size_t)max(slot[i], 0) * p.Hkv + h;
                    cp4z(to, static_cast<const uint32_t*>(p.k_scale) + at, slot[i] >= 0 ? 4u : 0u);
                    cp4z(to + 4, static_cast<const uint32_t*>(p.v_scale) + at, slot[i] >= 0 ? 4u : 0u);
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int sl = __shfl_sync(0xffffffffu, slot[i * RPI / 32], (i * RPI + rl) & 31);
                const int g = g0 + i;
                if (i < n)
                    cp16z(dst + 2048 * (g % R::NI) + 512 * (g / R::NI), codes + (size_t)max(sl, 0) * slot_bytes,
                          sl >= 0 ? 16u : 0u);
            }
            cp_async_arrive(&cc.full[cnt % R::kTiles]);
            if (values) step();
            else look_ahead();
            ++cnt;
            moved = true;
        }
        if (queries.more && (turn.free_at_start() || __all_sync(0xffffffffu, mbar_test(turn.bar(ctl), turn.parity())))) {
            queries.copy<D>(p, ctl, q);
            moved = true;
        }
        if (moved) {
            t0 = clock64();
            continue;
        }
        if (!live) __nanosleep(100);
        if (__any_sync(0xffffffffu, ctl.abort || clock64() - t0 > 4000000000ll)) {
            if (!ctl.abort) set_timeout(p.err, &ctl.abort);
            break;
        }
    }
    cp_async_wait_all();
}

// ---------------------------------------------------------------------------
// Matrix products: one warp, of which one thread issues them
//
// Scores of a block overwrite the weights of the stream's block before, which
// the product issued just before reads. Nothing but the order of issue is between the
// two: this assumes that the products of one thread go through the SM's tensor pipe
// in that order. What the PTX ISA promises of it is about products of the same
// accumulator and shape; here the accumulators differ (O and S), and for D = 64 the
// shapes, too (N = 64 and 128). It has held in every run; a wait for the product with V
// before each S instead costs 2 to 7 % (a prompt of 16384 1933 -> 2019 us, 16 mixed
// requests, INT8, 214 -> 226, 4 prompts of 512 35.4 -> 36.2). A commit covers all products
// before it, so that of a block's scores tells the softmax that the product with
// V before them is done, too.
// True in one thread of the (converged) warp. Under this predicate the compiler
// knows that a single thread is active, and hands the products' descriptors to
// the uniform registers that the instruction takes.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
                 : "=r"(r));
    return r != 0;
}

template <int D, int KV>
__device__ void issue_mma(const ChunkParams& p, Ctl& ctl, uint32_t q, uint32_t kv, BadValues bad) {
    constexpr int kSt = num_stages<D, KV>();
    constexpr bool kBf = KV == kKvBf16;
    constexpr uint32_t kIdS = idesc_chunk(kBf, kKeys, false), kIdO = idesc_chunk(kBf, D, true);
    const uint32_t tmem = ctl.tmem, id_s = kIdS | (p.negate ? kNegateA : 0u);   // a negative scale
    unsigned cnt = 0;                       // tiles of the ring before this segment
    unsigned np[2] = {0, 0};                // blocks of weights waited for, per stream
    bool ok = true;

    auto wait_full = [&](unsigned t) {
        if (!wait_bar(&ctl.kv_full[t % kSt], (t / kSt) & 1, &ctl.abort)) return false;
        fence_async_shared();
        return true;
    };
    // S of stream st from query tile buf and ring tile t
    auto qk = [&](int st, int buf, unsigned t, bool free, uint64_t* q_last) {
        const uint64_t a = sw128_kmajor_desc(q + buf * tile_bytes<D>());
        const uint64_t b = sw128_kmajor_desc(kv + (t % kSt) * tile_bytes<D>());
        if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t o = (uint64_t)((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
                mma_f16(tmem + 128 * st, a + o, b + o, id_s, k > 0);
            }
            mma_commit(&ctl.s_full[st]);
            if (free) mma_commit(&ctl.kv_empty[t % kSt]);
            if (q_last) mma_commit(q_last);
        }
        __syncwarp();
    };
    // O of stream st from its weights and ring tile t
    auto pv = [&](int st, unsigned t, bool add, bool free, bool done) {
        const uint64_t b = sw128_mnmajor_desc(kv + (t % kSt) * tile_bytes<D>(), kKeys * 128);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            if (!wait_bar(&ctl.p_full[st][part], np[st] & 1, &ctl.abort)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 4 * part; k < 4 * part + 4; ++k)
                    mma_f16_ta(tmem + kColO + D * st, tmem + 128 * st + kHalf * (k >> 2) + 8 * (k & 3),
                               b + (uint64_t)(k * 2048 >> 4), kIdO, add || k > 0);
                if (part == 0) mma_commit(&ctl.pv_half[st]);
                if (part == 1) {
                    if (free) mma_commit(&ctl.kv_empty[t % kSt]);
                    if (done) mma_commit(&ctl.pv_done[st]);
                }
            }
            __syncwarp();
        }
        ++np[st];
        return true;
    };

    Walk walk(p, ctl);
    Seg s;
    for (int k = 0; ok && walk.next(s); ++k) {
        const int nb = s.blocks();
        const bool narrow = s.ntok * p.G <= kStreamRows;
        uint64_t* const q_free = &ctl.q_free[k & 1];
        ok = (kBf ? wait_q(ctl, k)
                  : wait_bar(&ctl.q_ready[k & 1], (k >> 1) & 1, &ctl.abort)) && wait_full(cnt);
        if (!ok) break;
        // the segment before has left the tensor memory (and the notes on its values)
        auto free_o = [&]() {
            if (k == 0) return true;
            if (!wait_bar(&ctl.o_free, (k - 1) & 1, &ctl.abort)) return false;
            bad.clear(k - 1, D);
            return true;
        };
        if (!narrow) {
            qk(0, 0, cnt, false, nullptr);
            qk(1, 1, cnt, true, nb == 1 ? q_free : nullptr);
            ok = free_o();
            for (int j = 0; ok && j < nb; ++j) {
                const unsigned tv = cnt + 2 * j + 1, tk = tv + 1;
                const bool more = j + 1 < nb;
                ok = wait_full(tv) && (!more || wait_full(tk)) && pv(0, tv, j > 0, false, !more);
                if (ok && more) qk(0, 0, tk, false, nullptr);
                ok = ok && pv(1, tv, j > 0, true, !more);
                if (ok && more) qk(1, 1, tk, true, j + 2 == nb ? q_free : nullptr);
            }
        } else {
            // block j goes to stream j % 2. Block 1's keys come behind the look over block 0's
            // values, which waits for the last segment's notes to be cleared: where there are
            // any (they are complete, with that segment's last values), that comes first.
            const int m = min(2, nb), at = k > 0 && nb > 1 && bad.any(k - 1) ? 1 : m;
            for (int j = 0; ok && j <= m; ++j) {
                if (j == at) ok = free_o();
                if (j == m || !(ok = ok && wait_full(cnt + 2 * j))) break;
                qk(j, q_half(k, true), cnt + 2 * j, true, j + 1 == nb ? q_free : nullptr);
            }
            for (int j = 0; ok && j < nb; ++j) {
                const unsigned tv = cnt + 2 * j + 1, tk = tv + 3;
                const bool more = j + 2 < nb;
                ok = wait_full(tv) && pv(j & 1, tv, j >= 2, true, !more) && (!more || wait_full(tk));
                if (ok && more) qk(j & 1, q_half(k, true), tk, true, j + 3 == nb ? q_free : nullptr);
            }
        }
        cnt += 2 * nb;
    }
    if (!ok && !ctl.abort) set_timeout(p.err, &ctl.abort);
    // no product may still run when the tensor memory is given back
    if (elect_one()) mma_commit(&ctl.done);
    __syncwarp();
    wait_bar(&ctl.done, 0, &ctl.never);
}

// ---------------------------------------------------------------------------
// Softmax and results: a row per thread, four warps per stream
// ---------------------------------------------------------------------------

// 32 columns of the warp's 32 rows, a row per lane, times the rows' inv, as BF16
// to the rows' addresses (null: none). Four lanes exchange their rows' four
// 16-byte pieces first, so that a store covers 64 bytes of eight rows; of the
// lanes' own rows it wrote half sectors.
__device__ __forceinline__ void store32(bf16* out, const float (&o)[32], float inv) {
    const int lane = threadIdx.x & 31;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i].x = bf16x2_of(o[8 * i] * inv, o[8 * i + 1] * inv);
        v[i].y = bf16x2_of(o[8 * i + 2] * inv, o[8 * i + 3] * inv);
        v[i].z = bf16x2_of(o[8 * i + 4] * inv, o[8 * i + 5] * inv);
        v[i].w = bf16x2_of(o[8 * i + 6] * inv, o[8 * i + 7] * inv);
    }
    auto swap = [&](uint4& a, uint4& b, int bit) {
        // lanes with the bit give a and keep b, the others give b and keep a
        const bool up = lane & bit;
        uint4 give = up ? a : b;
        give.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
        give.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
        give.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
        give.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
        if (up) a = give;
        else b = give;
    };
    swap(v[0], v[1], 1);
    swap(v[2], v[3], 1);
    swap(v[0], v[2], 2);
    swap(v[1], v[3], 2);
    const unsigned long long mine = reinterpret_cast<unsigned long long>(out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // v[i]: piece lane % 4 of row 4 (lane / 4) + i
        const unsigned long long to = __shfl_sync(0xffffffffu, mine, (lane & ~3) + i);
        if (to) reinterpret_cast<uint4*>(to)[lane & 3] = v[i];
    }
}

// LONG: both halves of a block in the code, not a loop of them (see launch).
template <int D, int KV, bool LONG>
__device__ void softmax(const ChunkParams& p, Ctl& ctl, unsigned char* q, float2* stat, const float2* fac,
                        float* q_unit, BadValues bad) {
    constexpr bool kBf = KV == kKvBf16;
    constexpr float kUp = kBf ? 0.0f : 7.0f;   // weights are 2^(x - ref + kUp)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int st = warp >> 2;                   // stream
    const int lr = 32 * (warp & 3) + lane;      // lane of the tensor memory
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = ctl.tmem + lanes + 128 * st, to = ctl.tmem + lanes + kColO;
    const int inv_g = (65536 + p.G - 1) / p.G;
    const PartView parts = {p.part, D, p.part_rows};
    unsigned ns = 0, nm = 0, nv[2] = {0, 0};    // blocks of scores, merges, tiles of either stream
    unsigned blk = 0;                           // blocks before this segment
    bool ok = true;
    Walk walk(p, ctl);
    Seg s, next;
    bool more = walk.next(next);
    // segment k's queries, `next`
    auto prepare = [&](int k) {
        if (!(ok = wait_q(ctl, k))) return;
        const int rows = next.ntok * p.G, row = rows <= kStreamRows ? lr : kStreamRows * st + lr;
        // (of a narrow tile, the rows are its half's stream's)
        if (row - lane < rows && (rows > kStreamRows || q_half(k, true) == st)) {
            q_unit[(k & 3) * kTileRows + row] = q_to_f16<D>(q + st * tile_bytes<D>(), lr);
            fence_async_shared();
        }
        __syncwarp();
        // (two barriers: a stream without a block is ahead of the other by one segment at most)
        if (lane == 0) mbar_arrive(&ctl.q_ready[k & 1]);
    };
    if (more) copy_q<D, 8>(p, next, smem_u32(q), warp, &ctl.q_first);
    if (!kBf && more) prepare(0);
    for (int k = 0; ok && more; ++k) {
        s = next;
        const int nb = s.blocks();
        const int rows = s.ntok * p.G;
        const bool narrow = rows <= kStreamRows;
        const int row = narrow ? lr : kStreamRows * st + lr;
        const int tok = (row * inv_g) >> 16;
        const bool live = row < rows;
        const int limit = live ? s.pos0 + tok : -1;        // last key that the row sees
        float ref = -INFINITY, sum = 0.0f;
        float f = p.scale_log2, row_scale = f;     // a block's scores to units of log2
        int unit = 0;                              // O is in units of 2^unit
        const int step = narrow ? 2 : 1;
        const int mine = narrow ? (nb + 1 - st) / 2 : nb;  // blocks of this stream
        // A warp without a row of the tile has nothing to weigh: what its lanes of P hold
        // reaches no other row. It leaves its issue slots to the others (64 requests of 4
        // drafts, 20 rows a tile: 187 -> 180 us).
        const bool idle = row - lane >= rows;
        for (int j = 0; j < mine; ++j) {
            const int key0 = (s.j0 + (narrow ? st : 0) + j * step) * kKeys;
            ok = wait_bar(&ctl.s_full[st], ns & 1, &ctl.abort);
            if (!ok) break;
            ++ns;
            if (idle) {
                if (lane == 0) {
                    mbar_arrive(&ctl.p_full[st][0]);
                    mbar_arrive(&ctl.p_full[st][1]);
                }
                __syncwarp();
                continue;
            }
            tc_fence_after();
            int v_unit = 0;
            if (!kBf) {
                const float2 e = fac[(blk + (narrow ? st : 0) + j * step) % kFacRing];
                if (j == 0) row_scale *= q_unit[(k & 3) * kTileRows + row];
                f = fmaxf(row_scale * e.x, 1e-37f);      // (as the launcher's, see there)
                v_unit = __float_as_int(e.y);
                if (j == 0) unit = v_unit;
            }
#pragma unroll (LONG ? 2 : 1)
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t v[kHalf], w[kHalf / 2];
                tmem_ld64(ts + kHalf * hf, v);
                if (key0 + kHalf * hf + kHalf - 1 > s.pos0) {
                    const int lim = limit - key0 - kHalf * hf;
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) v[c] = c > lim ? 0xFF800000u : v[c];
                }
                float top, part;
                for (;;) {
                    const float base = kUp - (ref == -INFINITY ? 0.0f : ref);
                    const f32x2 f2v = pair(f, f), b2v = pair(base, base);
                    f32x2 acc[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
                    float mx[2] = {__uint_as_float(v[0]), __uint_as_float(v[1])};
#pragma unroll
                    for (int c = 0; c < kHalf / 2; ++c) {
                        const float x0 = __uint_as_float(v[2 * c]), x1 = __uint_as_float(v[2 * c + 1]);
                        if (c) mx[c & 1] = fmaxf(mx[c & 1], fmaxf(x0, x1));
                        else mx[0] = fmaxf(x0, x1);
                        float a, b;
                        split(fma2(pair(x0, x1), f2v, b2v), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        acc[c & 1] = add2(acc[c & 1], pair(a, b));
                        w[c] = kBf ? bf16x2_of(a, b) : f16x2_of(a, b);
                    }
                    float s0, s1;
                    split(add2(acc[0], acc[1]), s0, s1);
                    part = s0 + s1;
                    top = fmaxf(mx[0], mx[1]) * f;
                    const bool regrown = !kBf && hf == 0 && unit != v_unit;   // the same in all threads
                    if (!__any_sync(0xffffffffu, top > ref + kLazy) && !regrown) break;
                    const float up = fmaxf(ref, top);
                    const float a = ref == -INFINITY ? 0.0f : ex2(ref - up);
                    const float ao = kBf ? a : a * pow2(max(unit - v_unit, -126));   // v_unit only grows
                    unit = v_unit;
                    if (hf == 1 && !wait_bar(&ctl.pv_half[st], (ns - 1) & 1, &ctl.abort)) {
                        ok = false;
                        break;
                    }
                    if (j > 0 || hf == 1) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(to + D * st + c, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ao);
                            tmem_st32(to + D * st + c, o);
                        }
                    }
                    sum *= a;
                    ref = up;
                }
                sum += part;
                tmem_st32(ts + kHalf * hf, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[st][hf]);
            }
            if (!ok) break;
        }
        if (!ok) break;
        more = walk.next(next);
        if (!kBf && more) {
            prepare(k + 1);
            if (!ok) break;
        }

        // ---- results ----
        // A wide tile's stream holds its rows' O. Of a narrow tile both streams hold the same
        // rows, and each warp joins half of the columns: o u0 of one and o u1 of the other.
        const bool two = narrow && nb > 1;
        const bool none = limit < 0;
        float up = ref, all = sum, u0 = 1.0f, u1 = 0.0f;
        if (narrow) {
            // The segment before may be narrow, too, and its statistics still be read: a stream's
            // first scores do not wait for its results, so with one block a stream is here before
            // the other has left it.
            ok = k == 0 || wait_bar(&ctl.o_free, (k - 1) & 1, &ctl.abort);
            if (!ok) break;
            if (st == 0 || two) {
                stat[kStreamRows * st + lr] = make_float2(ref, sum);
                if (!idle) ctl.v_unit[st] = unit;  // (the same in all of these)
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.merge);
            ok = wait_bar(&ctl.merge, nm & 1, &ctl.abort);
            ++nm;
        }
        ok = ok && (narrow && st == 1 || wait_bar(&ctl.pv_done[st], nv[st] & 1, &ctl.abort));
        if (narrow) ok = ok && (st == 0 || wait_bar(&ctl.pv_done[0], nv[0] & 1, &ctl.abort)) &&
                         (!two || wait_bar(&ctl.pv_done[1], nv[1] & 1, &ctl.abort));
        ++nv[0];
        if (!narrow || two) ++nv[1];
        if (!ok) break;
        tc_fence_after();
        int first_col = 0, last_col = D;
        uint32_t o_col = to + D * st;
        if (narrow) {
            const float2 e0 = stat[lr], e1 = two ? stat[kStreamRows + lr] : make_float2(-INFINITY, 0.0f);
            up = fmaxf(e0.x, e1.x);
            u0 = e0.x == -INFINITY ? 0.0f : ex2(e0.x - up);
            u1 = e1.x == -INFINITY ? 0.0f : ex2(e1.x - up);
            all = e0.y * u0 + e1.y * u1;
            first_col = st * (D / 2);
            last_col = first_col + D / 2;
            o_col = to;
        }
        if (!kBf) {
            u0 *= pow2(narrow ? ctl.v_unit[0] : unit);
            if (two) u1 *= pow2(ctl.v_unit[1]);
        }
        const bool whole = s.head && s.tail;
        const float inv = none ? 0.0f : __fdividef(1.0f, all);
        bf16* const out = p.out + ((size_t)(s.row0 + (live ? tok : 0)) * p.Hq + s.h * p.G + (live ? row - tok * p.G : 0)) * D;
        float* const part = parts.slot(blockIdx.x, s.head);
#pragma unroll 1
        for (int c = first_col; c < last_col; c += 32) {
            uint32_t o[32];
            float x[32];
            tmem_ld32(o_col + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]) * u0;
            if (two) {
                tmem_ld32(o_col + D + c, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __fmaf_rn(__uint_as_float(o[i]), u1, x[i]);
            }
            if (whole) {
                store32(live ? out + c : nullptr, x, inv);
            } else if (live) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *parts.o(part, row, c / 4 + i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
        }
        if (!whole && live && (!narrow || st == 0)) *parts.stat(part, row) = make_float2(up, all);
        if (bad.any(s.k)) {                        // (noted before the products with V)
            __syncwarp();                          // the row's columns are written, by four lanes
            if (live) bad.add<D>(limit - BadValues::base(s), first_col, last_col, whole ? out : nullptr,
                                 reinterpret_cast<float*>(parts.o(part, row, 0)), 4 * parts.pad());
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.o_free);
        blk += nb;
    }
    if (!ok && !ctl.abort) set_timeout(p.err, &ctl.abort);
    cp_async_wait_all();
}

// ---------------------------------------------------------------------------

template <int D, int KV, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const ChunkParams p) {
    using Y = Lay<D, KV>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + Y::ctl);
    CodesCtl& cc = *reinterpret_cast<CodesCtl*>(smem + Y::codes);
    const int warp = threadIdx.x >> 5;
    const uint32_t q = smem_u32(smem + Y::q), kv = smem_u32(smem + Y::kv);
    if (threadIdx.x == 0) {
        for (int i = 0; i < Y::kSt; ++i) {
            mbar_init(&ctl.kv_full[i], 128);
            mbar_init(&ctl.kv_empty[i], 1);
        }
        for (int i = 0; i < raw_tiles<D, KV>(); ++i) {
            mbar_init(&cc.full[i], kFeeders * 32);
            mbar_init(&cc.empty[i], 4);
        }
        if (KV != kKvBf16) mbar_init(&cc.tops, 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.q_full[i], kFeeders * 32);
            mbar_init(&ctl.q_free[i], 1);
            mbar_init(&ctl.q_ready[i], 8);
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i][0], 4);
            mbar_init(&ctl.p_full[i][1], 4);
            mbar_init(&ctl.pv_half[i], 1);
            mbar_init(&ctl.pv_done[i], 1);
        }
        mbar_init(&ctl.q_first, 256);
        mbar_init(&ctl.o_free, 8);
        mbar_init(&ctl.merge, 8);
        mbar_init(&ctl.done, 1);
        ctl.abort = ctl.never = 0;
        ctl.bad_tile = -1;
        mbar_init_fence();
    }
    if (warp == 12) tmem_alloc(&ctl.tmem, kTmemCols);
    if (threadIdx.x < D) reinterpret_cast<uint32_t*>(smem + Y::bad)[threadIdx.x] = kNoBad;
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    find_part(p, ctl, smem + Y::stat);   // synchronises the CTA
    tc_fence_after();

    // Registers: a launch gives every thread 128; their sum over the four groups of
    // four warps stays 512.
    constexpr bool kBf = KV == kKvBf16;
    const BadValues bad = {reinterpret_cast<uint32_t*>(smem + Y::bad), ctl, p.err};
    float2* fac = reinterpret_cast<float2*>(smem + Y::fac);
    if (warp < 8) {
        set_max_regs_inc<152>();
        softmax<D, KV, LONG>(p, ctl, smem + Y::q, reinterpret_cast<float2*>(smem + Y::stat), fac,
                       reinterpret_cast<float*>(fac + kFacRing), bad);
    } else if (warp < 12) {
        set_max_regs_dec<104>();
        if constexpr (kBf) load_bf16<D>(p, ctl, kv, smem + Y::kv, bad);
        else convert_codes<D, KV>(p, ctl, cc, smem + Y::kv, smem + Y::raw, reinterpret_cast<uint2*>(smem + Y::pairs), fac, bad);
    } else {
        set_max_regs_dec<104>();
        if (warp == 12) issue_mma<D, KV>(p, ctl, q, kv, bad);
        else if constexpr (kBf) load_q<D>(p, ctl, q);
        else feed_codes<D, KV>(p, ctl, cc, q, smem + Y::raw, reinterpret_cast<uint2*>(smem + Y::pairs));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(ctl.tmem, kTmemCols);
}

// Second kernel: tiles that several parts hold. CTA c - 1 looks at part c's
// begin; of the k parts that begin inside one tile each joins a k-th of its
// rows. The rows' weights of all parts come first, into shared memory; then a
// thread adds up four columns of a row, eight threads side by side along it.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;                               // rows of a CTA, about
constexpr int kJoinWeights = 2 * (kTileRows + kMaxParts);   // (256 / k + 1) rows of k + 1 parts

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_chunk_join_kernel(const ChunkParams p) {
    __shared__ float s_w[kJoinWeights];
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x + 1;
    const int4* entry = reinterpret_cast<const int4*>(reinterpret_cast<const PlanEntry*>(p.ws) + c);
    const int4 e0 = __ldcg(entry), e1 = __ldcg(entry + 1);
    if (!e0.x) return;
    const int kf = e0.y, kl = e0.z, row0 = e0.w, rows = e1.x * p.G, pos0 = e1.y, h = e1.z;
    // of the tile's `share` parts this one takes a share of its rows, and of those
    // the CTAs along y shares again
    const int share = kl - kf + 1, n = share + 1;
    const int a0 = rows * (c - kf) / share, a1 = rows * (c - kf + 1) / share;
    const int r0 = a0 + (a1 - a0) * (int)blockIdx.y / (int)gridDim.y;
    const int r1 = a0 + (a1 - a0) * ((int)blockIdx.y + 1) / (int)gridDim.y;
    const PartView parts = {p.part, D, p.part_rows};
    auto slot_of_part = [&](int k) { return parts.slot(kf - 1 + k, k == 0); };
    for (int row = r0 + (int)threadIdx.x; row < r1; row += kJoinThreads) {
        float up = -INFINITY, sum = 0.0f;
        for (int k = 0; k < n; ++k) up = fmaxf(up, __ldcg(parts.stat(slot_of_part(k), row)).x);
        float* w = s_w + (row - r0) * n;
        for (int k = 0; k < n; ++k) {
            const float2 e = __ldcg(parts.stat(slot_of_part(k), row));
            // a part that saw nothing (or whose scores are all minus infinity) counts with its sum
            const float a = e.x == up ? 1.0f : ex2(e.x - up);
            sum = __fmaf_rn(e.y, a, sum);
            w[k] = a;
        }
        const float inv = pos0 + row / p.G < 0 ? 0.0f : __fdividef(1.0f, sum);
        for (int k = 0; k < n; ++k) w[k] *= inv;
    }
    __syncthreads();
    constexpr int C = D / 4;
    for (int at = threadIdx.x; at < (r1 - r0 + 3) / 4 * 4 * C; at += kJoinThreads) {
        // eight column groups of four rows per warp
        const int unit = at >> 5, l = at & 31;
        const int row = r0 + unit / (C / 8) * 4 + (l >> 3), cg = unit % (C / 8) * 8 + (l & 7);
        if (row >= r1) continue;
        const float* w = s_w + (row - r0) * n;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float4 v = __ldcg(parts.o(slot_of_part(k), row, cg));
            o.x = __fmaf_rn(v.x, w[k], o.x);
            o.y = __fmaf_rn(v.y, w[k], o.y);
            o.z = __fmaf_rn(v.z, w[k], o.z);
            o.w = __fmaf_rn(v.w, w[k], o.w);
        }
        const int t = row / p.G;
        bf16* out = p.out + ((size_t)(row0 + t) * p.Hq + h * p.G + row - t * p.G) * D;
        reinterpret_cast<uint2*>(out)[cg] = make_uint2(bf16x2_of(o.x, o.y), bf16x2_of(o.z, o.w));
    }
}

template <int D, int KV, bool LONG>
cudaError_t launch(const ChunkParams& p, int grid, const Launch& L) {
    auto kern = attn_chunk_kernel<D, KV, LONG>;
    constexpr size_t bytes = Lay<D, KV>::total;
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = once_per_context(reinterpret_cast<const void*>(kern), [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, kern, p)) != cudaSuccess) return e;
    // (no second launch for tables of up to 256 keys: 5 tokens past 32, 9.2 -> 8.2 us; with a
    // wider table they keep it, as the host does not know the contexts)
    if (grid == 1 || !may_divide(blocks_of(p.max_blocks * p.page))) return cudaSuccess;
    cfg.gridDim = dim3(grid - 1, (p.part_rows + kJoinRows - 1) / kJoinRows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_chunk_join_kernel<D>, p);
}

int part_rows(int T, int G) { return std::min(T, tile_tokens(G)) * G; }

// Parts that a call of these sizes can have at most.
int max_parts(int T, int B, int G, int Hkv, int max_ctx) {
    const long units = (long)Hkv * (T / tile_tokens(G) + B) * (kWideCost + (long)blocks_of(max_ctx));
    return (int)std::min<long>(kMaxParts, (units + kMinUnits - 1) / kMinUnits);
}

// Over a BF16 cache, requests of half a wide tile and more on average with a table for so
// many blocks of keys and more take the longer code of the softmax: a prompt of 16384 1969 -> 1912 us,
// 512 tokens at 16384 150 -> 147, a prompt of 8192 with heads of 64 386 -> 362, 8 requests
// of 256 to 1024 tokens past 1000 to 6000 276 -> 271. Shorter ones lose by it, as their CTAs
// spend much of their time on code that no cache holds yet: 4 prompts of 512 33 -> 36, 16
// requests of 1 to 256 tokens past 100 to 4000 103 -> 106; and single tokens: 64 past 1000
// to 8000 193 -> 195. The table's width stands for the contexts, which only the device knows:
// 4 prompts of 512 with a table for 16384 keys take 37.5 instead of 33.5.
constexpr int kLongBlocks = 48;

template <int D>
cudaError_t launch_kind(const ChunkParams& p, int grid, const Launch& L) {
    if (p.kv == kKvI8) return launch<D, kKvI8, false>(p, grid, L);
    if (p.kv == kKvI4) return launch<D, kKvI4, false>(p, grid, L);
    const bool is_long = blocks_of(p.max_blocks * p.page) >= kLongBlocks && p.T >= (long)p.B * (tile_tokens(p.G) / 2);
    return is_long ? launch<D, kKvBf16, true>(p, grid, L) : launch<D, kKvBf16, false>(p, grid, L);
}

}  // namespace

size_t attn_chunk_workspace_bytes(int T, int B, int Hq, int Hkv, int D, int max_ctx) {
    const int G = Hq / Hkv, parts = max_parts(T, B, G, Hkv, max_ctx);
    return plan_bytes() + (parts > 1 ? (size_t)parts * 2 * PartView::floats(D, part_rows(T, G)) * 4 : 0);
}

cudaError_t launch_attention_chunk(ChunkParams p, const Launch& L) {
    if (p.T <= 0 || p.B <= 0) return cudaSuccess;
    p.G = p.Hq / p.Hkv;
    p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(p.ws) + plan_bytes());
    p.part_rows = part_rows(p.T, p.G);
    const int grid = std::min(L.num_sms, max_parts(p.T, p.B, p.G, p.Hkv, p.max_blocks * p.page));
    // scores in units of log2; a scale of 0 stands as the smallest that leaves
    // masked scores at minus infinity
    p.negate = p.scale_log2 < 0.0f;
    if (p.negate) p.scale_log2 = -p.scale_log2;
    if (p.scale_log2 < 1e-37f) p.scale_log2 = 1e-37f;
    if (p.D == 128) return launch_kind<128>(p, grid, L);
    if (p.D == 64) return launch_kind<64>(p, grid, L);
    return cudaErrorInvalidValue;
}

}  // namespace a8w8
