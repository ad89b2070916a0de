// attn_i4.cu -- GQA decode attention over the 4-bit paged KV cache.
//
// A row (one KV head's D values of one token) stands for c s + m (kv_i4.cu), so
// for a query head q with scores in units of log2:
//   y_t = scale log2(e) (s_t sum_d q_d c_td + m_t sum_d q_d),
//   out = (sum_t p_t s_t c_t + sum_t p_t m_t) / sum_t p_t,  p_t = 2^(y_t - ref):
// both sums over codes are products of a real vector with small integers, and
// everything else is one number per (token, head).
//
// What bounds it: D + 8 bytes per (token, KV head) from HBM. At the measured
// copy rate an SM receives 32 tokens' rows (4.4 KB at D = 128) in about 190
// cycles, in which it issues at most 760 warp instructions, 380 of them on the
// integer pipe, for 8192 codes. So the two products run on the tensor cores
// (mma.sync m16n8k16 f16, 600 TFLOP/s here: 64 of the 190 cycles) and codes
// become operands without a conversion: an integer 0..15 in the lowest
// mantissa bits of an FP16 is the subnormal c 2^-24, in the next four bits c
// 2^-20, a whole byte c + 16 c' likewise, all exact, so a word of eight codes
// is four operand registers after four or five integer instructions.
// (mma.sync on e4m3 bytes, where a nibble is exact too, compiles to
// conversions and f16 instructions on sm_103a: 1131 instructions per tile of
// 32 tokens, 400 here.) The powers of two are taken back in the other operand
// or the result:
//   * q, scaled per head by a power of two to a maximum in [2^10, 2^11) (times
//     16 beside the low nibbles). FP16's last bit is 2^-24, so the eight
//     significant bits of a BF16 are exact from 2^-17 up, 2^-27 of the head's
//     largest |q|; a smaller value is off by at most 2^-25, 2^-35 of it. Tokens
//     are the rows, query heads the columns, so a group of up to 8 heads costs
//     one instruction per 16 tokens and 16 dimensions.
//   * the weights p_t s_t, rounded to FP16: 2^-11 relative, beside the 2^-8 of
//     the BF16 result. ref keeps the largest between 2^10 and 2^15, so that
//     what FP16 cannot hold lies 2^-34 below it. One 8 x 8 transpose
//     (movmatrix) per 8 tokens takes them from the score's layout into the
//     operand's.
// For V the contraction runs over tokens: a lane reads four tokens' bytes for
// its 16 dimensions per 16 tokens and pairs the halves of two words by one
// permute each; of a pair of dimensions it sums the low nibbles and the whole
// bytes, whose difference is 16 times the high nibbles' sum.
//
// Work is cut into tiles of 32 tokens of a request, numbered through all
// requests. A run is an equal share of the tiles, whatever the contexts; it
// is taken by the CTAs of all KV heads, a warp per head and four heads to a
// CTA where their number allows it, so that the rows of one token, which lie
// side by side, are read together (heads one after the other: 27 % more bytes
// from HBM, and 206 us against 140 for 64 requests of up to 16384 tokens). A
// warp copies its tiles with cp.async into a private ring, without a barrier.
// Runs that end inside a request leave (ref, sum, o) to a second kernel.
// Three CTAs of four warps fill an SM at 168 registers; four at 128 were
// slower (117 against 114 us, spills), and so were deeper rings (3 or 4
// stages: 113, 117), more and shorter runs (117 at twice as many), the next
// tile's scores ahead of this one's weights (114), and barriers that keep an
// SM's CTAs in step (116 to 129).
//
// Measured (40 query and 8 KV heads of 128, pages of 128 tokens; calls through
// the binding one after the other): 64 requests of 64 to 16384 tokens, 574 MB,
// 106 us (5.4 TB/s, 0.81 of the copy rate); 16 requests of 64 to 4096 tokens,
// 37 MB, 18.5 us. As replayed graphs 108.7 and 18.7 us; there the same kernels
// without the arithmetic take 99.5 and 15.5, without the copies behind the
// first two tiles 86.1 and 18.5. So long calls are bound by their copies, and
// short ones by the chain from the run search to the second kernel; neither
// the integer pipe, 50 % busy, nor HBM, 70 %, is full with three warps per
// scheduler. One request of 256 tokens: 4.5 us a kernel in a row of them.
#include <limits.h>

#include <algorithm>

#include "kernels.cuh"

namespace a8w8 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 32;            // tokens a warp takes at a time
constexpr int kStages = 2;           // ring depth per warp
constexpr int kCtasPerSm = 3;
constexpr int kMaxCtas = 152 * kCtasPerSm;
constexpr int kMinTiles = 4;         // tiles per run at least
constexpr int kPiece = 512;          // tiles a warp adds up before it joins them to its part
constexpr int kCombineThreads = 128;
constexpr int kJoin = 2;             // parts a warp of the second kernel loads at once
constexpr float kNoRef = -3.4e38f;   // ref of a warp that has seen no token: below every score

constexpr int code_bytes(int D) { return kTile * D / 2; }
constexpr int stage_bytes(int D) { return 2 * code_bytes(D) + kTile * 8; }
constexpr int ring_bytes(int D) { return kWarps * kStages * stage_bytes(D); }
// Beside the rings, the warps' (o, ref, sum) of the segment that just ended:
// the next segment's first copies run while they are joined.
constexpr int smem_bytes(int D, int HW) {
    return ring_bytes(D) + (HW == kWarps ? 0 : kWarps * 8 * (D + 4) * 4 + 2 * kWarps * 8 * 4);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], unsigned a0, unsigned a1, unsigned a2,
                                        unsigned a3, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned h2_of(float a, float b) {   // a in the low half
    unsigned r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// 8 x 8 halves, row lane / 4, columns 2 (lane % 4) and the next: transposed.
__device__ __forceinline__ unsigned transpose8(unsigned v) {
    unsigned r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Sums taken at one ref go to another, d higher, by the factor 2^-d, applied as
// 2^(-d/2) twice: refs differ by up to 174 with the V rows' scales alone (2^124
// to the 2^-50 that tiny ones count), past 2^-126, while the sum of the lower
// ones' weights, up to 2^60 a token, weighs as much as the others'.
__device__ __forceinline__ float half_step(float d) { return ex2(0.5f * d); }
__device__ __forceinline__ void cp16(unsigned s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(g) : "memory");
}
__device__ __forceinline__ void cp4z(unsigned s, const void* g, unsigned n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(g), "r"(n) : "memory");
}
__device__ __forceinline__ float bf_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(unsigned w) { return __uint_as_float(w & 0xFFFF0000u); }

// Tokens of request b: none where the context is out of range. Contexts and
// tables are read by plain loads, which see what the kernels before this one
// wrote (the read-only path need not, as such a kernel may still run when this
// one starts), and mostly from L1: a table entry from L2 comes back behind the
// copies under way, 129 us against 109 for 64 long requests.
__device__ __forceinline__ int tokens_of(const AttnI4Params& p, int b) {
    const int c = p.ctx_lens[b];
    return c < 0 || c > p.max_blocks * p.page ? 0 : c;
}
__host__ __device__ __forceinline__ int tiles_of(int tokens) { return (tokens + kTile - 1) / kTile; }

// Exclusive sum of v over the CTA's threads (total in `total`); `s` is one
// unsigned per warp.
__device__ __forceinline__ unsigned cta_exclusive(unsigned v, unsigned* s, unsigned& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s[w];
        total += s[w];
    }
    return before + x - v;
}

// The runs: run r of E begins at tile floor(r T / E) of T = sum_b tiles(b),
// request after request. Its HG = Hkv / HW CTAs stand side by side (CTA r HG +
// k takes heads k HW to k HW + HW - 1), so that the sectors that hold several
// heads' (s, m) words and the lines that hold their codes are read together.
struct Runs {
    unsigned T, E, q, rem;   // T = q E + rem
    __device__ __forceinline__ Runs(unsigned tiles, unsigned runs) {
        T = tiles;
        E = min((tiles + kMinTiles - 1) / kMinTiles, runs);
        q = E ? T / E : 0;
        rem = T - q * E;
    }
    __device__ __forceinline__ unsigned start(unsigned r) const { return q * r + rem * r / E; }
    __device__ __forceinline__ unsigned owner(unsigned tile) const {
        return (unsigned)((((unsigned long long)tile + 1) * E - 1) / T);
    }
};

// The workspace: what the second kernel has to join for each request, then
// two parts per run and KV head, each G heads of o [D], ref and sum: part 0 of
// the run's first segment, part 1 of its last one, if that is another (those
// between are whole requests, which only pass their pieces through part 1).
//   plan.x = 2 (first run) + (0 if the request is that run's first segment,
//   1 if it follows others), plan.y = last run; the same run twice: nothing to
//   join; plan.x = -1: no tokens.
struct PartView {
    float* base;
    int D, G;
    __device__ __forceinline__ float* o(unsigned slot, int head) const {
        return base + ((size_t)slot * G + head) * (D + 4);
    }
};
__host__ __device__ inline size_t plan_bytes(int B) { return ((size_t)B * 8 + 255) / 256 * 256; }

// Adds a piece of a segment (o [D], ref, sum) to the part that holds the ones
// before it, or writes the result of all: by one warp, where several share the
// heads, and in a loop of its own. Within the CTA's join the same cost short
// calls 2 to 4 % (64 requests of 256 tokens: 10.5 against 10.2 us).
template <int D>
__device__ __forceinline__ void add_piece(float* part, const float* piece, bf16* out, int lane) {
    const float2 a = *reinterpret_cast<const float2*>(part + D);
    const float2 b = *reinterpret_cast<const float2*>(piece + D);
    const float up = fmaxf(a.x, b.x), f = half_step(a.x - up), q = half_step(b.x - up);
    const float L = __fmaf_rn(a.y * f, f, b.y * q * q);
    for (int d = lane; d < D; d += 32) {
        const float o = __fmaf_rn(part[d] * f, f, piece[d] * q * q);
        if (out) out[d] = f2bf(__fdividef(o, L));
        else part[d] = o;
    }
    __syncwarp();                               // every lane has read (ref, sum)
    if (lane == 0 && !out) {
        part[D] = up;
        part[D + 1] = L;
    }
    __syncwarp();
}

template <int D>
struct Frag {
    static constexpr int KW = D / 32;   // 32-bit words of K codes per lane and token
    static constexpr int VW = D / 64;   // words of V codes per lane and token
};

// One CTA's share: the tiles of its run (or, with `whole`, all tiles of one
// (request, KV head) per CTA).
template <int D, int HW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_i4_kernel(const AttnI4Params p, const unsigned page_inv, const bool whole) {
    constexpr int KW = Frag<D>::KW, VW = Frag<D>::VW;
    constexpr int RB = D / 2;                   // bytes of a row's codes
    constexpr int TW = kWarps / HW;             // warps that share a head
    static_assert(HW * TW == kWarps, "warps are heads x token shares");
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ unsigned s_scan[kWarps];
    __shared__ unsigned s_first;
    __shared__ int s_b, s_tokens;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv;
    const int hw = warp % HW, tw = warp / HW;
    const int HG = p.Hkv / HW;                  // CTAs of a run
    const unsigned sbase = (unsigned)__cvta_generic_to_shared(smem);
    const unsigned ring = sbase + warp * kStages * stage_bytes(D);
    const unsigned char* rings = smem + warp * kStages * stage_bytes(D);

    pdl_wait();
    pdl_trigger();

    // ---- where the run begins -------------------------------------------------
    int b, h, j, tokens;           // the run's first tile: request, KV head, tile of the request
    int left;                      // tiles of the run from there on
    unsigned r = 0;                // the run
    int2* plan = reinterpret_cast<int2*>(p.part);
    if (whole) {
        b = blockIdx.x / p.Hkv;
        h = blockIdx.x - b * p.Hkv;
        j = 0;
        tokens = tokens_of(p, b);
        if (threadIdx.x == 0 && h == 0) {
            const int c = p.ctx_lens[b];
            if (c < 0 || c > p.max_blocks * p.page) set_error(p.err, 0x4u);
        }
        if (tokens == 0) {
            bf16* out = p.out + ((size_t)b * p.Hq + (size_t)h * G) * D;
            for (int i = threadIdx.x; i < G * D; i += kThreads) out[i] = __float2bfloat16_rn(0.0f);
            return;
        }
        left = tiles_of(tokens);
    } else {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        unsigned mine = 0;
        int last = 0;                           // tokens of the thread's last request
        for (int i = b0; i < b1; ++i) {
            const int n = last = tokens_of(p, i);
            if (blockIdx.x == 0 && n == 0) {
                plan[i] = make_int2(-1, -1);
                if (p.ctx_lens[i] != 0) set_error(p.err, 0x4u);
            }
            mine += tiles_of(n);
        }
        unsigned T;
        const unsigned before = cta_exclusive(mine, s_scan, T);
        const Runs runs(T, gridDim.x / HG);
        r = blockIdx.x / HG;
        h = (blockIdx.x - r * HG) * HW + hw;
        if (r >= runs.E) return;
        const unsigned x0 = runs.start(r), x1 = runs.start(r + 1);
        if (mine > 0 && x0 >= before && x0 - before < mine) {
            unsigned at = before;
            int i = b0, n = last;
            if (per > 1)
                for (; n = tokens_of(p, i), x0 - at >= (unsigned)tiles_of(n); ++i) at += tiles_of(n);
            s_b = i;
            s_first = at;
            s_tokens = n;
        }
        __syncthreads();
        b = s_b;
        tokens = s_tokens;
        j = x0 - s_first;
        left = x1 - x0;
        // the requests that begin in this run: which runs hold their parts
        if (blockIdx.x == r * HG && threadIdx.x == 0) {
            int rest = left;
            for (int i = b, at = j; rest > 0; ++i, at = 0) {
                const int n = tiles_of(tokens_of(p, i));
                if (n == 0) continue;
                if (at == 0) {
                    const unsigned last = x1 - rest + n - 1;   // its last tile
                    plan[i] = make_int2(2 * r + (i == b ? 0 : 1),
                                        n <= rest ? r : runs.owner(last));
                }
                rest -= n - at;
            }
        }
    }

    // ---- lane constants -----------------------------------------------------
    // Column n = 2 u + e of an 8-token group holds token 2 u + (e ^ (u >> 1)):
    // with the rows' 16-byte chunks exchanged on bit 1 of the token (D = 128),
    // neither a lane's K rows nor the four lanes' V rows meet in a bank.
    const int krow = 2 * (g >> 1) + ((g & 1) ^ (g >> 2));
    const unsigned koff = D == 128 ? krow * RB + ((t ^ (krow & 2)) * 16) : krow * RB + t * 8;
    const int vrow0 = 2 * t + (t >> 1), vrow1 = vrow0 ^ 1;
    const unsigned vin = D == 128 ? (((g >> 1) ^ (vrow0 & 2)) * 16) + (g & 1) * 8 : g * 4;
    const unsigned voff0 = vrow0 * RB + vin, voff1 = vrow1 * RB + vin;
    constexpr int CPR = RB / 16;                // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;               // rows one copy instruction covers
    const int crow = lane / CPR, cchunk = lane % CPR;
    const unsigned coff = D == 128 ? crow * RB + ((cchunk ^ (crow & 2)) * 16) : crow * RB + cchunk * 16;
    // the column that token `lane` stands in, for the (s, m) words
    const int mcol = (lane & ~7) + (lane & 6) + ((lane & 1) ^ ((lane >> 2) & 1));

    const unsigned rstride = (unsigned)p.Hkv * RB, mstride = (unsigned)p.Hkv * 4;
    const unsigned char* kc = p.c.k_codes + h * RB + cchunk * 16;
    const unsigned char* vc = p.c.v_codes + h * RB + cchunk * 16;
    const unsigned char* km = reinterpret_cast<const unsigned char*>(p.c.k_meta) + h * 4;
    const unsigned char* vm = reinterpret_cast<const unsigned char*>(p.c.v_meta) + h * 4;

    // ---- a segment: the run's tiles of one request, in pieces -----------------
    // A float32 sum of n like terms may be off by n 2^-24: where runs are long,
    // a segment is summed in pieces of kPiece tiles a warp (2048 weights a lane)
    // that are joined in its part's place in the workspace. The longest run
    // taken, 2^27 tokens, has 8192 pieces: 2^-13 + 2^-11 in all, beside the 2^-8
    // of the result's rounding. (One chain a run, 2^30 equal weights: 0.43 %.)
    int n_all, j1;                              // the request's tiles; the piece's end
    const int32_t* table;
    int blk[kStages], in_page[kStages], nblk, nin = 0;
    // The page and the place in it of token `lane` of tile i, asked for one
    // tile before the copies that need it (and not looked at before them).
    auto lookup = [&](int i, int& blk, int& in_page) {
        const unsigned tok = (unsigned)i * kTile + lane;
        blk = INT_MIN;                       // past the context
        if (i < j1 && (int)tok < tokens) {
            unsigned q = __umulhi(tok, page_inv), r = tok - q * p.page;
            if (r >= (unsigned)p.page) {
                ++q;
                r -= p.page;
            }
            blk = table[q];
            in_page = (int)r;
        }
    };
    // Copies tile i into ring stage st. A token without a row (past the
    // context, or a bad page) gets s = m = 0 and the codes of row 0, which
    // count nothing then.
    auto fetch = [&](int i, int st, int blk, int in_page) {
        if (i < j1) {                        // warp-uniform
            const bool ok = (unsigned)blk < (unsigned)p.num_blocks;
            if (!ok && (i * kTile + lane < tokens)) set_error(p.err, 0x2u);
            const unsigned slot = ok ? (unsigned)(blk * p.page + in_page) : 0u;
            const unsigned base = ring + st * stage_bytes(D);
#pragma unroll
            for (int k = 0; k < kTile / RPI; ++k) {
                const unsigned sl = __shfl_sync(0xffffffffu, slot, k * RPI + crow);
                const unsigned d = base + k * RPI * RB + coff;
                cp16(d, kc + (size_t)sl * rstride);
                cp16(d + code_bytes(D), vc + (size_t)sl * rstride);
            }
            const unsigned d = base + 2 * code_bytes(D) + mcol * 8;
            cp4z(d, km + (size_t)slot * mstride, ok ? 4u : 0u);
            cp4z(d + 4, vm + (size_t)slot * mstride, ok ? 4u : 0u);
        }
        cp_async_commit();
    };
    auto open = [&] {
        n_all = tiles_of(tokens);
        j1 = min(min(n_all, j + left), j + kPiece * TW);
        table = p.block_table + (size_t)b * p.max_blocks;
#pragma unroll
        for (int s = 0; s < kStages; ++s) lookup(j + tw + s * TW, blk[s], in_page[s]);
    };
    int4 raw[KW];                           // the query head's values, as loaded
    // The first tile is copied ahead, the ring's others once the query heads
    // stand ready: every warp's first tile comes before any warp's second.
    auto copy_first = [&] {
        fetch(j + tw, 0, blk[0], in_page[0]);
        const bf16* q = p.q + ((size_t)b * p.Hq + (size_t)h * G + (g < G ? g : 0)) * D + t * (D / 4);
#pragma unroll
        for (int w = 0; w < KW; ++w) raw[w] = g < G ? ld_cg_v4(q + 8 * w) : make_int4(0, 0, 0, 0);
    };
    open();
    copy_first();
    bool first = true;                          // the run's first segment
    bool from0 = j == 0;                        // the segment begins with its request
    bool joins = false, again = false;          // not the segment's, the run's first piece
    for (;; again = true) {
        // ---- the query heads ------------------------------------------------------
        // head g's dimensions of chunk t: for word w, elements (0, 4) and (2, 6)
        // times 16 meet the low nibbles of the masks, (1, 5) and (3, 7) the high
        unsigned qb[KW][4];
        f32x2 ch, qs;                           // score factors of heads 2 t, 2 t + 1
        {
            float sum = 0.0f, top = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                float f[8];
                unpack8(raw[w], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum += f[e];
                    top = fmaxf(top, fabsf(f[e]));
                }
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            // 2^e takes the largest |q| into [2^10, 2^11) (16 2^e stays finite; the
            // smallest BF16, 2^-133, is a normal FP16 then)
            const int e = max(-107, min(123, 137 - (int)(__float_as_uint(top) >> 23)));
            const float up = __uint_as_float((unsigned)(127 + e) << 23);
            const float sc = p.scale * 1.4426950408889634f;
            float f = __uint_as_float((unsigned)(127 + 20 - e) << 23) * sc;
            // a NaN shows in the sum; from 2^118 on FP16 would overflow
            if (!(fabsf(sum) <= 3e38f) || top >= 0x1p118f) f = __uint_as_float(0x7FC00000u);
            sum *= sc;
            ch = pair(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
            qs = pair(__shfl_sync(0xffffffffu, sum, 8 * t), __shfl_sync(0xffffffffu, sum, 8 * t + 4));
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                float f[8];
                unpack8(raw[w], f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float m = k & 1 ? up : up * 16.0f;
                    qb[w][k] = h2_of(f[k] * m, f[4 + k] * m);
                }
            }
        }

        // times 2^-24, rows: sums of the low nibbles (dimension 2 i of the lane's) and
        // of the whole bytes c_2i + 16 c_2i+1; columns: heads 2 t, 2 t + 1
        float acc[4 * VW][4];
#pragma unroll
        for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
        // of heads 2 t, 2 t + 1, over the lane's tokens
        float ref0 = 0.0f, ref1 = 0.0f, l0 = 0.0f, l1 = 0.0f, om0 = 0.0f, om1 = 0.0f;
        bool fresh = true;                      // no tile yet

#pragma unroll
        for (int s = 1; s < kStages; ++s) fetch(j + tw + s * TW, s, blk[s], in_page[s]);
        lookup(j + tw + kStages * TW, nblk, nin);
        int st = 0;
        for (int i = j + tw; i < j1; i += TW) {
            cp_async_wait_group<kStages - 1>();
            __syncwarp();
            const unsigned char* base = rings + st * stage_bytes(D);

            // ---- scores: token g of each 8, heads 2 t and 2 t + 1 --------------------
            float y0[4], y1[4], sv[4], mv[4];   // y - ref
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                unsigned ka[2][KW];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if constexpr (D == 128) {
                        const int4 v = *reinterpret_cast<const int4*>(base + 8 * (k + r) * RB + koff);
                        ka[r][0] = v.x;
                        ka[r][1] = v.y;
                        ka[r][2] = v.z;
                        ka[r][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(base + 8 * (k + r) * RB + koff);
                        ka[r][0] = v.x;
                        ka[r][1] = v.y;
                    }
                }
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const unsigned u0 = ka[0][w], u1 = ka[1][w], v0 = u0 >> 8, v1 = u1 >> 8;
                    mma_f16(c, u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u,
                            u1 & 0x00F000F0u, qb[w][0], qb[w][1]);
                    mma_f16(c, v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u,
                            v1 & 0x00F000F0u, qb[w][2], qb[w][3]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint2 mt = *reinterpret_cast<const uint2*>(base + 2 * code_bytes(D) +
                                                                     (8 * (k + r) + g) * 8);
                    const float ks = bf_lo(mt.x), km = bf_hi(mt.x);
                    sv[k + r] = bf_lo(mt.y);
                    mv[k + r] = bf_hi(mt.y);
                    const f32x2 y = fma2(mul2(pair(c[2 * r], c[2 * r + 1]), pair(ks, ks)), ch,
                                         fma2(qs, pair(km, km), pair(-ref0, -ref1)));
                    split(y, y0[k + r], y1[k + r]);
                }
            }
            if ((i + 1) * kTile > tokens) {     // the request's last tile
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i * kTile + 8 * k + krow >= tokens) y0[k] = y1[k] = -INFINITY;
            }

            // ---- weights -----------------------------------------------------------
            // ref is raised only where the tile's largest p times its largest s
            // passes 2^15, which bounds every weight; the raise takes the largest
            // p s to 2^10. s counts 2^-45 here and 2^-50 there at least, so that p
            // stays below 2^60 where rows are constant (s = 0): below s = 2^-74
            // the weights leave FP16's normal range, and sums of p m overflow
            // only for constant rows past 2^40
            float p0[4], p1[4];
            float bigp = 0.0f, bigs = 0x1p-45f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p0[k] = ex2(y0[k]);
                p1[k] = ex2(y1[k]);
                bigp = fmaxf(bigp, fmaxf(p0[k], p1[k]));
                bigs = fmaxf(bigs, fabsf(sv[k]));
            }
            if (fresh || __any_sync(0xffffffffu, bigp * bigs > 32768.0f)) {
                float z0 = kNoRef, z1 = kNoRef;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float ls = log2f(fmaxf(fabsf(sv[k]), 0x1p-50f));
                    z0 = fmaxf(z0, y0[k] + ls);
                    z1 = fmaxf(z1, y1[k] + ls);
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    z0 = fmaxf(z0, __shfl_xor_sync(0xffffffffu, z0, o));
                    z1 = fmaxf(z1, __shfl_xor_sync(0xffffffffu, z1, o));
                }
                // how far ref rises; on the first tile it stands at 0 with nothing
                // summed, and takes the tile's level whatever its sign
                const float low = fresh ? kNoRef : 0.0f;
                float d0 = fmaxf(low, z0 - 10.0f), d1 = fmaxf(low, z1 - 10.0f);
                if (d0 <= kNoRef) d0 = 0.0f;
                if (d1 <= kNoRef) d1 = 0.0f;
                const float f0 = fresh ? 0.0f : half_step(-d0), f1 = fresh ? 0.0f : half_step(-d1);
                ref0 += d0;
                ref1 += d1;
                fresh = false;
                l0 = l0 * f0 * f0;
                l1 = l1 * f1 * f1;
                om0 = om0 * f0 * f0;
                om1 = om1 * f1 * f1;
                const float a0 = f0 * f0, a1 = f1 * f1;
#pragma unroll
                for (int q = 0; q < 4 * VW; ++q) {
                    acc[q][0] *= a0;
                    acc[q][1] *= a1;
                    acc[q][2] *= a0;
                    acc[q][3] *= a1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p0[k] = ex2(y0[k] - d0);
                    p1[k] = ex2(y1[k] - d1);
                }
            }
            unsigned wb[4];                     // head g, tokens 2 t, 2 t + 1 of each 8
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const f32x2 pp = pair(p0[k], p1[k]);
                split(add2(pair(l0, l1), pp), l0, l1);
                split(fma2(pp, pair(mv[k], mv[k]), pair(om0, om1)), om0, om1);
                float w0, w1;
                split(mul2(pp, pair(sv[k], sv[k])), w0, w1);
                wb[k] = transpose8(h2_of(w0, w1));
            }

            // ---- o += V^T w ----------------------------------------------------------
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                unsigned x[4][VW];              // tokens 2 t, 2 t + 1 of two groups of 8
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const unsigned char* at = base + code_bytes(D) + (k + (r >> 1)) * 8 * RB +
                                              ((r & 1) ? voff1 : voff0);
                    if constexpr (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2*>(at);
                        x[r][0] = v.x;
                        x[r][1] = v.y;
                    } else {
                        x[r][0] = *reinterpret_cast<const unsigned*>(at);
                    }
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        // four dimensions of both tokens, one token per half
                        const unsigned u0 = __byte_perm(x[0][w], x[1][w], hf ? 0x7632 : 0x5410);
                        const unsigned u1 = __byte_perm(x[2][w], x[3][w], hf ? 0x7632 : 0x5410);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            // both tokens' byte s alone (one permute with zero for the
                            // upper one), then its low nibble
                            const unsigned b0 = s ? __byte_perm(u0, 0, 0x4341) : u0 & 0x00FF00FFu;
                            const unsigned b1 = s ? __byte_perm(u1, 0, 0x4341) : u1 & 0x00FF00FFu;
                            mma_f16(acc[4 * w + 2 * hf + s], b0 & 0x000F000Fu, b0,
                                    b1 & 0x000F000Fu, b1, wb[k], wb[k + 1]);
                        }
                    }
                }
            }
            __syncwarp();                       // the stage has been read
            fetch(i + kStages * TW, st, nblk, nin);
            lookup(i + (kStages + 1) * TW, nblk, nin);
            st = st + 1 == kStages ? 0 : st + 1;
        }
        // ---- the next piece's first copies, then what this one leaves -------------
        const int mb = b;
        const unsigned slot = 2 * (r * p.Hkv + h) + (first ? 0 : 1);
        const bool old = joins, ends = j1 == n_all, all = from0 && ends;
        left -= j1 - j;
        const bool more = left > 0;
        joins = more && !ends;
        j = joins ? j1 : 0;
        if (more) {
            if (!joins) {
                first = false;
                from0 = true;
                do {
                    tokens = tokens_of(p, ++b);
                } while (tokens == 0);
            }
            open();
        }
        if (TW > 1 && again) __syncthreads();   // the last piece's parts have been read
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            om0 += __shfl_xor_sync(0xffffffffu, om0, o);
            om1 += __shfl_xor_sync(0xffffffffu, om1, o);
        }
        if (fresh) ref0 = ref1 = kNoRef;
        // dimensions 4 VW 2 g + i of head 2 t + e
        constexpr int LD = 8 * VW;
        auto value = [&](int e, int i) {
            const float lo = acc[i >> 1][e];
            return i & 1 ? __fmaf_rn(acc[i >> 1][2 + e] - lo, 1048576.0f, e ? om1 : om0)
                         : __fmaf_rn(lo, 16777216.0f, e ? om1 : om0);
        };
        const PartView part = {p.part + plan_bytes(p.B) / 4, D, G};
        if constexpr (TW == 1) {
            float2 was[2];                      // (ref, sum) of the segment's pieces so far
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (old && 2 * t + e < G)
                    was[e] = *reinterpret_cast<const float2*>(part.o(slot, 2 * t + e) + D);
            __syncwarp();                       // read before lane g = 0 writes them again
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hd = 2 * t + e;
                if (hd >= G) continue;
                float L = e ? l1 : l0, ref = e ? ref1 : ref0, val[LD];
#pragma unroll
                for (int i = 0; i < LD; ++i) val[i] = value(e, i);
                if (old) {
                    const float* po = part.o(slot, hd);
                    const float up = fmaxf(ref, was[e].x);
                    const float f = half_step(ref - up), q = half_step(was[e].x - up);
                    ref = up;
                    L = __fmaf_rn(L * f, f, was[e].y * q * q);
#pragma unroll
                    for (int i = 0; i < LD; ++i)
                        val[i] = __fmaf_rn(val[i] * f, f, po[LD * g + i] * q * q);
                }
                if (all) {
                    bf16* po = p.out + ((size_t)mb * p.Hq + (size_t)h * G + hd) * D + LD * g;
#pragma unroll
                    for (int i = 0; i < LD; i += 8) {
                        unsigned w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(
                                __fdividef(val[i + 2 * k], L), __fdividef(val[i + 2 * k + 1], L));
                            w[k] = *reinterpret_cast<const unsigned*>(&v);
                        }
                        *reinterpret_cast<int4*>(po + i) = make_int4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    float* po = part.o(slot, hd);
#pragma unroll
                    for (int i = 0; i < LD; i += 4)
                        *reinterpret_cast<float4*>(po + LD * g + i) =
                            make_float4(val[i], val[i + 1], val[i + 2], val[i + 3]);
                    if (g == 0) {
                        po[D] = ref;
                        po[D + 1] = L;
                    }
                }
            }
            __syncwarp();
            if (more) copy_first();
        } else {
            float* so = reinterpret_cast<float*>(smem + ring_bytes(D));   // [warp][8][D + 4]
            float* sref = so + kWarps * 8 * (D + 4);                      // [warp][8]
            float* sl = sref + kWarps * 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hd = warp * 8 + 2 * t + e;
                if (g == 0) {
                    sref[hd] = e ? ref1 : ref0;
                    sl[hd] = e ? l1 : l0;
                }
                float* po = so + hd * (D + 4) + LD * g;
#pragma unroll
                for (int i = 0; i < LD; i += 4)
                    *reinterpret_cast<float4*>(po + i) = make_float4(
                        value(e, i), value(e, i + 1), value(e, i + 2), value(e, i + 3));
            }
            if (more) copy_first();
            __syncthreads();
            for (int i = threadIdx.x; i < HW * G * D; i += kThreads) {
                const int x = i / (G * D), hd = (i - x * G * D) / D, d = i % D;
                float top = kNoRef;
#pragma unroll
                for (int w = 0; w < TW; ++w) top = fmaxf(top, sref[(w * HW + x) * 8 + hd]);
                float o = 0.0f, L = 0.0f;
#pragma unroll
                for (int w = 0; w < TW; ++w) {
                    const int at = (w * HW + x) * 8 + hd;
                    const float f = half_step(sref[at] - top);
                    o = __fmaf_rn(f, f * so[at * (D + 4) + d], o);
                    L = __fmaf_rn(f, f * sl[at], L);
                }
                const int hx = h - hw + x;
                if (all && !old) {
                    p.out[((size_t)mb * p.Hq + (size_t)hx * G + hd) * D + d] = f2bf(__fdividef(o, L));
                } else {
                    float* po = old ? so + (x * 8 + hd) * (D + 4)   // this thread's own element
                                    : part.o(slot + 2 * (x - hw), hd);
                    po[d] = o;
                    if (d == 0) {
                        po[D] = top;
                        po[D + 1] = L;
                    }
                }
            }
            if (old) {
                __syncthreads();
#pragma unroll 1
                for (int k = warp; k < HW * G; k += kWarps) {
                    const int x = k / G, hd = k - x * G, hx = h - hw + x;
                    bf16* out = all ? p.out + ((size_t)mb * p.Hq + (size_t)hx * G + hd) * D : nullptr;
                    add_piece<D>(part.o(slot + 2 * (x - hw), hd), so + (x * 8 + hd) * (D + 4), out,
                                 lane);
                }
            }
        }
        if (!more) break;
    }
}

// Joins the parts of each (request, query head) that several CTAs share, and
// writes the zeros of requests without tokens. One CTA per query head and
// request; its warps take the parts two at a time, each
// with a running ref, and then join theirs.
template <int D>
__global__ void __launch_bounds__(kCombineThreads) attn_i4_combine_kernel(const AttnI4Params p) {
    constexpr int NW = kCombineThreads / 32, EL = D / 32;
    __shared__ float s_ref[NW], s_l[NW];
    __shared__ float so[NW][D];
    const int hq = blockIdx.x, b = blockIdx.y;
    const int G = p.Hq / p.Hkv, h = hq / G, hd = hq - h * G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bf16* out = p.out + ((size_t)b * p.Hq + hq) * D;
    pdl_wait();
    pdl_trigger();
    const int2 plan = __ldcg(reinterpret_cast<const int2*>(p.part) + b);
    if (plan.x < 0) {
        for (int d = threadIdx.x; d < D; d += kCombineThreads) out[d] = __float2bfloat16_rn(0.0f);
        return;
    }
    const int c0 = plan.x >> 1, c1 = plan.y;
    if (c0 == c1) return;                       // one CTA had all of it
    const PartView part = {p.part + plan_bytes(p.B) / 4, D, G};
    float ref = kNoRef, L = 0.0f, o[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) o[e] = 0.0f;
    for (int c = c0 + warp; c <= c1; c += kJoin * NW) {
        float2 rl[kJoin];
        float v[kJoin][EL];
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const int ck = c + k * NW;
            rl[k] = make_float2(kNoRef, 0.0f);
#pragma unroll
            for (int e = 0; e < EL; ++e) v[k][e] = 0.0f;
            if (ck <= c1) {
                const float* po = part.o(2u * (ck * p.Hkv + h) + (ck == c0 ? plan.x & 1 : 0), hd);
                rl[k] = __ldcg(reinterpret_cast<const float2*>(po + D));
#pragma unroll
                for (int e = 0; e < EL; ++e) v[k][e] = __ldcg(po + lane + 32 * e);
            }
        }
        float up = ref;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) up = fmaxf(up, rl[k].x);
        const float f = half_step(ref - up);
        ref = up;
        L = L * f * f;
#pragma unroll
        for (int e = 0; e < EL; ++e) o[e] = o[e] * f * f;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
            const float g = half_step(rl[k].x - up);
            L = __fmaf_rn(rl[k].y * g, g, L);
#pragma unroll
            for (int e = 0; e < EL; ++e) o[e] = __fmaf_rn(v[k][e] * g, g, o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) so[warp][lane + 32 * e] = o[e];
    if (lane == 0) {
        s_ref[warp] = ref;
        s_l[warp] = L;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kCombineThreads) {
        float top = kNoRef, O = 0.0f, Ls = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, s_ref[w]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = half_step(s_ref[w] - top);
            O = __fmaf_rn(f, f * so[w][d], O);
            Ls = __fmaf_rn(f, f * s_l[w], Ls);
        }
        out[d] = f2bf(__fdividef(O, Ls));
    }
}

// Tables of at most this many tokens go to one CTA per (request, KV head),
// without the run search and the second kernel. By the table's width, because
// the contexts are on the device: a wider table may hold one long request
// among short ones, which one CTA would take alone. Requests of 256 tokens, 40
// query and 8 KV heads of 128: one 4.6 us against 7.3 by runs, 16 5.0 against
// 8.3, 64 10.2 against 12.7, 256 29.8 against 29.3; at 1024 tokens each 8.6
// against 7.6, 9.0 / 10.3, 21.5 / 21.9, 65.1 / 67.4.
constexpr int kWholeCtx = 256;

// KV heads that a CTA's warps stand for when it takes a run.
int heads_per_cta(int Hkv) { return Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1; }
int runs_of(int B, int Hkv, int max_ctx) {
    const long tiles = (long)B * tiles_of(max_ctx);
    const long fit = kMaxCtas / (Hkv / heads_per_cta(Hkv));
    return (int)std::max(1L, std::min((tiles + kMinTiles - 1) / kMinTiles, fit));
}

template <typename Kern, typename... Args>
cudaError_t launch_i4(Kern kern, dim3 grid, int block, size_t smem, const Launch& L, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int HW>
cudaError_t launch_runs(const AttnI4Params& p, int grid, bool whole, const Launch& L) {
    const size_t smem = smem_bytes(D, HW);
    cudaError_t e = once_per_context((const void*)attn_i4_kernel<D, HW>, [&] {
        return cudaFuncSetAttribute(attn_i4_kernel<D, HW>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    const unsigned inv = 0xFFFFFFFFu / (unsigned)p.page;
    return launch_i4(attn_i4_kernel<D, HW>, dim3(grid), kThreads, smem, L, p, inv, whole);
}

template <int D>
cudaError_t launch_attention_i4_d(const AttnI4Params& p, const Launch& L) {
    const int max_ctx = p.max_blocks * p.page;
    if (max_ctx <= kWholeCtx) return launch_runs<D, 1>(p, p.B * p.Hkv, true, L);
    const int HW = heads_per_cta(p.Hkv), grid = runs_of(p.B, p.Hkv, max_ctx) * (p.Hkv / HW);
    cudaError_t e = HW == 4   ? launch_runs<D, 4>(p, grid, false, L)
                    : HW == 2 ? launch_runs<D, 2>(p, grid, false, L)
                              : launch_runs<D, 1>(p, grid, false, L);
    if (e != cudaSuccess) return e;
    return launch_i4(attn_i4_combine_kernel<D>, dim3(p.Hq, p.B), kCombineThreads, 0, L, p);
}

}  // namespace

long attn_i4_run_tokens(int B, int Hkv, int max_ctx) {
    const long tiles = (long)B * tiles_of(max_ctx);
    return max_ctx <= kWholeCtx ? max_ctx : (tiles / runs_of(B, Hkv, max_ctx) + 1) * kTile;
}

size_t attn_i4_part_bytes(int B, int Hq, int Hkv, int D, int max_ctx) {
    if (max_ctx <= kWholeCtx) return 0;
    return plan_bytes(B) + (size_t)runs_of(B, Hkv, max_ctx) * 2 * Hq * (D + 4) * 4;
}

cudaError_t launch_attention_i4(const AttnI4Params& p, const Launch& L) {
    if (p.B == 0) return cudaSuccess;
    if (p.D == 128) return launch_attention_i4_d<128>(p, L);
    if (p.D == 64) return launch_attention_i4_d<64>(p, L);
    return cudaErrorInvalidValue;
}

}  // namespace a8w8
