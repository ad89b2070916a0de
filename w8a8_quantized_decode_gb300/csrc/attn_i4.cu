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
// copy rate an SM receives 16 tokens' rows (2.2 KB at D = 128) in about 95
// cycles, in which it can issue 380 warp instructions; unpacking 4096 codes to
// 16-bit floats alone would take half of them. An integer 0..15 in a byte is,
// read as e4m3, exactly c 2^-9 (c < 8 is a subnormal, 8..15 the first binade),
// so a word of eight codes becomes two operand registers of mma.sync
// m16n8k32 e4m3 with two masks and a shift, and no conversion. The other
// operand is split into e4m3 parts whose products with the codes are exact
// and summed in float32 by the tensor cores (measured on this GPU: 2100
// TFLOP/s against 600 for bf16 m16n8k16, sums exact to float32 rounding):
//   * q, scaled by a power of two to a maximum in [128, 256): two parts of
//     four significant bits hold the eight of a BF16, down to 2^-21 of the
//     head's largest |q|. Query heads are rows 0..7 of the A operand, their
//     low parts (times 2^5) rows 8..15: one instruction does both.
//   * the weights p_t s_t: rounded to FP16 (2^-11 relative; beside the BF16
//     result's 2^-8 this is what keeps them out of its error) and split into
//     three parts of one common scale, so that all add into one accumulator;
//     ref keeps the largest between 128 and 448, and the last bit of e4m3
//     stands 2^-17 below that.
// The score accumulator holds (head, token) pairs in the same lanes that the
// weights' operand needs them in (tokens are permuted alike for K and V), so
// nothing is exchanged between the two products. For V the contraction runs
// over tokens: a lane reads 8 tokens' bytes for its 16 dimensions and
// transposes 4 x 4 bytes with eight permutes.
//
// Work is cut into tiles of 32 tokens of one (request, KV head), numbered
// through all requests; a CTA takes an equal run of them, whatever the
// contexts, and its four warps take the run's tiles in turn, each with a
// private cp.async ring (no CTA barrier inside a run). Runs that end inside a
// (request, KV head) leave their (ref, sum, o) to a second kernel.
#include "kernels.cuh"

namespace a8w8 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 32;            // tokens a warp takes at a time
constexpr int kStages = 3;           // ring depth per warp
constexpr int kCtasPerSm = 4;
constexpr int kMaxCtas = 152 * kCtasPerSm;
constexpr int kMinTiles = 4;         // tiles per CTA at least: one per warp
constexpr int kCombineThreads = 128;
constexpr float kNoRef = -1e30f;     // ref of a head that has seen no token

constexpr int code_bytes(int D) { return kTile * D / 2; }
constexpr int stage_bytes(int D) { return 2 * code_bytes(D) + kTile * 8; }
constexpr int merge_bytes(int D) { return kWarps * 8 * (D + 4) * 4 + 2 * kWarps * 8 * 4; }
constexpr int smem_bytes(int D) {
    const int ring = kWarps * kStages * stage_bytes(D);
    return ring > merge_bytes(D) ? ring : merge_bytes(D);
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], unsigned a0, unsigned a1, unsigned a2,
                                         unsigned a3, unsigned b0, unsigned b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two floats as e4m3 bytes (a in the low byte), and two e4m3 bytes as FP16.
__device__ __forceinline__ unsigned short e4m3_of(float a, float b) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ unsigned short e4m3_of_h2(unsigned h) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ unsigned h2_of_e4m3(unsigned short e) {
    unsigned r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(e));
    return r;
}
__device__ __forceinline__ unsigned h2_of(float a, float b) {
    unsigned r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ unsigned h2_sub(unsigned a, unsigned b) {
    unsigned r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 h2_floats(unsigned h) {
    float2 f;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
__device__ __forceinline__ unsigned join16(unsigned short lo, unsigned short hi) {
    return (unsigned)lo | (unsigned)hi << 16;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void cp16z(unsigned s, const void* g, unsigned n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(g), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4z(unsigned s, const void* g, unsigned n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(g), "r"(n) : "memory");
}
__device__ __forceinline__ uint2 lds_v2(unsigned s) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(s));
    return r;
}
__device__ __forceinline__ unsigned lds_1(unsigned s) {
    unsigned r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(s));
    return r;
}
__device__ __forceinline__ float bf_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(unsigned w) { return __uint_as_float(w & 0xFFFF0000u); }

// Tiles of request b: none where the context is out of range.
__device__ __forceinline__ int tokens_of(const AttnI4Params& p, int b) {
    const int c = __ldg(p.ctx_lens + b);
    return c < 0 || c > p.max_blocks * p.page ? 0 : c;
}
__device__ __forceinline__ int tiles_of(int tokens) { return (tokens + kTile - 1) / kTile; }

// Exclusive sum of v over the CTA's NT threads (total in `total`).
template <int NT>
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
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += s[w];
        total += s[w];
    }
    return before + x - v;
}

// The runs: CTA c of E takes tiles [c T / E, (c + 1) T / E) of T = Hkv sum_b
// tiles(b), request after request, KV heads inside a request.
__device__ __forceinline__ long run_ctas(long T, int grid) {
    const long e = (T + kMinTiles - 1) / kMinTiles;
    return e < grid ? e : grid;
}

struct PartView {
    float* base;
    int D, G;
    __device__ float* o(long slot, int head) const {
        return base + (slot * G + head) * (long)(D + 4);
    }
};

template <int D>
struct Frag {
    static constexpr int KW = D / 32;   // 32-bit words of K codes per lane and token
    static constexpr int VW = D / 64;   // words of V codes per lane and token
};

// One CTA's share: the tiles of its run (or, with `whole`, all tiles of one
// (request, KV head) per CTA).
template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    attn_i4_kernel(const AttnI4Params p, const unsigned page_inv, const bool whole) {
    constexpr int KW = Frag<D>::KW, VW = Frag<D>::VW;
    constexpr int RB = D / 2;                   // bytes of a row's codes
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long s_scan[kWarps];
    __shared__ long s_first;
    __shared__ int s_b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv;
    const unsigned sbase = (unsigned)__cvta_generic_to_shared(smem);
    const unsigned ring = sbase + warp * kStages * stage_bytes(D);

    pdl_wait();
    pdl_trigger();

    // ---- where the run begins -------------------------------------------------
    long x0, x1;                   // the run's tiles
    int b, h, j, tokens;           // its first tile: request, KV head, tile
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
        x0 = 0;
        x1 = tiles_of(tokens);
    } else {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        long mine = 0;
        for (int i = b0; i < b1; ++i) {
            if (blockIdx.x == 0) {
                const int c = p.ctx_lens[i];
                if (c < 0 || c > p.max_blocks * p.page) set_error(p.err, 0x4u);
            }
            mine += tiles_of(tokens_of(p, i));
        }
        long total;
        const long before = cta_exclusive<kThreads>(mine, s_scan, total);
        const long T = total * p.Hkv, E = run_ctas(T, gridDim.x);
        if (blockIdx.x >= E) return;
        x0 = T * blockIdx.x / E;
        x1 = T * (blockIdx.x + 1) / E;
        if (mine > 0 && x0 >= before * p.Hkv && x0 < (before + mine) * p.Hkv) {
            long at = before;
            int i = b0;
            for (;; ++i) {
                const int n = tiles_of(tokens_of(p, i));
                if (x0 < (at + n) * p.Hkv) break;
                at += n;
            }
            s_b = i;
            s_first = at * p.Hkv;
        }
        __syncthreads();
        b = s_b;
        tokens = tokens_of(p, b);
        const long in = x0 - s_first;
        h = (int)(in / tiles_of(tokens));
        j = (int)(in - (long)h * tiles_of(tokens));
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

    bool first = true;                          // the run's first segment
    while (x0 < x1) {
        const int n_all = tiles_of(tokens);
        const int j1 = (int)min((long)n_all, j + (x1 - x0));
        const int32_t* table = p.block_table + (size_t)b * p.max_blocks;

        // Copies tile i of the segment's request into ring stage st: a token's
        // row number once per lane, handed to the lanes that copy its chunks.
        auto fetch = [&](int i, int st) {
            const unsigned tok = (unsigned)i * kTile + lane;
            int slot = -1;
            if (i < j1 && (int)tok < tokens) {
                unsigned q = __umulhi(tok, page_inv), r = tok - q * p.page;
                if (r >= (unsigned)p.page) {
                    ++q;
                    r -= p.page;
                }
                const int blk = __ldg(table + q);
                if (blk >= 0 && blk < p.num_blocks) slot = blk * p.page + (int)r;
                else set_error(p.err, 0x2u);
            }
            if (i < j1) {                        // warp-uniform
                const unsigned base = ring + st * stage_bytes(D);
#pragma unroll
                for (int k = 0; k < kTile / RPI; ++k) {
                    const int sl = __shfl_sync(0xffffffffu, slot, k * RPI + crow);
                    const size_t off = sl < 0 ? 0 : ((size_t)sl * p.Hkv + h) * RB + cchunk * 16;
                    const unsigned n = sl < 0 ? 0u : 16u;
                    const unsigned d = base + k * RPI * RB + coff;
                    cp16z(d, p.c.k_codes + off, n);
                    cp16z(d + code_bytes(D), p.c.v_codes + off, n);
                }
                const size_t row = slot < 0 ? 0 : (size_t)slot * p.Hkv + h;
                const unsigned n = slot < 0 ? 0u : 4u;
                const unsigned d = base + 2 * code_bytes(D) + mcol * 8;
                cp4z(d, p.c.k_meta + 2 * row, n);
                cp4z(d + 4, p.c.v_meta + 2 * row, n);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s) fetch(j + warp + s * kWarps, s);

        // ---- the query heads' parts ---------------------------------------------
        unsigned qa[KW][4];
        float ch, qsum;                         // score factors of head g
        {
            const bf16* q = p.q + ((size_t)b * p.Hq + (size_t)h * G + (g < G ? g : 0)) * D + t * (D / 4);
            float sum = 0.0f, top = 0.0f;
            int4 raw[KW];
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                raw[w] = g < G ? ld_cg_v4(q + 8 * w) : make_int4(0, 0, 0, 0);
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
            // 2^e takes the largest |q| into [128, 256)
            const int e = max(-111, min(110, 134 - (int)(__float_as_uint(top) >> 23)));
            const float up = __uint_as_float((unsigned)(127 + e) << 23);
            const float sc = p.scale * 1.4426950408889634f;
            ch = __uint_as_float((unsigned)(127 + 9 - e) << 23) * sc;
            qsum = sum * sc;
            // a NaN shows in the sum; above 2^118 the parts would saturate
            if (!(fabsf(sum) <= 3e38f) || top >= 3.3e35f) ch = __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                float f[8];
                unpack8(raw[w], f);
#pragma unroll
                for (int o = 0; o < 2; ++o) {   // even elements: low nibbles; odd: high
                    unsigned short hi[2], lo[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float a = f[4 * k + o] * up, c = f[4 * k + 2 + o] * up;
                        hi[k] = e4m3_of(a, c);
                        const float2 r = h2_floats(h2_of_e4m3(hi[k]));
                        lo[k] = e4m3_of((a - r.x) * 32.0f, (c - r.y) * 32.0f);
                    }
                    qa[w][2 * o] = join16(hi[0], hi[1]);
                    qa[w][2 * o + 1] = join16(lo[0], lo[1]);
                }
            }
        }

        float acc[4 * VW][4];                   // o 2^-9: rows dims, columns heads 2 t, 2 t + 1
#pragma unroll
        for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
        float ref = kNoRef, l = 0.0f, om = 0.0f;   // of head g, over the lane's tokens

        int st = 0;
        for (int i = j + warp; i < j1; i += kWarps) {
            cp_async_wait_group<kStages - 1>();
            __syncwarp();
            const unsigned base = ring + st * stage_bytes(D);

            // ---- scores: head g, tokens 8 k + (2 t, 2 t + 1) of the tile --------
            float y[8], sv[8], mv[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned kw[KW];
                if constexpr (D == 128) {
                    const int4 v = lds_v4(base + 8 * k * RB + koff);
                    kw[0] = v.x;
                    kw[1] = v.y;
                    kw[2] = v.z;
                    kw[3] = v.w;
                } else {
                    const uint2 v = lds_v2(base + 8 * k * RB + koff);
                    kw[0] = v.x;
                    kw[1] = v.y;
                }
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < KW; ++w)
                    mma_e4m3(c, qa[w][0], qa[w][1], qa[w][2], qa[w][3], kw[w] & 0x0F0F0F0Fu,
                             (kw[w] >> 4) & 0x0F0F0F0Fu);
                const int4 mt = lds_v4(base + 2 * code_bytes(D) + (8 * k + 2 * t) * 8);
                const float a0 = __fmaf_rn(c[2], 0.03125f, c[0]) * ch;
                const float a1 = __fmaf_rn(c[3], 0.03125f, c[1]) * ch;
                y[2 * k] = __fmaf_rn(a0, bf_lo(mt.x), qsum * bf_hi(mt.x));
                y[2 * k + 1] = __fmaf_rn(a1, bf_lo(mt.z), qsum * bf_hi(mt.z));
                sv[2 * k] = bf_lo(mt.y);
                mv[2 * k] = bf_hi(mt.y);
                sv[2 * k + 1] = bf_lo(mt.w);
                mv[2 * k + 1] = bf_hi(mt.w);
            }
            if ((i + 1) * kTile > tokens) {     // the request's last tile
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int tok = i * kTile + 8 * (k >> 1) + 2 * t + ((k & 1) ^ (t >> 1));
                    if (tok >= tokens) y[k] = -INFINITY;
                }
            }

            // ---- weights -----------------------------------------------------------
            // ref is raised only where a weight would pass e4m3's 448 (or a
            // probability with s near 0 would pass 2^90); the raise takes the
            // tile's largest to 128
            float pr[8], wt[8];
            float big = 0.0f, bigp = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                pr[k] = ex2(y[k] - ref);
                wt[k] = pr[k] * sv[k];
                big = fmaxf(big, fabsf(wt[k]));
                bigp = fmaxf(bigp, pr[k]);
            }
            if (__any_sync(0xffffffffu, big > 448.0f || bigp > 1.2e27f)) {
                float z = kNoRef;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    z = fmaxf(z, y[k] + log2f(fmaxf(fabsf(sv[k]), 8.3e-25f)));
                z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 1));
                z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 2));
                const float up = fmaxf(ref, z - 7.0f);
                const float f = ex2(ref - up);
                ref = up;
                l *= f;
                om *= f;
                const float f0 = __shfl_sync(0xffffffffu, f, 8 * t);
                const float f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
                for (int q = 0; q < 4 * VW; ++q) {
                    acc[q][0] *= f0;
                    acc[q][1] *= f1;
                    acc[q][2] *= f0;
                    acc[q][3] *= f1;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    pr[k] = ex2(y[k] - ref);
                    wt[k] = pr[k] * sv[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                l += pr[k];
                om = __fmaf_rn(pr[k], mv[k], om);
            }
            unsigned wb[3][2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                unsigned r0 = h2_of(wt[4 * q], wt[4 * q + 1]), r1 = h2_of(wt[4 * q + 2], wt[4 * q + 3]);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const unsigned short e0 = e4m3_of_h2(r0), e1 = e4m3_of_h2(r1);
                    wb[k][q] = join16(e0, e1);
                    if (k < 2) {
                        r0 = h2_sub(r0, h2_of_e4m3(e0));
                        r1 = h2_sub(r1, h2_of_e4m3(e1));
                    }
                }
            }

            // ---- o += V^T w ----------------------------------------------------------
            unsigned x[2][4][VW];               // [token quad][token][word]
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned at = base + code_bytes(D) + (2 * q + (k >> 1)) * 8 * RB +
                                        ((k & 1) ? voff1 : voff0);
                    if constexpr (D == 128) {
                        const uint2 v = lds_v2(at);
                        x[q][k][0] = v.x;
                        x[q][k][1] = v.y;
                    } else {
                        x[q][k][0] = lds_1(at);
                    }
                }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                unsigned T[2][4];               // byte d of the quad's four tokens
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const unsigned a = __byte_perm(x[q][0][w], x[q][1][w], 0x5140);
                    const unsigned c = __byte_perm(x[q][2][w], x[q][3][w], 0x5140);
                    const unsigned d = __byte_perm(x[q][0][w], x[q][1][w], 0x7362);
                    const unsigned f = __byte_perm(x[q][2][w], x[q][3][w], 0x7362);
                    T[q][0] = __byte_perm(a, c, 0x5410);
                    T[q][1] = __byte_perm(a, c, 0x7632);
                    T[q][2] = __byte_perm(d, f, 0x5410);
                    T[q][3] = __byte_perm(d, f, 0x7632);
                }
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const unsigned a0 = T[0][d] & 0x0F0F0F0Fu, a1 = (T[0][d] >> 4) & 0x0F0F0F0Fu;
                    const unsigned a2 = T[1][d] & 0x0F0F0F0Fu, a3 = (T[1][d] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        mma_e4m3(acc[4 * w + d], a0, a1, a2, a3, wb[k][0], wb[k][1]);
                }
            }
            __syncwarp();                       // the stage has been read
            fetch(i + kStages * kWarps, st);
            st = st + 1 == kStages ? 0 : st + 1;
        }
        cp_async_wait_group<0>();
        __syncthreads();                        // the rings become the merge buffer

        // ---- the four warps' parts ---------------------------------------------
        float* so = reinterpret_cast<float*>(smem);              // [warp][8][D + 4]
        float* sref = so + kWarps * 8 * (D + 4);                 // [warp][8]
        float* sl = sref + kWarps * 8;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        om += __shfl_xor_sync(0xffffffffu, om, 1);
        om += __shfl_xor_sync(0xffffffffu, om, 2);
        if (t == 0) {
            sref[warp * 8 + g] = ref;
            sl[warp * 8 + g] = l;
        }
        {
            const float m0 = __shfl_sync(0xffffffffu, om, 8 * t);
            const float m1 = __shfl_sync(0xffffffffu, om, 8 * t + 4);
            float* r0 = so + (warp * 8 + 2 * t) * (D + 4) + 8 * VW * g;
            float* r1 = r0 + (D + 4);
#pragma unroll
            for (int q = 0; q < 4 * VW; q += 2) {
                *reinterpret_cast<float4*>(r0 + 2 * q) =
                    make_float4(__fmaf_rn(acc[q][0], 512.0f, m0), __fmaf_rn(acc[q][2], 512.0f, m0),
                                __fmaf_rn(acc[q + 1][0], 512.0f, m0), __fmaf_rn(acc[q + 1][2], 512.0f, m0));
                *reinterpret_cast<float4*>(r1 + 2 * q) =
                    make_float4(__fmaf_rn(acc[q][1], 512.0f, m1), __fmaf_rn(acc[q][3], 512.0f, m1),
                                __fmaf_rn(acc[q + 1][1], 512.0f, m1), __fmaf_rn(acc[q + 1][3], 512.0f, m1));
            }
        }
        __syncthreads();
        const bool all = j == 0 && j1 == n_all;
        const PartView part = {p.part, D, G};
        for (int i = threadIdx.x; i < G * D; i += kThreads) {
            const int hd = i / D, d = i - hd * D;
            float top = sref[hd];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sref[w * 8 + hd]);
            float o = 0.0f, L = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sref[w * 8 + hd] - top);
                o = __fmaf_rn(f, so[(w * 8 + hd) * (D + 4) + d], o);
                L = __fmaf_rn(f, sl[w * 8 + hd], L);
            }
            if (all) {
                p.out[((size_t)b * p.Hq + (size_t)h * G + hd) * D + d] = f2bf(__fdividef(o, L));
            } else {
                float* po = part.o(2L * blockIdx.x + (first ? 0 : 1), hd);
                po[d] = o;
                if (d == 0) {
                    po[D] = top;
                    po[D + 1] = L;
                }
            }
        }
        __syncthreads();                        // the buffer becomes the rings again

        // ---- the next segment -----------------------------------------------------
        x0 += j1 - j;
        j = 0;
        first = false;
        if (x0 < x1 && ++h == p.Hkv) {
            h = 0;
            do {
                tokens = tokens_of(p, ++b);
            } while (tokens == 0);
        }
    }
}

// Joins the parts of each (request, query head) that several CTAs share, and
// writes the zeros of requests without tokens. One CTA per query head and
// request; its warps take the parts in turn.
template <int D>
__global__ void __launch_bounds__(kCombineThreads)
    attn_i4_combine_kernel(const AttnI4Params p, const int grid) {
    constexpr int NW = kCombineThreads / 32, E = D / 32;
    __shared__ long s_scan[NW];
    __shared__ float s_max[NW];
    __shared__ float so[NW][D];
    __shared__ float s_l[NW];
    pdl_wait();
    pdl_trigger();
    const int hq = blockIdx.x, b = blockIdx.y;
    const int G = p.Hq / p.Hkv, h = hq / G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bf16* out = p.out + ((size_t)b * p.Hq + hq) * D;
    const int n = tiles_of(tokens_of(p, b));
    if (n == 0) {
        for (int d = threadIdx.x; d < D; d += kCombineThreads) out[d] = __float2bfloat16_rn(0.0f);
        return;
    }
    long all = 0, before = 0;
    for (int i = threadIdx.x; i < p.B; i += kCombineThreads) {
        const int m = tiles_of(tokens_of(p, i));
        all += m;
        if (i < b) before += m;
    }
    long total, total_before;
    cta_exclusive<kCombineThreads>(all, s_scan, total);
    __syncthreads();
    cta_exclusive<kCombineThreads>(before, s_scan, total_before);
    const long T = total * p.Hkv, Ec = run_ctas(T, grid);
    const long a0 = total_before * p.Hkv + (long)h * n, a1 = a0 + n;
    const int c0 = (int)(((a0 + 1) * Ec - 1) / T), c1 = (int)((a1 * Ec - 1) / T);
    if (c0 == c1) return;                       // one CTA had all of it
    const PartView part = {p.part, D, G};
    const int hd = hq - h * G;
    // CTA c0's part is its run's first segment only if the run begins with it
    const bool c0_first = T * c0 / Ec >= a0;
    auto slot = [&](int c) { return 2L * c + (c == c0 && !c0_first ? 1 : 0); };
    float top = kNoRef;
    for (int c = c0 + (int)threadIdx.x; c <= c1; c += kCombineThreads)
        top = fmaxf(top, __ldcg(part.o(slot(c), hd) + D));
    top = warp_max(top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_max[w]);
    float o[E], L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int c = c0 + warp; c <= c1; c += NW) {
        const float* po = part.o(slot(c), hd);
        const float f = ex2(__ldcg(po + D) - top);
        L = __fmaf_rn(f, __ldcg(po + D + 1), L);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __fmaf_rn(f, __ldcg(po + lane + 32 * e), o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kCombineThreads) {
        float O = 0.0f, Ls = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            O += so[w][d];
            Ls += s_l[w];
        }
        out[d] = f2bf(__fdividef(O, Ls));
    }
}

// Contexts of at most this many tokens go to one CTA per (request, KV head).
constexpr int kWholeCtx = 256;

int grid_of(int B, int Hkv, int max_ctx) {
    const long tiles = (long)B * Hkv * ((max_ctx + kTile - 1) / kTile);
    const long e = (tiles + kMinTiles - 1) / kMinTiles;
    return (int)(e < kMaxCtas ? e : kMaxCtas);
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

template <int D>
cudaError_t launch_attention_i4_d(const AttnI4Params& p, const Launch& L) {
    const size_t smem = smem_bytes(D);
    cudaError_t e = once_per_context((const void*)attn_i4_kernel<D>, [&] {
        return cudaFuncSetAttribute(attn_i4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem);
    });
    if (e != cudaSuccess) return e;
    const unsigned inv = 0xFFFFFFFFu / (unsigned)p.page;
    const int max_ctx = p.max_blocks * p.page;
    if (max_ctx <= kWholeCtx)
        return launch_i4(attn_i4_kernel<D>, dim3(p.B * p.Hkv), kThreads, smem, L, p, inv, true);
    const int grid = grid_of(p.B, p.Hkv, max_ctx);
    e = launch_i4(attn_i4_kernel<D>, dim3(grid), kThreads, smem, L, p, inv, false);
    if (e != cudaSuccess) return e;
    return launch_i4(attn_i4_combine_kernel<D>, dim3(p.Hq, p.B), kCombineThreads, 0, L, p, grid);
}

}  // namespace

size_t attn_i4_part_bytes(int B, int Hq, int Hkv, int D, int max_ctx) {
    if (max_ctx <= kWholeCtx) return 0;
    return (size_t)grid_of(B, Hkv, max_ctx) * 2 * (Hq / Hkv) * (D + 4) * 4;
}

cudaError_t launch_attention_i4(const AttnI4Params& p, const Launch& L) {
    if (p.B == 0) return cudaSuccess;
    if (p.D == 128) return launch_attention_i4_d<128>(p, L);
    if (p.D == 64) return launch_attention_i4_d<64>(p, L);
    return cudaErrorInvalidValue;
}

}  // namespace a8w8
