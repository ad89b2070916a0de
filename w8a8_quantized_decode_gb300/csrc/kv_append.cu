// kv_append.cu -- a chunk's fused QKV rows into a paged cache: per-head norm and
// rotation of queries and keys, keys and values written at their slots in any
// cache form.
//
// Per query and key head x of a row (w and the norm only where w is given):
//   xn = bf16( x w / sqrt(mean x^2 + eps) ),
//   y_i = bf16( xn_i c_i - xn_{i+D/2} s_i ), y_{i+D/2} = bf16( xn_{i+D/2} c_i + xn_i s_i ),
// c + i s = e^{i p theta^{-2i/D}} from the table of hi + lo float pairs, each
// rounding that of the exact value (as the layers' norm_rope_head has it for squares
// in float32's range). Keys and values then are stored as they are, or quantised by
// the row (quant.cu, kv_i4.cu).
//
// What bounds it: HBM, 2 (Hq + 2 Hkv) D bytes of a token in, 2 Hq D and the
// cache's row out. What stands against it is arithmetic: in pairs of floats
// (common.cuh) the norm and rotation take about 60 instructions an element. So
// they run in float32 with a bound on how far the result is from the exact one:
// both ends of that interval are rounded, and where they agree this is the exact
// value's rounding (rotated values from 2^-100; below, the last bit may differ).
// Otherwise the one value is done again in pairs.
//   norm: every x^2 is exact, and so is x w; of the root's argument the 7 roundings
//     of the sum and the one of eps count half, then come the root's own, the
//     product's and the interval's: 7 x 2^-24 of the value, 8 taken;
//   rotation: two products, the table's two lo parts, the sum and the interval's
//     ends: 4 x 2^-24 (|xn c| + |xn' s|) and what is beyond first order, 4.2 taken.
//
// A head belongs to D / 8 lanes of 8 values, four of either half, so that a
// rotation's two values are in one lane. A warp takes the heads of one token in turns, its sines
// and cosines in registers; how many turns a warp takes depends on the number of
// tokens (launch).
//
// Measured (GB300, a graph's launch): 16384 tokens of 40 / 8 heads of 128, BF16: 130 us,
// 3.7 TB/s of 6.8 that a copy reaches (INT8 154, 4-bit 144); some 250 instructions a turn of
// 256 values keep the issue slots 70 % busy. 64 tokens: 4.7 us, one: 2.6. A zero takes its
// lane's eight values past the float32 form: with one in most heads the 16384 tokens take 436 us.
#include <algorithm>

#include "kernels.cuh"
#include "quant_i4.cuh"

namespace a8w8 {

namespace {

constexpr int kThreads = 128;
constexpr int kFill = 32;              // warps a multiprocessor, at least, before a warp takes a second turn
// Largest relative distance of the normed value's interval ends from the float32 one,
// and of a rotated value's from |xn c| + |xn' s|: the counts of the comment above.
constexpr float kNormErr = 8.0f / (1 << 24), kRotErr = 4.2f / (1 << 24);
constexpr unsigned kErrSlot = 0x1u, kErrPos = 0x10u;

template <int LPR>
__device__ __forceinline__ f2 row_sum_f2(f2 v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
        f2 t;
        t.hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
        t.lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
        v = f2_add(v, t);
    }
    return v;
}

// Value e of 8, and its place taken by the BF16 bits r.
__device__ __forceinline__ float value(const int4& v, int e) {
    const int i = e >> 1, w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return __uint_as_float((unsigned)w >> (16 * (e & 1)) << 16);
}
__device__ __forceinline__ void put(int4& v, int e, bf16 r) {
    const int i = e >> 1, sh = 16 * (e & 1), keep = ~(0xFFFF << sh), to = __bfloat16_as_ushort(r) << sh;
    if (i == 0) v.x = (v.x & keep) | to;
    if (i == 1) v.y = (v.y & keep) | to;
    if (i == 2) v.z = (v.z & keep) | to;
    if (i == 3) v.w = (v.w & keep) | to;
}
// The values of mask `differ` (16 bits each, those that are not zero) as a mask of 8 bits.
__device__ __forceinline__ unsigned open_of(const unsigned (&differ)[4]) {
    unsigned open = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) open |= (differ[e >> 1] >> (16 * (e & 1)) & 0xFFFFu ? 1u : 0u) << e;
    return open;
}

// Of the lane's 8 values of a head (four at w, four at w + D / 2 of the weights) those
// in `open` normed in pairs of floats, in place of those in y. Every lane of the warp
// calls this.
template <int D>
__device__ __noinline__ int4 norm_exact(int4 raw, int4 y, unsigned open, const bf16* w, float eps) {
    float x[8];
    unpack8(raw, x);
    f2 ss = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) f2_acc(ss, __fmul_rn(x[e], x[e]));
    const f2 inv = rms_inv(row_sum_f2<D / 8>(ss), D, eps);
#pragma unroll 1
    for (; open; open &= open - 1) {
        const int e = __ffs(open) - 1;
        put(y, e, norm_bf16(value(raw, e), bf2f(w[(e & 3) + (e >> 2) * (D / 2)]), inv));
    }
    return y;
}

// An overflow of pairs of floats is NaN: r, or where it is not finite the float's value.
__device__ __forceinline__ bf16 finite_or(bf16 r, float plain) {
    return (__bfloat16_as_ushort(r) & 0x7F80u) == 0x7F80u ? f2bf(plain) : r;
}

// The same for heads whose squares, or products with a weight, leave float32's range: the
// head and eps in units that bring the largest |x| to about 1 and eps to 4 at most.
// Beside an infinity, every finite value norms to zero.
template <int D>
__device__ __noinline__ int4 norm_far(int4 raw, int4 y, unsigned open, const bf16* w, float eps) {
    float x[8];
    unpack8(raw, x);
    unsigned top = 0u;                   // the largest |x|, as bits: NaN is above infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    int unit = (int)(top >> 23) - 126;
    if (eps > 0.0f) unit = max(unit, ((int)(__float_as_uint(eps) >> 23) - 127) >> 1);
    const float up = __uint_as_float((unsigned)(127 - min(max(unit, -126), 126)) << 23);
    f2 ss = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) f2_acc(ss, __fmul_rn(__fmul_rn(x[e], up), __fmul_rn(x[e], up)));
    f2 inv = rms_inv(row_sum_f2<D / 8>(ss), D, __fmul_rn(__fmul_rn(eps, up), up));
    if (top == 0x7F800000u) inv = f2{0.0f, 0.0f};
#pragma unroll 1
    for (; open; open &= open - 1) {
        const int e = __ffs(open) - 1;
        const f2 v = f2_mulf(inv, __fmul_rn(value(raw, e), up));
        const float we = bf2f(w[(e & 3) + (e >> 2) * (D / 2)]);
        put(y, e, finite_or(f2_to_bf16(f2_mulf(v, we)), __fmul_rn(v.hi, we)));
    }
    return y;
}

// Of the lane's 8 values x those in `open` rotated in pairs of floats, in place of
// those in y. `rope` is the lane's first angle in the position's row of the table.
template <int D>
__device__ __noinline__ int4 rotate_exact(int4 x, int4 y, unsigned open, const float* rope) {
#pragma unroll 1
    for (; open; open &= open - 1) {
        const int e = __ffs(open) - 1;
        const float* t = rope + (e & 3);
        const float xa = value(x, e), xb = value(x, e ^ 4);
        const f2 a = f2_mulf(f2{t[0], t[D]}, xa), b = f2_mulf(f2{t[D / 2], t[3 * D / 2]}, xb);
        put(y, e, finite_or(f2_to_bf16(e & 4 ? f2_add(a, b) : f2_sub(a, b)),
                            e & 4 ? t[0] * xa + t[D / 2] * xb : t[0] * xa - t[D / 2] * xb));
    }
    return y;
}

__device__ __forceinline__ void unpack_pairs(const int4& v, f32x2 (&f)[4]) {
    float x[8];
    unpack8(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(x[2 * i], x[2 * i + 1]);
}
// Whether some |weight| is 2^59 or more: of a head whose sum of squares is finite, |x|
// is below 2^64.
__device__ __forceinline__ bool far_weights(const int4& w) {
    const unsigned a = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    return max(a >> 16, a & 0xFFFFu) >= (127u + 59u) << 7;
}
__device__ __forceinline__ unsigned bf16x2(f32x2 v) {
    float a, b;
    split(v, a, b);
    return as_u32(__floats2bfloat162_rn(a, b));
}

// The lane's 8 values of a head, normed (with w, where the mean square is from 10^-12 to
// `limit` by this) and rotated: in float32, both ends of the interval that holds the
// exact value rounded to BF16, and where those differ by the above.
template <int D>
__device__ __forceinline__ int4 rotate(int4 raw, const bf16* w, const f32x2 (&wf)[4], float limit, float eps,
                                       const float* rope, const f32x2 (&c)[2], const f32x2 (&s)[2]) {
    constexpr int LPR = D / 8;
    f32x2 x[4];
    unpack_pairs(raw, x);
    int4 xn = raw;
    if (__any_sync(0xffffffffu, w != nullptr)) {       // (the lanes of two heads may differ)
        float ss, s1;
        split(add2(fma2(x[0], x[0], mul2(x[1], x[1])), fma2(x[2], x[2], mul2(x[3], x[3]))), ss, s1);
        ss += s1;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float square = __fmaf_rn(ss, 1.0f / D, eps), inv = __frsqrt_rn(square);
        unsigned open = 0u;
        const bool in = square > 1e-12f && square < limit;
        if (w) {
            const float lo = inv * (1.0f - kNormErr), hi = inv * (1.0f + kNormErr);
            const f32x2 lo2 = pair(lo, lo), hi2 = pair(hi, hi);
            unsigned o[4], differ[4];
            float small = INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 t = mul2(x[e], wf[e]);
                float a, b;
                split(t, a, b);
                small = fminf(fminf(small, fabsf(a)), fabsf(b));
                o[e] = bf16x2(mul2(t, lo2));
                differ[e] = o[e] ^ bf16x2(mul2(t, hi2));
            }
            xn = make_int4(o[0], o[1], o[2], o[3]);
            // (products out of the normal numbers' range have other errors; zeros among them,
            // which are exact, come here too)
            if ((small < 1e-17f && ss != 0.0f) || !in) open = 0xFFu;
            else if ((differ[0] | differ[1]) | (differ[2] | differ[3])) open = open_of(differ);
        }
        if (__any_sync(0xffffffffu, open != 0u))
            xn = __all_sync(0xffffffffu, in) ? norm_exact<D>(raw, xn, open, w, eps) : norm_far<D>(raw, xn, open, w, eps);
        unpack_pairs(xn, x);
    }
    const f32x2 up = pair(kRotErr, kRotErr), down = pair(-kRotErr, -kRotErr), minus = pair(-1.0f, -1.0f);
    unsigned o[4], differ[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // x c - x' s of the lower half, x c + x' s of the upper one
        const f32x2 a = mul2(x[e], c[e & 1]), b = mul2(x[e ^ 2], s[e & 1]), r = e < 2 ? fma2(b, minus, a) : add2(a, b);
        float a0, a1, b0, b1;
        split(a, a0, a1);
        split(b, b0, b1);
        const f32x2 size = pair(fabsf(a0) + fabsf(b0), fabsf(a1) + fabsf(b1));
        o[e] = bf16x2(fma2(size, up, r));
        differ[e] = o[e] ^ bf16x2(fma2(size, down, r));
    }
    int4 y = make_int4(o[0], o[1], o[2], o[3]);
    if ((differ[0] | differ[1]) | (differ[2] | differ[3])) y = rotate_exact<D>(xn, y, open_of(differ), rope);
    return y;
}

// The lane's 8 values of a row, four of either half from 4 j on, into the cache, rows
// of LPR lanes; nothing is written without `live`.
template <int D>
__device__ __forceinline__ void store_halves(bf16* to, int4 v) {
    *reinterpret_cast<int2*>(to) = make_int2(v.x, v.y);
    *reinterpret_cast<int2*>(to + D / 2) = make_int2(v.z, v.w);
}

template <int D, int KV>
__device__ __forceinline__ void store_row(int4 v, void* rows, void* scales, size_t at, int j, bool live) {
    constexpr int LPR = D / 8;
    if (KV == kKvBf16) {
        if (live) store_halves<D>(static_cast<bf16*>(rows) + at * D + 4 * j, v);
    } else if (KV == kKvI8) {
        float x[8];
        unpack8(v, x);
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float sc = __fdiv_rn(top, 127.0f), rc = quant_recip(sc);
        unsigned lo = 0u, hi = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo |= (unsigned)(quant_code(x[e], sc, rc) & 0xFF) << (8 * e);
            hi |= (unsigned)(quant_code(x[4 + e], sc, rc) & 0xFF) << (8 * e);
        }
        if (live) {
            unsigned* to = static_cast<unsigned*>(rows) + at * (D / 4) + j;
            to[0] = lo;
            to[D / 8] = hi;
            if (j == 0) static_cast<float*>(scales)[at] = sc;
        }
    } else {
        const int4 raw[1] = {v};
        unsigned code[1];
        const unsigned meta = quant_row_i4<LPR, 1>(raw, code);
        if (live) {
            unsigned short* to = static_cast<unsigned short*>(rows) + at * (D / 4) + j;
            to[0] = (unsigned short)code[0];
            to[D / 8] = (unsigned short)(code[0] >> 16);
            if (j == 0) static_cast<unsigned*>(scales)[at] = meta;
        }
    }
}

// Warp w takes `turns` turns of 32 / (D / 8) heads of token w / per.
template <int D, int KV>
__global__ void __launch_bounds__(kThreads, 7) kv_append_kernel(const AppendParams p, int turns, int per) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    pdl_wait();
    pdl_trigger();
    const unsigned warp = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, j = lane % LPR;
    const unsigned t = warp / (unsigned)per;
    if (t >= (unsigned)p.T) return;
    const int part = (int)(warp - t * per);
    int pos = __ldcg(p.positions + t);
    long slot = __ldcg(p.slot_mapping + t);
    if (part == 0 && lane == 0) {
        if (pos >= p.max_pos) set_error(p.err, kErrPos);
        if (slot >= p.num_slots) set_error(p.err, kErrSlot);
    }
    const bool token = pos >= 0 && pos < p.max_pos;
    if (!token) pos = 0;
    const bool write = token && slot >= 0 && slot < p.num_slots;
    const float* rope = p.rope + (size_t)pos * 2 * D + 4 * j;
    const int first = p.q_out ? 0 : p.Hq, all = p.Hq + 2 * p.Hkv;
    const int h0 = first + part * turns * RPW, h1 = min(all, h0 + turns * RPW);
    const float4 ca = *reinterpret_cast<const float4*>(rope);
    const float4 sa = *reinterpret_cast<const float4*>(rope + D / 2);
    const f32x2 c[2] = {pair(ca.x, ca.y), pair(ca.z, ca.w)}, s[2] = {pair(sa.x, sa.y), pair(sa.z, sa.w)};
    auto halves = [](const int2& a, const int2& b) { return make_int4(a.x, a.y, b.x, b.y); };
    const bf16* row = p.qkv + (size_t)t * p.ld + 4 * j;
    auto load = [&](int h) {
        const int at = min(h + lane / LPR, all - 1);
        const int2* from = reinterpret_cast<const int2*>(row + (size_t)at * D);
        return halves(__ldcs(from), __ldcs(from + D / 8));
    };
    const bf16 *wq = p.q_norm_w ? p.q_norm_w + 4 * j : nullptr, *wk = p.k_norm_w ? p.k_norm_w + 4 * j : nullptr;
    f32x2 wf[4];
    const bf16* w = nullptr;
    float limit = 3e38f;                 // of the mean square, 0 for far weights
    int kind = -1;                       // of the heads that w belongs to: queries, keys
    int4 next = load(h0);
#pragma unroll 1
    for (int h = h0; h < h1; h += RPW) {
        int4 v = next;
        if (h + RPW < h1) next = load(h + RPW);
        const int at = h + lane / LPR;
        const bool in = at < h1;
        // A turn's heads may be of two kinds: rows are rotated where any is a query or key,
        // and each takes its own weights.
        if (h < p.Hq + p.Hkv && token) {
            const int mine = at < p.Hq ? 0 : 1;
            if (mine != kind) {
                kind = mine;
                w = mine ? wk : wq;
                if (w) {
                    const int2* from = reinterpret_cast<const int2*>(w);
                    const int4 packed = halves(from[0], from[D / 8]);
                    unpack_pairs(packed, wf);
                    limit = far_weights(packed) ? 0.0f : 3e38f;
                }
            }
            const int4 y = rotate<D>(v, w, wf, limit, p.eps, rope, c, s);
            if (at < p.Hq + p.Hkv) v = y;
        }
        if (at < p.Hq) {
            if (in) {
                if (!token) v = make_int4(0, 0, 0, 0);
                store_halves<D>(p.q_out + ((size_t)t * p.Hq + at) * D + 4 * j, v);
            }
        }
        if (h + RPW > p.Hq) {             // some row of the turn goes to the cache
            const bool key = at < p.Hq + p.Hkv;
            const int kvh = at - p.Hq - (key ? 0 : p.Hkv);
            const size_t to = (size_t)(write ? slot : 0) * p.Hkv + max(kvh, 0);
            store_row<D, KV>(v, key ? p.k : p.v, key ? p.k_scale : p.v_scale, to, j,
                             write && in && at >= p.Hq);
        }
    }
}

template <int D, int KV>
cudaError_t launch(const AppendParams& p, const Launch& L) {
    constexpr int RPW = 32 / (D / 8);
    const int heads = (p.q_out ? p.Hq : 0) + 2 * p.Hkv;
    const int all = (heads + RPW - 1) / RPW;
    // turns a warp: all of a token's where there are warps enough to fill the SMs, fewer
    // where tokens are few
    const long fill = (long)L.num_sms * kFill;
    const int turns = (int)std::min<long>(all, std::max<long>(1, (long)p.T * all / fill));
    const int per = (all + turns - 1) / turns;
    const long warps = (long)p.T * per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<D, KV>, p, turns, per);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, const Launch& L) {
    if (p.T <= 0) return cudaSuccess;
    if (p.D == 128)
        return p.kv == kKvBf16 ? launch<128, kKvBf16>(p, L)
               : p.kv == kKvI8 ? launch<128, kKvI8>(p, L) : launch<128, kKvI4>(p, L);
    if (p.D == 64)
        return p.kv == kKvBf16 ? launch<64, kKvBf16>(p, L)
               : p.kv == kKvI8 ? launch<64, kKvI8>(p, L) : launch<64, kKvI4>(p, L);
    return cudaErrorInvalidValue;
}

}  // namespace a8w8
