// quant_i4.cuh -- a row of the 4-bit KV cache from its BF16 values (the form is
// described in kv_i4.cu).
#pragma once

#include "common.cuh"

namespace a8w8 {

__device__ __forceinline__ __nv_bfloat162 as_bf162(unsigned u) {
    return *reinterpret_cast<__nv_bfloat162*>(&u);
}
__device__ __forceinline__ unsigned as_u32(__nv_bfloat162 h) {
    return *reinterpret_cast<unsigned*>(&h);
}

// The row's (s, m) word and the lane's codes. LPR lanes hold the row, P pieces of
// eight values each; every lane of the warp calls this.
template <int LPR, int P>
__device__ __forceinline__ unsigned quant_row_i4(const int4 (&raw)[P], unsigned (&codes)[P]) {
    // maximum and negated minimum side by side, NaN taken over
    __nv_bfloat162 mx = as_bf162(raw[0].x), mn = mx;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = i == 0 ? 1 : 0; j < 4; ++j) {
            mx = __hmax2_nan(mx, as_bf162(w[j]));
            mn = __hmin2_nan(mn, as_bf162(w[j]));
        }
    }
    __nv_bfloat162 r = __halves2bfloat162(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx)),
                                          __hneg(__hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn))));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        r = __hmax2_nan(r, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    const float top = __bfloat162float(__low2bfloat16(r));
    const __nv_bfloat16 mb = __hneg(__high2bfloat16(r));
    const float m = __bfloat162float(mb);
    const float range = __fsub_rn(top, m);
#pragma unroll
    for (int i = 0; i < P; ++i) codes[i] = 0u;
    if (!isfinite(range)) return 0x7FC07FC0u;   // NaN, NaN
    // Quotients without a division: the float product with R = RN(1 / y) and
    // one correction by the exact remainder (as quant_code in common.cuh),
    // where neither R nor the remainder leaves the normal range.
    constexpr float kR15 = 1.0f / 15.0f;
    const bool plain = !(range >= 1.6e-29f && range <= 1.2e30f);   // about 2^-96, 2^100
    float sf;
    if (plain) {
        sf = __fdiv_rn(range, 15.0f);
    } else {
        sf = __fmul_rn(range, kR15);
        sf = __fmaf_rn(__fmaf_rn(-sf, 15.0f, range), kR15, sf);
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(sf);
    const float s = __bfloat162float(sb);
    const unsigned meta = as_u32(__halves2bfloat162(sb, mb));
    if (s == 0.0f) return meta;
    float x[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) unpack8(raw[i], x[i]);
    if (plain) {
#pragma unroll
        for (int e = 0; e < 8 * P; ++e) {
            const float q = fminf(__fdiv_rn(__fsub_rn(x[e / 8][e % 8], m), s), 15.0f);
            codes[e / 8] |= (unsigned)__float2int_rn(q) << (4 * (e % 8));
        }
        return meta;
    }
    // The quotient is at most 15 (1 + 2^-8) here, so its rounding needs no
    // clamp: adding 2^23 leaves rne(q) in the low bits, and eight of them join
    // by multiply-adds, the exponents' bits adding up to a constant.
    const float R = __frcp_rn(s);
    const f32x2 ms = pair(-m, -m), ns = pair(-s, -s), Rs = pair(R, R),
                big = pair(8388608.0f, 8388608.0f);
    unsigned acc[P] = {};
#pragma unroll
    for (int e = 6; e >= 0; e -= 2)
#pragma unroll
        for (int h = 0; h < P; ++h) {
            const f32x2 d = add2(pair(x[h][e], x[h][e + 1]), ms);
            const f32x2 q0 = mul2(d, Rs);
            float lo, hi;
            split(add2(fma2(fma2(q0, ns, d), Rs, q0), big), lo, hi);
            acc[h] = (acc[h] * 16u + __float_as_uint(hi)) * 16u + __float_as_uint(lo);
        }
#pragma unroll
    for (int h = 0; h < P; ++h) codes[h] = acc[h] - 0xFB000000u;
    return meta;
}

}  // namespace a8w8
