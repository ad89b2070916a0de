// kv_i4.cu -- rows into and out of the 4-bit KV cache.
//
// A row is one KV head's D values of one token. It is held as D 4-bit codes
// and one pair (s, m) of BF16:
//   m = min x (a BF16 value, so exact), s = bf16_rne((max x - m) / 15),
//   c = clamp(rne((x - m) / s), 0, 15), s == 0 giving c = 0,
// the differences and quotients in IEEE float32, and stands for c s + m: the
// product is exact in float32 (4 + 8 significant bits). Two codes share a
// byte: element 2j in the low nibble of byte j. Rounding s to BF16 moves the
// row's largest value by at most 15 s 2^-9 (0.03 steps) beside the half step
// of the code, and keeps the pair in one 32-bit word: D / 2 + 4 bytes a row.
// A row that holds a NaN or an infinity, or whose range overflows float32, has
// s = m = NaN and codes 0: it reads as NaN.
//
// Both kernels are bound by HBM: a (token, head) pair of rows is 4 D bytes of
// BF16 and D + 8 of cache. A row belongs to D / 8 lanes of 16 BF16 bytes and
// one 32-bit word of codes each, so every access is a full vector and a
// warp's stores of one row are contiguous; K and V of the row are in flight
// together.
#include "kernels.cuh"

namespace a8w8 {

namespace {

constexpr int kI4Threads = 256;

__device__ __forceinline__ __nv_bfloat162 as_bf162(unsigned u) {
    return *reinterpret_cast<__nv_bfloat162*>(&u);
}
__device__ __forceinline__ unsigned as_u32(__nv_bfloat162 h) {
    return *reinterpret_cast<unsigned*>(&h);
}

// The row's (s, m) word and the lane's eight codes. LPR lanes hold the row,
// eight values each; every lane of the warp calls this.
template <int LPR>
__device__ __forceinline__ unsigned quant_row_i4(const int4& raw, unsigned& codes) {
    const __nv_bfloat162 h0 = as_bf162(raw.x), h1 = as_bf162(raw.y), h2 = as_bf162(raw.z),
                         h3 = as_bf162(raw.w);
    // maximum and negated minimum side by side, NaN taken over
    const __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(h0, h1), __hmax2_nan(h2, h3));
    const __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(h0, h1), __hmin2_nan(h2, h3));
    const __nv_bfloat16 hi = __hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx));
    const __nv_bfloat16 lo = __hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn));
    __nv_bfloat162 r = __halves2bfloat162(hi, __hneg(lo));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        r = __hmax2_nan(r, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    const float top = __bfloat162float(__low2bfloat16(r));
    const __nv_bfloat16 mb = __hneg(__high2bfloat16(r));
    const float m = __bfloat162float(mb);
    const float range = __fsub_rn(top, m);
    codes = 0u;
    if (!isfinite(range)) return 0x7FC07FC0u;   // NaN, NaN
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(range, 15.0f));
    const float s = __bfloat162float(sb);
    const unsigned meta = as_u32(__halves2bfloat162(sb, mb));
    if (s == 0.0f) return meta;
    float x[8];
    unpack8(raw, x);
    if (!(s >= 7.9e-31f && s <= 1.2e30f)) {   // about 2^-100, 2^100: see below
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = __float2int_rn(fminf(__fdiv_rn(__fsub_rn(x[e], m), s), 15.0f));
            codes |= (unsigned)c << (4 * e);
        }
        return meta;
    }
    // x / s without a division: the float quotient by R = RN(1 / s) and one
    // correction by the exact remainder (as quant_code in common.cuh), where
    // neither R nor the remainder leaves the normal range. The quotient is at
    // most 15 (1 + 2^-8) there, so its rounding needs no clamp: adding 2^23
    // leaves rne(q) in the low bits, and eight of them join by multiply-adds,
    // the exponents' bits adding up to a constant.
    const float R = __frcp_rn(s);
    const f32x2 ms = pair(-m, -m), ns = pair(-s, -s), Rs = pair(R, R),
                big = pair(8388608.0f, 8388608.0f);
    unsigned acc = 0u;
#pragma unroll
    for (int e = 6; e >= 0; e -= 2) {
        const f32x2 d = add2(pair(x[e], x[e + 1]), ms);
        const f32x2 q0 = mul2(d, Rs);
        float lo, hi;
        split(add2(fma2(fma2(q0, ns, d), Rs, q0), big), lo, hi);
        acc = (acc * 16u + __float_as_uint(hi)) * 16u + __float_as_uint(lo);
    }
    codes = acc - 0xFB000000u;
    return meta;
}

template <int D>
__global__ void __launch_bounds__(kI4Threads)
    kv_write_i4_kernel(const bf16* __restrict__ k, const bf16* __restrict__ v, int T, int Hkv,
                       const int32_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_codes,
                       uint8_t* __restrict__ v_codes, bf16* __restrict__ k_meta,
                       bf16* __restrict__ v_meta, long num_slots, unsigned* err) {
    constexpr int LPR = D / 8;
    pdl_wait();
    pdl_trigger();
    const long row = ((long)blockIdx.x * kI4Threads + threadIdx.x) / LPR;   // token * Hkv + head
    const int j = threadIdx.x % LPR;
    const bool in = row < (long)T * Hkv;
    const long t = in ? row / Hkv : 0;
    const int hh = (int)(in ? row - t * Hkv : 0);
    long slot = in ? (long)__ldg(slot_mapping + t) : -1;
    if (slot >= num_slots) {
        if (j == 0 && hh == 0) set_error(err, 0x1u);
        slot = -1;
    }
    int4 kr = make_int4(0, 0, 0, 0), vr = kr;
    if (slot >= 0) {
        kr = ld_stream_v4(k + (size_t)row * D + 8 * j);
        vr = ld_stream_v4(v + (size_t)row * D + 8 * j);
    }
    unsigned kc, vc;
    const unsigned km = quant_row_i4<LPR>(kr, kc);
    const unsigned vm = quant_row_i4<LPR>(vr, vc);
    if (slot < 0) return;
    const size_t dst = (size_t)slot * Hkv + hh;
    reinterpret_cast<unsigned*>(k_codes)[dst * LPR + j] = kc;
    reinterpret_cast<unsigned*>(v_codes)[dst * LPR + j] = vc;
    if (j == 0) {
        reinterpret_cast<unsigned*>(k_meta)[dst] = km;
        reinterpret_cast<unsigned*>(v_meta)[dst] = vm;
    }
}

// Eight values of a row from their codes: c s + m rounded to BF16 once (the
// float32 sum is the one rounding before it; c s is exact).
__device__ __forceinline__ int4 dequant8(unsigned codes, unsigned meta) {
    const float s = __uint_as_float(meta << 16), m = __uint_as_float(meta & 0xFFFF0000u);
    unsigned o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __fmaf_rn((float)((codes >> (8 * e)) & 15u), s, m);
        const float b = __fmaf_rn((float)((codes >> (8 * e + 4)) & 15u), s, m);
        o[e] = as_u32(__floats2bfloat162_rn(a, b));
    }
    return make_int4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kI4Threads)
    kv_read_i4_kernel(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes,
                      const bf16* __restrict__ k_meta, const bf16* __restrict__ v_meta,
                      long num_slots, const int32_t* __restrict__ slot_mapping, int T, int Hkv,
                      bf16* __restrict__ k, bf16* __restrict__ v, unsigned* err) {
    constexpr int LPR = D / 8;
    pdl_wait();
    pdl_trigger();
    const long row = ((long)blockIdx.x * kI4Threads + threadIdx.x) / LPR;
    const int j = threadIdx.x % LPR;
    if (row >= (long)T * Hkv) return;
    const long t = row / Hkv;
    const int hh = (int)(row - t * Hkv);
    const long slot = __ldg(slot_mapping + t);
    int4 ko = make_int4(0, 0, 0, 0), vo = ko;
    if (slot >= num_slots) {
        if (j == 0 && hh == 0) set_error(err, 0x1u);
    } else if (slot >= 0) {
        const size_t src = (size_t)slot * Hkv + hh;
        const unsigned kc = __ldcg(reinterpret_cast<const unsigned*>(k_codes) + src * LPR + j);
        const unsigned vc = __ldcg(reinterpret_cast<const unsigned*>(v_codes) + src * LPR + j);
        const unsigned km = __ldcg(reinterpret_cast<const unsigned*>(k_meta) + src);
        const unsigned vm = __ldcg(reinterpret_cast<const unsigned*>(v_meta) + src);
        ko = dequant8(kc, km);
        vo = dequant8(vc, vm);
    }
    *reinterpret_cast<int4*>(k + (size_t)row * D + 8 * j) = ko;
    *reinterpret_cast<int4*>(v + (size_t)row * D + 8 * j) = vo;
}

template <typename Kern, typename... Args>
cudaError_t launch_rows_i4(Kern kern, long rows, int D, const Launch& L, Args... args) {
    const long per = kI4Threads / (D / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per - 1) / per));
    cfg.blockDim = dim3(kI4Threads);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_kv_write_i4(const bf16* k, const bf16* v, int T, int Hkv, int D,
                               const int32_t* slot_mapping, const KvI4& c, long num_slots,
                               unsigned* err, const Launch& L) {
    const long rows = (long)T * Hkv;
    if (rows == 0) return cudaSuccess;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    auto kern = D == 128 ? kv_write_i4_kernel<128> : kv_write_i4_kernel<64>;
    return launch_rows_i4(kern, rows, D, L, k, v, T, Hkv, slot_mapping, c.k_codes, c.v_codes,
                          c.k_meta, c.v_meta, num_slots, err);
}

cudaError_t launch_kv_read_i4(const KvI4& c, long num_slots, const int32_t* slot_mapping, int T,
                              int Hkv, int D, bf16* k, bf16* v, unsigned* err, const Launch& L) {
    const long rows = (long)T * Hkv;
    if (rows == 0) return cudaSuccess;
    if (D != 64 && D != 128) return cudaErrorInvalidValue;
    auto kern = D == 128 ? kv_read_i4_kernel<128> : kv_read_i4_kernel<64>;
    return launch_rows_i4(kern, rows, D, L, c.k_codes, c.v_codes, c.k_meta, c.v_meta, num_slots,
                          slot_mapping, T, Hkv, k, v, err);
}

}  // namespace a8w8
