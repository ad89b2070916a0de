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
// BF16 and D + 8 of cache. What stands against it is the issue rate of the
// per-row work (s and its reciprocal, the reduction), which all lanes of a row
// do: a row belongs to D / 16 lanes of 16 values in two 16-byte pieces, half
// the lanes that one piece each would take (95 warp instructions per pair of
// rows of 128 values instead of 147), and the pieces of one load or store lie
// side by side (a lane's two pieces together made half sectors, and the read
// half as long again). K and V of the row are in flight together. 16384 tokens
// of 8 heads of 128, write and read in turn, calls queued: 170 MB in 28.2 us
// (6.0 TB/s, 0.90 of the copy rate); as a replayed graph 30.8.
#include "kernels.cuh"

namespace a8w8 {

namespace {

// Write and read of 16384 tokens 30.8 us as a replayed graph, 32.8 at 256, 39 at
// 64; of 2048 tokens 9.0, 10.3, 8.5.
constexpr int kI4Threads = 128;

__device__ __forceinline__ __nv_bfloat162 as_bf162(unsigned u) {
    return *reinterpret_cast<__nv_bfloat162*>(&u);
}
__device__ __forceinline__ unsigned as_u32(__nv_bfloat162 h) {
    return *reinterpret_cast<unsigned*>(&h);
}

// Sixteen bytes of a row that is read once. Not by the read-only path: the
// kernel that writes the rows may still run when this grid starts.
__device__ __forceinline__ int4 ld_row_v4(const bf16* p) {
    return __ldcs(reinterpret_cast<const int4*>(p));
}

// The row's (s, m) word and the lane's sixteen codes. LPR lanes hold the row,
// sixteen values each; every lane of the warp calls this.
template <int LPR>
__device__ __forceinline__ unsigned quant_row_i4(const int4 (&raw)[2], unsigned (&codes)[2]) {
    // maximum and negated minimum side by side, NaN taken over
    __nv_bfloat162 mx = as_bf162(raw[0].x), mn = mx;
    const int w[7] = {raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        mx = __hmax2_nan(mx, as_bf162(w[i]));
        mn = __hmin2_nan(mn, as_bf162(w[i]));
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
    codes[0] = codes[1] = 0u;
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
    float x[2][8];
    unpack8(raw[0], x[0]);
    unpack8(raw[1], x[1]);
    if (plain) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
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
    unsigned acc[2] = {0u, 0u};
#pragma unroll
    for (int e = 6; e >= 0; e -= 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x2 d = add2(pair(x[h][e], x[h][e + 1]), ms);
            const f32x2 q0 = mul2(d, Rs);
            float lo, hi;
            split(add2(fma2(fma2(q0, ns, d), Rs, q0), big), lo, hi);
            acc[h] = (acc[h] * 16u + __float_as_uint(hi)) * 16u + __float_as_uint(lo);
        }
    codes[0] = acc[0] - 0xFB000000u;
    codes[1] = acc[1] - 0xFB000000u;
    return meta;
}

template <int D>
__global__ void __launch_bounds__(kI4Threads)
    kv_write_i4_kernel(const bf16* k, const bf16* v, int T, int Hkv, const int32_t* slot_mapping,
                       uint8_t* k_codes, uint8_t* v_codes, bf16* k_meta, bf16* v_meta,
                       long num_slots, unsigned* err) {
    constexpr int LPR = D / 16;
    pdl_wait();
    pdl_trigger();
    // token * Hkv + head, at most 2^31 and some
    const unsigned row = blockIdx.x * (kI4Threads / LPR) + threadIdx.x / LPR;
    const int j = threadIdx.x % LPR;
    const unsigned t = row / (unsigned)Hkv, hh = row - t * Hkv;
    long slot = t < (unsigned)T ? (long)__ldcg(slot_mapping + t) : -1;
    int4 kr[2], vr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        kr[i] = vr[i] = make_int4(0, 0, 0, 0);
        if (t < (unsigned)T) {
            kr[i] = ld_row_v4(k + (size_t)row * D + 8 * (j + LPR * i));
            vr[i] = ld_row_v4(v + (size_t)row * D + 8 * (j + LPR * i));
        }
    }
    if (slot >= num_slots) {
        if (j == 0 && hh == 0) set_error(err, 0x1u);
        slot = -1;
    }
    unsigned kc[2], vc[2];
    const unsigned km = quant_row_i4<LPR>(kr, kc);
    const unsigned vm = quant_row_i4<LPR>(vr, vc);
    if (slot < 0) return;
    const size_t dst = (size_t)slot * Hkv + hh;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        reinterpret_cast<unsigned*>(k_codes)[dst * 2 * LPR + j + LPR * i] = kc[i];
        reinterpret_cast<unsigned*>(v_codes)[dst * 2 * LPR + j + LPR * i] = vc[i];
    }
    if (j == 0) {
        reinterpret_cast<unsigned*>(k_meta)[dst] = km;
        reinterpret_cast<unsigned*>(v_meta)[dst] = vm;
    }
}

// Eight values of a row from their codes: c s + m rounded to BF16 once (the
// float32 sum is the one rounding before it; c s is exact). A code joins the
// exponent of 2^23, of which it is the lowest bits.
__device__ __forceinline__ int4 dequant8(unsigned codes, unsigned meta) {
    const float s = __uint_as_float(meta << 16), m = __uint_as_float(meta & 0xFFFF0000u);
    const f32x2 ss = pair(s, s), mm = pair(m, m), big = pair(-8388608.0f, -8388608.0f);
    unsigned o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a = __uint_as_float((codes >> (8 * e) & 15u) | 0x4B000000u);
        const float b = __uint_as_float((codes >> (8 * e + 4) & 15u) | 0x4B000000u);
        float lo, hi;
        split(fma2(add2(pair(a, b), big), ss, mm), lo, hi);
        o[e] = as_u32(__floats2bfloat162_rn(lo, hi));
    }
    return make_int4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kI4Threads)
    kv_read_i4_kernel(const uint8_t* k_codes, const uint8_t* v_codes, const bf16* k_meta,
                      const bf16* v_meta, long num_slots, const int32_t* slot_mapping, int T,
                      int Hkv, bf16* k, bf16* v, unsigned* err) {
    constexpr int LPR = D / 16;
    pdl_wait();
    pdl_trigger();
    const unsigned row = blockIdx.x * (kI4Threads / LPR) + threadIdx.x / LPR;
    const int j = threadIdx.x % LPR;
    const unsigned t = row / (unsigned)Hkv, hh = row - t * Hkv;
    if (t >= (unsigned)T) return;
    const long slot = __ldcg(slot_mapping + t);
    int4 ko[2], vo[2];
    ko[0] = ko[1] = vo[0] = vo[1] = make_int4(0, 0, 0, 0);
    if (slot >= num_slots) {
        if (j == 0 && hh == 0) set_error(err, 0x1u);
    } else if (slot >= 0) {
        const size_t src = (size_t)slot * Hkv + hh;
        unsigned kc[2], vc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kc[i] = __ldcg(reinterpret_cast<const unsigned*>(k_codes) + src * 2 * LPR + j + LPR * i);
            vc[i] = __ldcg(reinterpret_cast<const unsigned*>(v_codes) + src * 2 * LPR + j + LPR * i);
        }
        const unsigned km = __ldcg(reinterpret_cast<const unsigned*>(k_meta) + src);
        const unsigned vm = __ldcg(reinterpret_cast<const unsigned*>(v_meta) + src);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ko[i] = dequant8(kc[i], km);
            vo[i] = dequant8(vc[i], vm);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // streaming stores: the BF16 rows, four times the cache's bytes, leave L2
        // to what is still to be read (30.8 against 32.4 us)
        __stcs(reinterpret_cast<int4*>(k + (size_t)row * D + 8 * (j + LPR * i)), ko[i]);
        __stcs(reinterpret_cast<int4*>(v + (size_t)row * D + 8 * (j + LPR * i)), vo[i]);
    }
}

template <typename Kern, typename... Args>
cudaError_t launch_rows_i4(Kern kern, long rows, int D, const Launch& L, Args... args) {
    const long per = kI4Threads / (D / 16);
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
