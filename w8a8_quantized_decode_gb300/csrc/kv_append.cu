// kv_append.cu -- a chunk's fused QKV rows into a paged cache: per-head norm and
// rotation of queries and keys, keys and values written at their slots in any
// cache form.
//
// Per query and key head x of a row (w and the norm only where w is given):
//   xn = bf16( x w / sqrt(mean x^2 + eps) ),
//   y_i = bf16( xn_i c_i - xn_{i+D/2} s_i ), y_{i+D/2} = bf16( xn_{i+D/2} c_i + xn_i s_i ),
// c + i s = e^{i p theta^{-2i/D}} from the table of hi + lo float pairs, each
// rounding that of the exact value (as the layers' norm_rope_head). Keys and
// values then are stored as they are, or quantised by the row (quant.cu,
// kv_i4.cu).
//
// What bounds it: HBM, 2 (Hq + 2 Hkv) D bytes of a token in, 2 Hq D and the
// cache's row out. What stands against it is arithmetic: in pairs of floats
// (common.cuh) the norm and rotation take about 60 instructions an element. So
// they run in float32 first, with a bound on how far the result is from the
// exact one: where no boundary between two BF16 values lies that near, its
// rounding is the exact value's. Otherwise (some 6 % of a warp's turns) the
// warp's heads are done again in pairs.
//   norm: every x^2 is exact, and so is x w; of the root's argument the 7 roundings
//     of the sum and the one of eps count half, then come the root's own and the
//     product's: 6 x 2^-24 of the value, 6 units in the last place at most;
//   rotation: two products, the table's two lo parts and the sum, together 3 x
//     2^-24 (|xn c| + |xn' s|), and one more for the ends of the interval.
//
// A head belongs to D / 8 lanes of 8 values; a rotation's partner value is in the
// lane half a head away. A warp takes the heads of one token in turns, its sines
// and cosines in registers; how many turns a warp takes depends on the number of
// tokens (launch).
#include <algorithm>

#include "kernels.cuh"
#include "quant_i4.cuh"

namespace a8w8 {

namespace {

constexpr int kThreads = 128;
constexpr int kFill = 32;              // warps a multiprocessor, at least, before a warp takes a second turn
constexpr unsigned kErrSlot = 0x1u, kErrPos = 0x10u;

// Whether the normed v of x, at most 6 units in its last place from the exact
// value, is too near a midpoint between BF16 values (low half 0x8000) to be
// rounded, not finite, or so small (2^-67) that a product on its way may have
// been below the normal numbers.
__device__ __forceinline__ bool near_midpoint(float v, float x) {
    const unsigned u = __float_as_uint(v), ex = (u >> 23) & 255u;
    return (u & 0xFFFFu) - 0x7FF9u <= 14u || (ex - 60u >= 195u && x != 0.0f);
}
// r of the exact value within e: its BF16 bits, and whether e leaves them open.
__device__ __forceinline__ unsigned round_within(float r, float e, bool& open) {
    const unsigned both = as_u32(__floats2bfloat162_rn(r - e, r + e));
    open |= (both >> 16) != (both & 0xFFFFu);
    return both & 0xFFFFu;
}

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

// The lane's 8 values of a head, normed and rotated in pairs of floats. `rope` is
// the position's row of the table, i0 the lane's first angle, upper whether it
// holds the head's upper half. Every lane of the warp calls this.
template <int D>
__device__ __noinline__ int4 rotate_exact(int4 raw, const bf16* w, float eps, const float* rope, int i0,
                                          bool upper) {
    constexpr int LPR = D / 8;
    float x[8];
    unpack8(raw, x);
    if (__any_sync(0xffffffffu, w != nullptr)) {
        f2 ss = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 8; ++e) f2_acc(ss, __fmul_rn(x[e], x[e]));
        const f2 inv = rms_inv(row_sum_f2<LPR>(ss), D, eps);
        if (w) {
            float wf[8];
            unpack8(ld_nc_v4(w), wf);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = bf2f(norm_bf16(x[e], wf[e], inv));
        }
    }
    unsigned o[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float partner = __shfl_xor_sync(0xffffffffu, x[e], LPR / 2);
        const float* t = rope + i0 + e;
        const f2 a = f2_mulf(f2{__ldg(t), __ldg(t + D)}, x[e]);
        const f2 b = f2_mulf(f2{__ldg(t + D / 2), __ldg(t + 3 * D / 2)}, partner);
        const bf16 y = f2_to_bf16(upper ? f2_add(a, b) : f2_sub(a, b));
        o[e >> 1] |= (unsigned)__bfloat16_as_ushort(y) << (16 * (e & 1));
    }
    return make_int4(o[0], o[1], o[2], o[3]);
}

// The same in float32 where its bounds decide every rounding, otherwise by the above.
template <int D>
__device__ __forceinline__ int4 rotate(int4 raw, const bf16* w, const float (&wf)[8], float eps,
                                       const float* rope, const float (&c)[8], const float (&s)[8], int i0,
                                       bool upper) {
    constexpr int LPR = D / 8;
    float x[8];
    unpack8(raw, x);
    bool open = false;
    int4 xn = raw;
    if (__any_sync(0xffffffffu, w != nullptr)) {       // (the lanes of two heads may differ)
        float ss = ((x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3])) +
                   ((x[4] * x[4] + x[5] * x[5]) + (x[6] * x[6] + x[7] * x[7]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float square = __fmaf_rn(ss, 1.0f / D, eps), inv = __frsqrt_rn(square);
        if (w) {
            open = square < 1e-30f;
            unsigned o[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float a = x[e] * wf[e] * inv, b = x[e + 1] * wf[e + 1] * inv;
                open |= near_midpoint(a, x[e]) | near_midpoint(b, x[e + 1]);
                o[e >> 1] = as_u32(__floats2bfloat162_rn(a, b));
            }
            xn = make_int4(o[0], o[1], o[2], o[3]);
            unpack8(xn, x);
        }
    }
    int4 other;
    other.x = __shfl_xor_sync(0xffffffffu, xn.x, LPR / 2);
    other.y = __shfl_xor_sync(0xffffffffu, xn.y, LPR / 2);
    other.z = __shfl_xor_sync(0xffffffffu, xn.z, LPR / 2);
    other.w = __shfl_xor_sync(0xffffffffu, xn.w, LPR / 2);
    float z[8];
    unpack8(other, z);
    unsigned o[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // s carries the sign of the lane's half
        const float a = x[e] * c[e], b = z[e] * s[e], size = fabsf(a) + fabsf(b);
        open |= size < 1e-30f && size != 0.0f;
        o[e >> 1] |= round_within(a + b, size * 3e-7f, open) << (16 * (e & 1));
    }
    if (__any_sync(0xffffffffu, open)) return rotate_exact<D>(raw, w, eps, rope, i0, upper);
    return make_int4(o[0], o[1], o[2], o[3]);
}

// The lane's 8 values of a row into the cache, rows of LPR lanes; nothing is written without `live`.
template <int D, int KV>
__device__ __forceinline__ void store_row(int4 v, void* rows, void* scales, size_t at, int j, bool live) {
    constexpr int LPR = D / 8;
    if (KV == kKvBf16) {
        if (live) *reinterpret_cast<int4*>(static_cast<bf16*>(rows) + at * D + 8 * j) = v;
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
            *reinterpret_cast<uint2*>(static_cast<int8_t*>(rows) + at * D + 8 * j) = make_uint2(lo, hi);
            if (j == 0) static_cast<float*>(scales)[at] = sc;
        }
    } else {
        const int4 raw[1] = {v};
        unsigned code[1];
        const unsigned meta = quant_row_i4<LPR, 1>(raw, code);
        if (live) {
            static_cast<unsigned*>(rows)[at * LPR + j] = code[0];
            if (j == 0) static_cast<unsigned*>(scales)[at] = meta;
        }
    }
}

// Warp w takes `turns` turns of 32 / (D / 8) heads of token w / per.
template <int D, int KV>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p, int turns, int per) {
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
    const bool upper = j >= LPR / 2;
    const int i0 = 8 * (j % (LPR / 2));
    const float* rope = p.rope + (size_t)pos * 2 * D;
    const int first = p.q_out ? 0 : p.Hq, all = p.Hq + 2 * p.Hkv;
    const int h0 = first + part * turns * RPW, h1 = min(all, h0 + turns * RPW);
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(rope + i0 + e));
        const float4 b = __ldg(reinterpret_cast<const float4*>(rope + D / 2 + i0 + e));
        c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
        s[e] = b.x, s[e + 1] = b.y, s[e + 2] = b.z, s[e + 3] = b.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = upper ? s[e] : -s[e];
    const bf16* row = p.qkv + (size_t)t * p.ld + 8 * j;
    auto load = [&](int h) {
        const int at = min(h + lane / LPR, all - 1);
        return __ldcs(reinterpret_cast<const int4*>(row + (size_t)at * D));
    };
    const bf16 *wq = p.q_norm_w ? p.q_norm_w + 8 * j : nullptr, *wk = p.k_norm_w ? p.k_norm_w + 8 * j : nullptr;
    float wf[8];
    const bf16* w = nullptr;
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
        if (h < p.Hq + p.Hkv) {
            const int mine = at < p.Hq ? 0 : 1;
            if (mine != kind) {
                kind = mine;
                w = mine ? wk : wq;
                if (w) unpack8(ld_nc_v4(w), wf);
            }
            const int4 y = rotate<D>(v, w, wf, p.eps, rope, c, s, i0, upper);
            if (at < p.Hq + p.Hkv) v = y;
        }
        if (at < p.Hq) {
            if (in) {
                if (!token) v = make_int4(0, 0, 0, 0);
                *reinterpret_cast<int4*>(p.q_out + ((size_t)t * p.Hq + at) * D + 8 * j) = v;
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
