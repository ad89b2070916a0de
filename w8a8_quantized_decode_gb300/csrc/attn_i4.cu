// attn_i4.cu -- GQA decode attention over the 4-bit paged KV cache.
//
// K_t = c s + m of the token's row (kv_i4.cu), so score_t = scale (s sum_d q_d
// c_d + m sum_d q_d), and out = sum_t p_t V_t / sum_t p_t with p_t =
// exp(score_t - max), in float32, narrowed to BF16 once.
#include "kernels.cuh"

namespace a8w8 {

namespace {

constexpr int kI4Warps = 4;

// One CTA per (query head, request); a warp takes every fourth token, a lane
// D / 32 elements, with the running maximum and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(32 * kI4Warps) attn_i4_kernel(const AttnI4Params p) {
    constexpr int E = D / 32;
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x, b = blockIdx.y;
    const int kvh = h / (p.Hq / p.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int ctx = p.ctx_lens[b];
    if (ctx < 0 || ctx > p.max_blocks * p.page) {
        if (threadIdx.x == 0) set_error(p.err, 0x4u);
        ctx = 0;
    }
    float q[E], o[E], qs = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf2f(p.q[((size_t)b * p.Hq + h) * D + lane * E + e]) * p.scale;
        qs += q[e];
        o[e] = 0.0f;
    }
    qs = warp_sum(qs);
    float m = -INFINITY, l = 0.0f;
    for (int t = warp; t < ctx; t += kI4Warps) {
        const int blk = p.block_table[(size_t)b * p.max_blocks + t / p.page];
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!ok && lane == 0) set_error(p.err, 0x2u);
        float kc[E], vc[E], s = 0.0f;
        float2 km = {0.0f, 0.0f}, vm = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) kc[e] = vc[e] = 0.0f;
        if (ok) {
            const size_t row = ((size_t)blk * p.page + t % p.page) * p.Hkv + kvh;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = lane * E + e;
                kc[e] = (float)((p.c.k_codes[row * (D / 2) + d / 2] >> (4 * (d & 1))) & 15);
                vc[e] = (float)((p.c.v_codes[row * (D / 2) + d / 2] >> (4 * (d & 1))) & 15);
            }
            km = {bf2f(p.c.k_meta[2 * row]), bf2f(p.c.k_meta[2 * row + 1])};
            vm = {bf2f(p.c.v_meta[2 * row]), bf2f(p.c.v_meta[2 * row + 1])};
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * kc[e];
        s = warp_sum(s) * km.x + qs * km.y;
        const float mn = fmaxf(m, s);
        const float f = expf(m - mn), w = expf(s - mn);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * (vc[e] * vm.x + vm.y);
        m = mn;
    }
    __shared__ float so[kI4Warps][D], sm[kI4Warps], sl[kI4Warps];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * kI4Warps) {
        float mx = -INFINITY, L = 0.0f, O = 0.0f;
        for (int w = 0; w < kI4Warps; ++w) mx = fmaxf(mx, sm[w]);
        for (int w = 0; w < kI4Warps && ctx > 0; ++w) {
            if (w >= ctx) break;
            const float f = expf(sm[w] - mx);
            L += sl[w] * f;
            O += so[w][d] * f;
        }
        p.out[((size_t)b * p.Hq + h) * D + d] = f2bf(ctx > 0 ? O / L : 0.0f);
    }
}

}  // namespace

size_t attn_i4_part_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_attention_i4(const AttnI4Params& p, const Launch& L) {
    if (p.B == 0) return cudaSuccess;
    if (p.D != 64 && p.D != 128) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.Hq, p.B);
    cfg.blockDim = dim3(32 * kI4Warps);
    cfg.stream = L.stream;
    return cudaLaunchKernelEx(&cfg, p.D == 128 ? attn_i4_kernel<128> : attn_i4_kernel<64>, p);
}

}  // namespace a8w8
