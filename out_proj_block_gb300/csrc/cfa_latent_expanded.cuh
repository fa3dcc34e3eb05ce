// cfa_latent_expanded.cuh -- attention of prompts over expanded keys and values.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  m = max_j s_j,
//   s_j = scale log2(e) (q_nope . k_j + q_rope . k_rope_j);  lse = (m + log2 sum_j w_j) ln 2
//
// A warp for a token's head goes over its keys one by one.
#pragma once

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_tile.cuh"

namespace cfa {

// Offsets that are in order within [0, n]; by all threads of the block.
__device__ __forceinline__ bool latent_offsets_ok(const int *cu, int B, int n) {
    bool bad = false;
    for (int b = threadIdx.x; b <= B; b += blockDim.x) {
        const int c = __ldcg(cu + b), before = b > 0 ? __ldcg(cu + b - 1) : 0;
        bad |= c < before || c > n;
    }
    return !__syncthreads_or(bad);
}

// The request of token t, or -1.
__device__ __forceinline__ int latent_request(const int *cu, int B, int t) {
    int lo = 0, hi = B;  // first request whose end is above t
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (__ldcg(cu + mid + 1) > t) hi = mid;
        else lo = mid + 1;
    }
    return lo < B && t >= __ldcg(cu + lo) ? lo : -1;
}

__global__ void __launch_bounds__(256) latent_expanded_kernel(const __grid_constant__ LatentExpandedParams p) {
    const int t = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    grid_dependency_wait();
    const bool a = latent_offsets_ok(p.cu, p.B, p.T), c = latent_offsets_ok(p.cu_k, p.B, p.S);
    if (!(a && c) && t == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadLengthBit);
    const int b = a && c ? latent_request(p.cu, p.B, t) : -1;
    if (b >= 0 && h < p.H) {
        const int k0 = __ldcg(p.cu_k + b), len = __ldcg(p.cu_k + b + 1) - k0;
        const int see = min(len, len - (__ldcg(p.cu + b + 1) - t) + 1);
        float q[kLatQ / 32], o[kLatV / 32] = {}, m = -INFINITY, l = 0.f;
        const uint16_t *qp = p.q + t * p.q_stride + h * kLatQ;
#pragma unroll
        for (int i = 0; i < kLatQ / 32; ++i) q[i] = bf16_bits(qp[lane + 32 * i]);
        for (int j = 0; j < see; ++j) {
            const uint16_t *kv = p.kv + (k0 + j) * p.kv_stride + h * kLatKv;
            const uint16_t *kr = p.k_rope + (k0 + j) * p.k_rope_stride;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < kLatN / 32; ++i) s = fmaf(q[i], bf16_bits(kv[lane + 32 * i]), s);
#pragma unroll
            for (int i = 0; i < kLatR / 32; ++i) s = fmaf(q[kLatN / 32 + i], bf16_bits(kr[lane + 32 * i]), s);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
            s *= p.scale_log2;
            const float n = fmaxf(m, s), f = n == -INFINITY ? 0.f : n;
            const float g = fast_exp2(m - f), w = fast_exp2(s - f);
            m = n;
            l = l * g + w;
#pragma unroll
            for (int i = 0; i < kLatV / 32; ++i) o[i] = fmaf(w, bf16_bits(kv[kLatN + lane + 32 * i]), o[i] * g);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t *out = p.out + (static_cast<size_t>(t) * p.H + h) * kLatV;
#pragma unroll
        for (int i = 0; i < kLatV / 32; ++i) out[lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
        if (p.lse && lane == 0) p.lse[static_cast<size_t>(t) * p.H + h] = (m + log2f(l)) * 0.69314718055994531f;
    }
    grid_dependents_launch();
}

}  // namespace cfa
