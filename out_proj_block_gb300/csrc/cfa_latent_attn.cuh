// cfa_latent_attn.cuh -- attention of folded queries over paged latent rows.
//
//   o = sum_j w_j row_j[:512] / sum_j w_j,  w_j = 2^(s_j - m),  s_j = scale log2(e) q . row_j,
//   m = max_j s_j;  lse = (m + log2 sum_j w_j) ln 2
//
// A warp for a token's head goes over its rows one by one.
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

__global__ void __launch_bounds__(256) latent_attention_kernel(const __grid_constant__ LatentAttnParams p) {
    const int t = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    grid_dependency_wait();
    const bool ok = latent_offsets_ok(p.cu, p.B, p.T);
    if (!ok && t == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadLengthBit);
    const int b = ok ? latent_request(p.cu, p.B, t) : -1;
    if (b >= 0 && h < p.H) {
        int len = __ldcg(p.lens + b);
        if (len < 0 || len > static_cast<long long>(p.width) * p.page_size) {
            len = 0;
            atomicOr(p.status, kStatusBadLengthBit);
        }
        const int see = min(len, len - (__ldcg(p.cu + b + 1) - t) + 1);
        float q[kLatRow / 32], o[kLatC / 32] = {}, m = -INFINITY, l = 0.f;
        const uint16_t *qp = p.q + (static_cast<size_t>(t) * p.H + h) * kLatRow;
#pragma unroll
        for (int i = 0; i < kLatRow / 32; ++i) q[i] = bf16_bits(qp[lane + 32 * i]);
        for (int j = 0; j < see; ++j) {
            const int id = __ldcg(p.tables + static_cast<size_t>(b) * p.width + j / p.page_size);
            float r[kLatRow / 32], s = 0.f;
            const bool there = id >= 0 && id < p.n_pages;
            if (!there) atomicOr(p.status, kStatusBadPageBit);
            const uint16_t *row = p.pages + (static_cast<size_t>(there ? id : 0) * p.page_size + j % p.page_size) * kLatRow;
#pragma unroll
            for (int i = 0; i < kLatRow / 32; ++i) {
                r[i] = there ? bf16_bits(row[lane + 32 * i]) : 0.f;
                s = fmaf(q[i], r[i], s);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
            s *= p.scale_log2;
            const float n = fmaxf(m, s), f = n == -INFINITY ? 0.f : n;
            const float g = fast_exp2(m - f), w = fast_exp2(s - f);
            m = n;
            l = l * g + w;
#pragma unroll
            for (int i = 0; i < kLatC / 32; ++i) o[i] = fmaf(w, r[i], o[i] * g);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t *out = p.out + (static_cast<size_t>(t) * p.H + h) * kLatC;
#pragma unroll
        for (int i = 0; i < kLatC / 32; ++i) out[lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
        if (p.lse && lane == 0) p.lse[static_cast<size_t>(t) * p.H + h] = (m + log2f(l)) * 0.69314718055994531f;
    }
    grid_dependents_launch();
}

}  // namespace cfa
