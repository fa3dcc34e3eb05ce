// cfa_latent_heads.cuh -- the products of each head with its part of W_kvb [512, H * 256]:
//   fold     y[t, h, c] = sum_d x[t, h, d] W[c, h * 256 + d]          128 -> 512
//   unfold   y[t, h, d] = sum_c x[t, h, c] W[c, h * 256 + 128 + d]    512 -> 128
#pragma once

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_tile.cuh"

namespace cfa {

__global__ void __launch_bounds__(256) latent_fold_kernel(const __grid_constant__ LatentHeadsParams p) {
    const int h = blockIdx.y;
    grid_dependency_wait();
    for (int t = blockIdx.x * 64; t < min(p.T, static_cast<int>(blockIdx.x + 1) * 64); ++t) {
        const uint16_t *x = p.x + t * p.x_stride + h * kLatQ;
        uint16_t *y = p.y + (static_cast<size_t>(t) * p.H + h) * kLatRow;
        for (int c = threadIdx.x; c < kLatRow; c += 256) {
            if (c >= kLatC) {
                y[c] = x[kLatN + c - kLatC];
                continue;
            }
            const uint16_t *w = p.w + static_cast<size_t>(c) * p.H * kLatKv + h * kLatKv;
            float s = 0.f;
            for (int d = 0; d < kLatN; ++d) s = fmaf(bf16_bits(x[d]), bf16_bits(w[d]), s);
            y[c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
        }
    }
    grid_dependents_launch();
}

__global__ void __launch_bounds__(256) latent_unfold_kernel(const __grid_constant__ LatentHeadsParams p) {
    const int h = blockIdx.y;
    grid_dependency_wait();
    for (int t = blockIdx.x * 64 + threadIdx.x / 128; t < min(p.T, static_cast<int>(blockIdx.x + 1) * 64); t += 2) {
        const uint16_t *x = p.x + t * p.x_stride + h * kLatC;
        const int d = threadIdx.x % 128;
        const uint16_t *w = p.w + h * kLatKv + kLatN + d;
        float s = 0.f;
        for (int c = 0; c < kLatC; ++c) s = fmaf(bf16_bits(x[c]), bf16_bits(w[static_cast<size_t>(c) * p.H * kLatKv]), s);
        p.y[(static_cast<size_t>(t) * p.H + h) * kLatV + d] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
    grid_dependents_launch();
}

}  // namespace cfa
