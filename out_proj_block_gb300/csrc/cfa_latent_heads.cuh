// cfa_latent_heads.cuh -- the products of each head with its part of W_kvb [512, H * 256]:
//   fold     y[t, h, c] = sum_d x[t, h, d] W[c, h * 256 + d]          128 -> 512
//   unfold   y[t, h, d] = sum_c x[t, h, c] W[c, h * 256 + 128 + d]    512 -> 128
// in fp32, each result rounded to bf16 once.
//
// These are the kernels for few tokens (many: cfa_latent_heads_mma.cuh): the weights, 128 KB a head, bound
// them, and the latency of getting them. So a block asks for everything it needs before it waits, and the work
// is split into many small blocks, over the result's columns; unfold's four warps each take a quarter of the sum,
// joined in their order. mma.sync is enough.
//
// Measured (one GB300, calls back to back from Python, which itself takes 4.5 us): 4 tokens of 128 heads in 5.3 us
// (17.6 MB, floor 2.6); 1 token out 5.1 us (floor 2.5). The rule between the two forms is in
// cfa_latent.cu.
#pragma once

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_paged_device.cuh"
#include "cfa_tensor.cuh"

namespace cfa {

// 16 bytes, or zeros where there is no source.
__device__ __forceinline__ void cp_async_16_or_0(uint8_t *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

constexpr int kHeadsCols = 128;   // columns of a fold block's result
// Rows of 256 bytes as 16-byte chunks, rows of a group of eight apart in the banks.
__device__ __forceinline__ int heads_at(int row, int chunk) { return row * 256 + ((chunk ^ (row & 7)) << 4); }

// A block takes 16 tokens and 128 of the 512 latent dims. Shared memory: 128 rows of W, 16 of x.
__global__ void __launch_bounds__(128) latent_fold_kernel(const __grid_constant__ LatentHeadsParams p) {
    __shared__ __align__(128) uint8_t w[kHeadsCols * 256], x[kHeadsTokens * 256];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * kHeadsTokens, h = blockIdx.y, c0 = blockIdx.z * kHeadsCols, tokens = min(kHeadsTokens, p.T - t0);
    const size_t row_w = static_cast<size_t>(p.H) * kLatKv;
    grid_dependency_wait();
    const uint16_t *src_w = p.w + c0 * row_w + h * kLatKv, *src_x = p.x + t0 * p.x_stride + h * kLatQ;
#pragma unroll
    for (int i = 0; i < kHeadsCols * 16 / 128; ++i) {
        const int at = tid + i * 128, row = at >> 4, chunk = at & 15;
        cp_async_16(smem_addr(w + heads_at(row, chunk)), src_w + row * row_w + 8 * chunk);
    }
#pragma unroll
    for (int i = 0; i < kHeadsTokens * 16 / 128; ++i) {
        const int at = tid + i * 128, row = at >> 4, chunk = at & 15;
        cp_async_16_or_0(x + heads_at(row, chunk), row < tokens ? src_x + row * p.x_stride + 8 * chunk : src_x, row < tokens);
    }
    uint16_t *y = p.y + (static_cast<size_t>(t0) * p.H + h) * kLatRow;
    const size_t row_y = static_cast<size_t>(p.H) * kLatRow;
    if (c0 == 0 && tid < tokens * 8)  // the rotated dims pass through
        *reinterpret_cast<uint4 *>(y + (tid >> 3) * row_y + kLatC + 8 * (tid & 7)) =
            *reinterpret_cast<const uint4 *>(src_x + (tid >> 3) * p.x_stride + kLatN + 8 * (tid & 7));
    cp_async_wait_all();
    __syncthreads();
    float acc[4][4] = {};
    const int n0 = warp * 32;
#pragma unroll
    for (int k = 0; k < kLatN / 16; ++k) {
        uint32_t a[4], b[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            ldmatrix_x4(b[j], smem_addr(w + heads_at(n0 + 16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1))));
        ldmatrix_x4(a, smem_addr(x + heads_at(lane & 15, 2 * k + (lane >> 4))));
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_16x8x16(acc[j], a, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint32_t *>(x + heads_at((lane >> 2) + 8 * e, n0 / 8 + j) + 4 * (lane & 3)) =
                pack2_bf16_cvt(acc[j][2 * e], acc[j][2 * e + 1]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeadsTokens * 16 / 128; ++i) {
        const int at = tid + i * 128, row = at >> 4, chunk = at & 15;
        if (row < tokens) *reinterpret_cast<uint4 *>(y + row * row_y + c0 + 8 * chunk) = *reinterpret_cast<const uint4 *>(x + heads_at(row, chunk));
    }
    grid_dependents_launch();
}

// A block takes 16 tokens and 32 dims, each of its warps a quarter of the latent dims.
struct UnfoldSmem {
    static constexpr int kW = 0, kX = kLatC * 64, kSum = kX + 16 * kLatC * 2;  // [512][32], [16][512], [4][16][32] floats
    static constexpr int kBytes = kSum + 4 * 16 * 32 * 4;
};
__global__ void __launch_bounds__(128) latent_unfold_kernel(const __grid_constant__ LatentHeadsParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using S = UnfoldSmem;
    uint8_t *w = smem + S::kW, *x = smem + S::kX;
    float *sum = reinterpret_cast<float *>(smem + S::kSum);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * 16, h = blockIdx.y, d0 = blockIdx.z * 32, tokens = min(16, p.T - t0);
    const size_t row_w = static_cast<size_t>(p.H) * kLatKv;
    grid_dependency_wait();
    const uint16_t *src_w = p.w + h * kLatKv + kLatN + d0, *src_x = p.x + t0 * p.x_stride + h * kLatC;
#pragma unroll
    for (int i = 0; i < kLatC * 4 / 128; ++i) {
        const int at = tid + i * 128, row = at >> 2, chunk = at & 3;
        cp_async_16(smem_addr(w + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4)), src_w + row * row_w + 8 * chunk);
    }
#pragma unroll
    for (int i = 0; i < 16 * 64 / 128; ++i) {
        const int at = tid + i * 128, row = at >> 6, chunk = at & 63;
        cp_async_16_or_0(x + row * 1024 + ((chunk ^ (row & 7)) << 4), row < tokens ? src_x + row * p.x_stride + 8 * chunk : src_x,
                         row < tokens);
    }
    cp_async_wait_all();
    __syncthreads();
    float acc[4][4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t a[4];
        ldmatrix_x4(a, smem_addr(x + (lane & 15) * 1024 + (((16 * warp + 2 * k + (lane >> 4)) ^ (lane & 7)) << 4)));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t b[4];
            const int row = 128 * warp + 16 * k + (lane & 15);
            ldmatrix_x4_trans(b, smem_addr(w + row * 64 + (((2 * j + (lane >> 4)) ^ ((row >> 1) & 3)) << 4)));
            mma_16x8x16(acc[2 * j], a, b[0], b[1]);
            mma_16x8x16(acc[2 * j + 1], a, b[2], b[3]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2 *>(sum + (warp * 16 + (lane >> 2) + 8 * e) * 32 + 8 * j + 2 * (lane & 3)) =
                make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
    __syncthreads();
    const int row = tid >> 3, col = 4 * (tid & 7);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(sum + (k * 16 + row) * 32 + col);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    if (row < tokens)
        *reinterpret_cast<uint2 *>(p.y + (static_cast<size_t>(t0 + row) * p.H + h) * kLatV + d0 + col) =
            make_uint2(pack2_bf16_cvt(s.x, s.y), pack2_bf16_cvt(s.z, s.w));
    grid_dependents_launch();
}

}  // namespace cfa
