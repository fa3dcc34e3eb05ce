// cfa_latent_cache.cuh -- a token's latent row into the paged cache, its queries rotated.
//
//   row = [g x / sqrt(mean x^2 + eps) | rope(k, n)],  q = [q_nope | rope(q_rope, n)]
//
// where pair i of the 64 rotated dims at position n turns by n f_i:
//   (x0, x1) -> m (x0 cos - x1 sin, x1 cos + x0 sin),
// (x0, x1) = dims (i, i + 32) or (2i, 2i + 1). Angles are fractions of a turn in 64-bit fixed
// point (n * turns_i modulo 2^64 is exact), so that far positions cost no accuracy. Sums and
// products are fp32, each result is rounded to bf16 once.
//
// A block takes one token and 32 heads of its queries, with all of a thread's loads on
// their way before the first is used; one block more a token makes the cache row.
//
// Measured (one GB300): 4096 tokens of 128 heads into a new q_out 62 us (412 MB: 98% of what a copy reaches), memory
// bounds it; one token of 8 heads 7 us, the call's own time on the host.
#pragma once

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_paged_device.cuh"
#include "cfa_tile.cuh"

namespace cfa {

// Eight rotated dims, or twice eight where halves form the pairs (b: dims 32 on), in place.
template <bool kInterleaved>
__device__ __forceinline__ void latent_turn(uint4 &a, uint4 &b, const float2 *r) {
    float x[8], y[8];
    unpack8_bf16(a, x);
    if constexpr (kInterleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] = x[2 * e] * r[e].x - x[2 * e + 1] * r[e].y;
            y[2 * e + 1] = x[2 * e + 1] * r[e].x + x[2 * e] * r[e].y;
        }
    } else {
        float z[8];
        unpack8_bf16(b, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = x[e] * r[e].x - z[e] * r[e].y;
            z[e] = z[e] * r[e].x + x[e] * r[e].y;
        }
        b = make_uint4(pack2_bf16_cvt(z[0], z[1]), pack2_bf16_cvt(z[2], z[3]), pack2_bf16_cvt(z[4], z[5]),
                       pack2_bf16_cvt(z[6], z[7]));
    }
    a = make_uint4(pack2_bf16_cvt(y[0], y[1]), pack2_bf16_cvt(y[2], y[3]), pack2_bf16_cvt(y[4], y[5]),
                   pack2_bf16_cvt(y[6], y[7]));
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kLatAppendThreads)
latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
    // a unit is what a thread turns at once: 16 bytes, or 16 and the other half's 16
    constexpr int kUnits = kInterleaved ? 8 : 4, kPairs = 32 / kUnits;
    constexpr int kTurns = kLatAppendHeads * kUnits / kLatAppendThreads;      // units of a thread
    constexpr int kCopies = kLatAppendHeads * (kLatN / 8) / kLatAppendThreads;  // chunks to copy
    __shared__ float2 cs[kLatR / 2];
    __shared__ float sums[2];
    const int t = blockIdx.x, tid = threadIdx.x, part = static_cast<int>(blockIdx.y);
    const bool row = part == static_cast<int>(gridDim.y) - 1;
    grid_dependency_wait();
    const int slot = __ldcg(p.slots + t);
    const int pos = __ldcg(p.positions + t);
    const int h0 = part * kLatAppendHeads, heads = min(kLatAppendHeads, p.n_heads - h0);
    const int unit = tid % kUnits;
    uint4 a[kTurns], b[kTurns], c[kCopies];
    const uint16_t *q = p.q + t * p.q_stride + h0 * kLatQ, *in = p.a + t * p.a_stride;
    if (!row) {
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            const int h = tid / kUnits + j * (kLatAppendThreads / kUnits);
            if (h >= heads) continue;
            const uint16_t *src = q + h * kLatQ + kLatN + 8 * unit;
            a[j] = *reinterpret_cast<const uint4 *>(src);
            if (!kInterleaved) b[j] = *reinterpret_cast<const uint4 *>(src + kLatR / 2);
        }
        if (p.copy) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) {
                const int i = tid + j * kLatAppendThreads, h = i / (kLatN / 8);
                if (h < heads) c[j] = *reinterpret_cast<const uint4 *>(q + h * kLatQ + 8 * (i % (kLatN / 8)));
            }
        }
    } else if (tid < 64) {
        a[0] = *reinterpret_cast<const uint4 *>(in + 8 * tid);
        c[0] = *reinterpret_cast<const uint4 *>(p.g_kv + 8 * tid);
    } else if (tid < 64 + kUnits) {
        a[0] = *reinterpret_cast<const uint4 *>(in + kLatC + 8 * unit);
        if (!kInterleaved) b[0] = *reinterpret_cast<const uint4 *>(in + kLatC + 8 * unit + kLatR / 2);
    }
    if (p.rope && tid < kLatR / 2) {
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * p.turns[tid];
        // the signed upper half counts half turns in units of 2^-31
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cn);
        cs[tid] = make_float2(cn * p.magnitude, sn * p.magnitude);
    }
    if (slot >= p.n_rows && tid == 0) atomicOr(p.status, kStatusBadPageBit);
    const bool live = slot >= 0 && slot < p.n_rows;
    float x[8], ss = 0.f;
    if (row && tid < 64) {
        unpack8_bf16(a[0], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if ((tid & 31) == 0) sums[tid >> 5] = ss;
    }
    __syncthreads();
    if (live) {
        const float2 *r = cs + kPairs * unit;
        if (!row) {
            uint16_t *out = p.q_out + (static_cast<size_t>(t) * p.n_heads + h0) * kLatQ;
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                const int h = tid / kUnits + j * (kLatAppendThreads / kUnits);
                if (h >= heads) continue;
                uint16_t *dst = out + h * kLatQ + kLatN + 8 * unit;
                if (p.rope) latent_turn<kInterleaved>(a[j], b[j], r);
                *reinterpret_cast<uint4 *>(dst) = a[j];
                if (!kInterleaved) *reinterpret_cast<uint4 *>(dst + kLatR / 2) = b[j];
            }
            if (p.copy) {
#pragma unroll
                for (int j = 0; j < kCopies; ++j) {
                    const int i = tid + j * kLatAppendThreads, h = i / (kLatN / 8);
                    if (h < heads) *reinterpret_cast<uint4 *>(out + h * kLatQ + 8 * (i % (kLatN / 8))) = c[j];
                }
            }
        } else {
            uint16_t *dst = p.pages + static_cast<size_t>(slot) * kLatRow;
            if (tid < 64) {
                const float f = 1.f / sqrtf((sums[0] + sums[1]) / kLatC + p.eps);
                float g[8];
                unpack8_bf16(c[0], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * f * g[e];
                *reinterpret_cast<uint4 *>(dst + 8 * tid) =
                    make_uint4(pack2_bf16_cvt(x[0], x[1]), pack2_bf16_cvt(x[2], x[3]), pack2_bf16_cvt(x[4], x[5]),
                               pack2_bf16_cvt(x[6], x[7]));
            } else if (tid < 64 + kUnits) {
                if (p.rope) latent_turn<kInterleaved>(a[0], b[0], r);
                *reinterpret_cast<uint4 *>(dst + kLatC + 8 * unit) = a[0];
                if (!kInterleaved) *reinterpret_cast<uint4 *>(dst + kLatC + 8 * unit + kLatR / 2) = b[0];
            }
        }
    }
    grid_dependents_launch();
}

}  // namespace cfa
