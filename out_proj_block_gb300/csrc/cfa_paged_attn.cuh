// cfa_paged_attn.cuh -- attention of a ragged batch over a prefix that all its
// requests share and each request's own pages.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = scale log2(e) q . k_j,
//   m = max_j s_j;  lse = (m + log2 sum_j w_j) ln 2
//
// over the prefix's keys and, of request b's own len_b keys, those up to
// len_b - n_b + i for its i-th of n_b query tokens. A row without keys is 0
// with lse -inf.
#pragma once

#include <cuda_bf16.h>

#include "cfa_device.cuh"
#include "cfa_paged.h"
#include "cfa_tile.cuh"

namespace cfa {

// One warp per (token, head), one key at a time: the running maximum and sum
// in one pass, each lane holding D/32 dims of q and of the output.
template <int D>
__global__ void __launch_bounds__(256)
paged_attention_simple_kernel(const PagedAttnParams p) {
    constexpr int E = D / 32;
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = item / p.n_heads, h = item % p.n_heads;
    // every block checks the offsets: they bound the rows
    int bad = 0;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x)
        bad |= p.cu[b] < 0 || p.cu[b + 1] < p.cu[b] || p.cu[b + 1] > p.T;
    bad = __syncthreads_or(bad);
    if (bad) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLengthBit);
        return;
    }
    if (t >= p.cu[p.B] || t < p.cu[0]) return;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo, n = p.cu[b + 1] - p.cu[b];
    int len = p.lens[b];
    if (len < 0 || len > static_cast<long long>(p.width) * p.page_size) {
        if (lane == 0) atomicOr(p.status, kStatusBadLengthBit);
        len = 0;
    }
    const int mine = min(len, max(0, len - n + (t - p.cu[b]) + 1));
    const int kvh = h / (p.n_heads / p.n_kv);
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e)
        q[e] = bf16_bits(p.q[t * p.q_stride + h * D + lane * E + e]) * p.scale_log2;
    auto keys = [&](const int *table, int count) {
        for (int j = 0; j < count; ++j) {
            const int page = table[j / p.page_size];
            const bool there = page >= 0 && page < p.n_pages;
            if (!there && lane == 0) atomicOr(p.status, kStatusBadPageBit);
            const size_t row = ((static_cast<size_t>(there ? page : 0) * p.n_kv + kvh) * p.page_size +
                                j % p.page_size) * D + lane * E;
            float s = 0.f, v[E];
            for (int e = 0; e < E; ++e) {
                s += there ? q[e] * bf16_bits(p.k_pages[row + e]) : 0.f;
                v[e] = there ? bf16_bits(p.v_pages[row + e]) : 0.f;
            }
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
            const float mn = fmaxf(m, s), a = fast_exp2(m - mn), w = fast_exp2(s - mn);
            m = mn;
            l = l * a + w;
            for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * v[e];
        }
    };
    keys(p.prefix_table, p.prefix_len);
    keys(p.tables + static_cast<size_t>(b) * p.width, mine);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; ++e)
        p.out[(static_cast<size_t>(t) * p.n_heads + h) * D + lane * E + e] =
            __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
    if (p.lse && lane == 0)
        p.lse[static_cast<size_t>(t) * p.n_heads + h] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace cfa
