// cfa_paged_cache.cuh -- the bookkeeping and the writing side of a paged
// cache: block tables and slot maps from request lengths, and the rotary
// embedding of new q and k with the append of k and v to their pages.
#pragma once

#include "cfa_device.cuh"
#include "cfa_paged.h"
#include "cfa_tile.cuh"

namespace cfa {

// ------------------------------------------------- block tables and slot maps
//
//   have_b = ceil(lens_b / ps), need_b = ceil((lens_b + fresh_b) / ps)
//   rank_b = sum_{i < b} (need_i - have_i)            cu_b = sum_{i < b} fresh_i
//   tables[b][have_b + j] = free[taken + rank_b + j]  for j < need_b - have_b
//   token i of request b: position base + lens_b + i, slot = page * ps + offset
//
// All or nothing: where the pages, the token rows or the table's width do not
// suffice, or a length is negative, nothing is granted (no table entry
// changes, every cu is 0, every slot -1) and the status word says why.
//
// Every block scans all the lengths by itself (at most 8 KB, from L2), so that
// no block waits for another; its share of the tokens and of the new pages then
// comes from two binary searches in shared memory. A page of this call is taken
// from the free list directly, never read back from the table that other blocks
// are writing. lens_out and pool_out may be lens and pool: the last block to
// finish writes them, when every block has read the inputs.
__global__ void __launch_bounds__(kTablesThreads)
paged_tables_kernel(const TablesParams p) {
    extern __shared__ int sh[];
    const int B = p.B, ps = p.page_size, tid = threadIdx.x;
    int *cu = sh, *rank = sh + B + 1, *len = rank + B + 1;
    __shared__ int warp_sum[2][kTablesThreads / 32];
    __shared__ int bad;
    __shared__ bool last;
    if (tid == 0) bad = 0;
    grid_dependency_wait();
    __syncthreads();

    const int per = (B + kTablesThreads - 1) / kTablesThreads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
    int flags = 0, tokens = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        int l = p.lens[b], f = p.fresh[b];
        if (l < 0 || f < 0 || static_cast<long long>(l) + f > static_cast<long long>(p.width) * ps ||
            f > p.n_slots) {
            flags |= 1;
            l = f = 0;
        }
        len[b] = l;
        cu[b] = f;  // exclusive sums below
        const int extra = (l + f + ps - 1) / ps - (l + ps - 1) / ps;
        rank[b] = extra;
        tokens += f;
        pages += extra;
    }
    // exclusive sums over the threads: at most 1024 * 2^17 tokens and
    // 1024 * 2^18 pages, below 2^31
    const int lane = tid & 31, warp = tid >> 5;
    int st = tokens, sp = pages;
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(~0u, st, o), c = __shfl_up_sync(~0u, sp, o);
        if (lane >= o) st += a, sp += c;
    }
    if (lane == 31) warp_sum[0][warp] = st, warp_sum[1][warp] = sp;
    if (flags) atomicOr(&bad, flags);
    __syncthreads();
    int at = st - tokens, ar = sp - pages;
    for (int w = 0; w < warp; ++w) at += warp_sum[0][w], ar += warp_sum[1][w];
    for (int b = b0; b < b1; ++b) {
        const int f = cu[b], e = rank[b];
        cu[b] = at;
        rank[b] = ar;
        at += f;
        ar += e;
    }
    if (b0 < b1 && b1 == B) cu[B] = at, rank[B] = ar;
    __syncthreads();
    const int total = cu[B], grant = rank[B];
    const int taken = p.pool[0], there = min(p.pool[1], p.n_free);
    const bool invalid = bad != 0 || total > p.n_slots || taken < 0;
    const bool none = !invalid && grant > max(there - taken, 0);
    const bool ok = !invalid && !none;

    const int nthreads = gridDim.x * kTablesThreads, gid = blockIdx.x * kTablesThreads + tid;
    // the last request whose sum is at most x (requests without tokens or pages share theirs
    // with the next one)
    auto find = [&](const int *sum, int x) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sum[mid] <= x) lo = mid; else hi = mid;
        }
        return lo;
    };
    for (int t = gid; t < p.n_slots; t += nthreads) {
        int pos = 0, slot = -1;
        if (ok && t < total) {
            const int b = find(cu, t);
            const int at_b = len[b] + t - cu[b], j = at_b / ps, have = (len[b] + ps - 1) / ps;
            const int page = j < have ? p.tables[static_cast<size_t>(b) * p.width + j]
                                      : p.free_pages[taken + rank[b] + j - have];
            pos = p.base + at_b;
            slot = page * ps + at_b - j * ps;
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
    if (ok)
        for (int r = gid; r < grant; r += nthreads) {
            const int b = find(rank, r);
            const int have = (len[b] + ps - 1) / ps;
            p.tables[static_cast<size_t>(b) * p.width + have + r - rank[b]] = p.free_pages[taken + r];
        }
    for (int b = gid; b <= B; b += nthreads) p.cu[b] = ok ? cu[b] : 0;

    __syncthreads();
    if (tid == 0) last = gridDim.x == 1 || atomic_add_acq_rel_gpu(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (last) {
        if (tid == 0) {
            *p.ticket = 0;
            p.pool_out[0] = taken + (ok ? grant : 0);
            p.pool_out[1] = p.pool[1];
            if (invalid) atomicOr(p.status, kStatusBadLengthBit);
            if (none) atomicOr(p.status, kStatusNoPagesBit);
        }
        for (int b = tid; b < B; b += kTablesThreads)
            p.lens_out[b] = ok ? len[b] + cu[b + 1] - cu[b] : p.lens[b];
    }
    grid_dependents_launch();
}

// ------------------------------------------------------------ rotary append
//
// Pair i of a head at position n turns by the angle n f_i:
//   (x0, x1) -> m (x0 cos - x1 sin, x1 cos + x0 sin)
// with (x0, x1) = dims (i, i + rd/2) or (2i, 2i + 1); dims from rd on pass
// through. The angle is held as a fraction of a turn in 64-bit fixed point:
// n * turns_i modulo 2^64 is exact, so a far position costs no accuracy (an
// fp32 angle at position 2^22 would be off by 0.25 rad), and the reduction
// that the sine needs is the wrap-around of the integer product.
//
// One block per token: the cosines and sines of its position are made once in
// shared memory for all the heads; then every thread moves 16-byte chunks.
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float2 cs[64];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int d = p.d, half = p.rd / 2;
    grid_dependency_wait();
    const int pos = p.positions[t], slot = p.slots[t];
    if (tid < half) {
        const unsigned long long a =
            static_cast<unsigned long long>(static_cast<long long>(pos)) * p.turns[tid];
        // the signed upper half counts half turns in units of 2^-31
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 0x1p-31f, &s, &c);
        cs[tid] = make_float2(c * p.magnitude, s * p.magnitude);
    }
    if (slot >= p.n_rows && tid == 0) atomicOr(p.status, kStatusBadPageBit);
    const bool live = slot >= 0 && slot < p.n_rows;
    __syncthreads();
    if (!live) {
        grid_dependents_launch();
        return;
    }
    const int page = slot / p.page_size, off = slot - page * p.page_size;
    // chunks of a head: rotated units first, then 8 dims each that pass through
    const int rot = p.interleaved ? p.rd / 8 : p.rd / 16;
    const int units = rot + (d - p.rd) / 8;
    const int n_rot = (p.n_heads + p.n_kv) * units, n = n_rot + p.n_kv * (d / 8);
    auto cache_row = [&](uint16_t *pages, int h) {
        return pages + ((static_cast<size_t>(page) * p.n_kv + h) * p.page_size + off) * d;
    };
    for (int i = tid; i < n; i += kAppendThreads) {
        if (i >= n_rot) {
            const int h = (i - n_rot) / (d / 8), c = (i - n_rot) % (d / 8);
            *reinterpret_cast<uint4 *>(cache_row(p.v_pages, h) + 8 * c) =
                *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + h * d + 8 * c);
            continue;
        }
        const int h = i / units, u = i % units;
        const uint16_t *src = h < p.n_heads ? p.q + t * p.q_stride + h * d
                                            : p.k + t * p.k_stride + (h - p.n_heads) * d;
        uint16_t *dst = h < p.n_heads ? p.q_out + (static_cast<size_t>(t) * p.n_heads + h) * d
                                      : cache_row(p.k_pages, h - p.n_heads);
        if (u >= rot) {
            const int c = p.rd + 8 * (u - rot);
            *reinterpret_cast<uint4 *>(dst + c) = *reinterpret_cast<const uint4 *>(src + c);
        } else if (p.interleaved) {
            float x[8];
            unpack8_bf16(*reinterpret_cast<const uint4 *>(src + 8 * u), x);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 r = cs[4 * u + e];
                y[e] = pack2_bf16(x[2 * e] * r.x - x[2 * e + 1] * r.y, x[2 * e + 1] * r.x + x[2 * e] * r.y);
            }
            *reinterpret_cast<uint4 *>(dst + 8 * u) = make_uint4(y[0], y[1], y[2], y[3]);
        } else {
            float x[8], z[8];
            unpack8_bf16(*reinterpret_cast<const uint4 *>(src + 8 * u), x);
            unpack8_bf16(*reinterpret_cast<const uint4 *>(src + half + 8 * u), z);
            uint32_t y[4], w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 r = cs[8 * u + 2 * e], s = cs[8 * u + 2 * e + 1];
                y[e] = pack2_bf16(x[2 * e] * r.x - z[2 * e] * r.y, x[2 * e + 1] * s.x - z[2 * e + 1] * s.y);
                w[e] = pack2_bf16(z[2 * e] * r.x + x[2 * e] * r.y, z[2 * e + 1] * s.x + x[2 * e + 1] * s.y);
            }
            *reinterpret_cast<uint4 *>(dst + 8 * u) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4 *>(dst + half + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    grid_dependents_launch();
}

}  // namespace cfa
