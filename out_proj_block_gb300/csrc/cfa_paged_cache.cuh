// cfa_paged_cache.cuh -- the bookkeeping and the writing side of a paged
// cache: block tables and slot maps from request lengths, and the rotary
// embedding of new q and k with the append of k and v to their pages.
#pragma once

#include "cfa_device.cuh"
#include "cfa_paged.h"
#include "cfa_paged_device.cuh"
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
// suffice, or a length or a counter of the pool is negative, nothing is granted (no table entry
// changes, every cu is 0, every slot -1) and the status word says why.
//
// Every block scans all the lengths by itself (at most 8 KB, from L2), so that
// no block waits for another; its share of the tokens and of the new pages then
// comes from two binary searches in shared memory. A page of this call is taken
// from the free list directly, never read back from the table that other blocks
// are writing. lens_out and pool_out may be lens and pool: the last block to
// finish writes them, when every block has read the inputs. Launch latency bounds it:
// a call takes 7.6 us for 16 requests and 8.1 us for 512 with 64 prompt chunks (some
// 65,000 new tokens, 0.57 MB), of which the host's share is 7.
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
    const int taken = p.pool[0], left = paged_pool_left(taken, p.pool[1], p.n_free);
    const bool invalid = bad != 0 || total > p.n_slots || left < 0;
    const bool none = !invalid && grant > left;
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
            if (page >= 0 && page <= p.max_page) slot = page * ps + at_b - j * ps;
            else atomicOr(p.status, kStatusBadPageBit);
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
// One block per token. A thread keeps one chunk of a head's dims (16 bytes, or a pair of
// chunks where the layout pairs halves) and goes through the heads, so that its cosines and
// sines stay in registers; they are made once for the block in shared memory while the first
// chunks of q, k and v are already on their way (several of each: they would otherwise wait for
// memory one after the other). Instructions count: choosing head and chunk anew for every 16
// bytes took 24 us at 4096 tokens of 32/8 heads x 128 (100.7 MB). So does that some blocks of
// an SM load while others store, which small blocks do best: 256 threads took 21.3 us there,
// 128 18.9, 64 17.3 (5.8 TB/s). The bytes bound it at many tokens, the launch at few.
template <bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 8)
paged_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ float2 cs[64];
    constexpr int U = kInterleaved ? 4 : 2, kPairs = kInterleaved ? 4 : 8;  // loads ahead; pairs of a unit
    const int t = blockIdx.x, tid = threadIdx.x, threads = blockDim.x, d = p.d, half = p.rd / 2;
    grid_dependency_wait();
    const int slot = __ldcg(p.slots + t);
    const int pos = __ldcg(p.positions + t);
    // units of a head: the rotated ones first, then 8 dims each that pass through
    const int rot = kInterleaved ? p.rd / 8 : p.rd / 16, units = rot + (d - p.rd) / 8;
    const int first = tid / p.by_units, unit = tid - first * units, step = p.heads_a_pass;
    const bool turns = unit < rot;
    const int at = turns ? 8 * unit : p.rd + 8 * (unit - rot);
    const int heads = first < step ? p.n_heads + p.n_kv : 0;
    const uint16_t *q = p.q + t * p.q_stride + at, *k = p.k + t * p.k_stride + at;
    const uint16_t *v = p.v + t * p.v_stride + 8 * tid;
    const int v_chunks = p.n_kv * d / 8;
    uint4 a[U], b[U], c[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = h0 + j * step;
            if (h >= heads) continue;
            const uint16_t *src = h < p.n_heads ? q + h * d : k + (h - p.n_heads) * d;
            a[j] = *reinterpret_cast<const uint4 *>(src);
            if (!kInterleaved && turns) b[j] = *reinterpret_cast<const uint4 *>(src + half);
        }
    };
    auto load_v = [&](int i0) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (tid + i0 + j * threads < v_chunks)
                c[j] = *reinterpret_cast<const uint4 *>(v + 8 * (i0 + j * threads));
    };
    load(first);
    load_v(0);
    if (tid < half) {
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * p.turns[tid];
        // the signed upper half counts half turns in units of 2^-31
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cn);
        cs[tid] = make_float2(cn * p.magnitude, sn * p.magnitude);
    }
    if (slot >= p.n_rows && tid == 0) atomicOr(p.status, kStatusBadPageBit);
    __syncthreads();
    if (slot >= 0 && slot < p.n_rows) {
        float2 r[kPairs];
#pragma unroll
        for (int e = 0; e < kPairs; ++e) r[e] = turns ? cs[kPairs * unit + e] : make_float2(1.f, 0.f);
        const int page = slot / p.by_page, off = slot - page * p.page_size;
        const size_t row = (static_cast<size_t>(page) * p.n_kv * p.page_size + off) * d;
        const size_t head_rows = static_cast<size_t>(p.page_size) * d;
        uint16_t *q_out = p.q_out + static_cast<size_t>(t) * p.n_heads * d + at, *k_out = p.k_pages + row + at;
        for (int h0 = first; h0 < heads; h0 += U * step) {
            if (h0 > first) load(h0);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = h0 + j * step;
                if (h >= heads) continue;
                uint16_t *dst = h < p.n_heads ? q_out + h * d : k_out + (h - p.n_heads) * head_rows;
                if (turns) {
                    float x[8], y[8];
                    unpack8_bf16(a[j], x);
                    if constexpr (kInterleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            y[2 * e] = x[2 * e] * r[e].x - x[2 * e + 1] * r[e].y;
                            y[2 * e + 1] = x[2 * e + 1] * r[e].x + x[2 * e] * r[e].y;
                        }
                    } else {
                        float z[8];
                        unpack8_bf16(b[j], z);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y[e] = x[e] * r[e].x - z[e] * r[e].y;
                            z[e] = z[e] * r[e].x + x[e] * r[e].y;
                        }
                        *reinterpret_cast<uint4 *>(dst + half) =
                            make_uint4(pack2_bf16_cvt(z[0], z[1]), pack2_bf16_cvt(z[2], z[3]),
                                       pack2_bf16_cvt(z[4], z[5]), pack2_bf16_cvt(z[6], z[7]));
                    }
                    a[j] = make_uint4(pack2_bf16_cvt(y[0], y[1]), pack2_bf16_cvt(y[2], y[3]),
                                      pack2_bf16_cvt(y[4], y[5]), pack2_bf16_cvt(y[6], y[7]));
                }
                *reinterpret_cast<uint4 *>(dst) = a[j];
            }
        }
        const int shift = d == 128 ? 4 : 3;  // chunks of a head
        uint16_t *v_out = p.v_pages + row;
        for (int i0 = 0; tid + i0 < v_chunks; i0 += U * threads) {
            if (i0 > 0) load_v(i0);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int i = tid + i0 + j * threads;
                if (i < v_chunks)
                    *reinterpret_cast<uint4 *>(v_out + (i >> shift) * head_rows + 8 * (i & ((1 << shift) - 1))) = c[j];
            }
        }
    }
    grid_dependents_launch();
}

}  // namespace cfa
