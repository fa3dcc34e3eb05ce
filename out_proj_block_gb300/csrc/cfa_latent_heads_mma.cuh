// cfa_latent_heads_mma.cuh -- the products of cfa_latent_heads.cuh for many tokens, on tcgen05.
//
// A job is 128 tokens of a head and, folding, 256 of the 512 latent dims (8 instructions of 128 x 256 x 16),
// unfolding, the 128 value dims (32 of 128 x 128 x 16). Blocks, one to an SM, take runs of jobs in the
// order of heads and tokens, so that a head's weights are loaded once or twice (64 KB, two buffers; 128 KB, one) and
// stay in shared memory while the tokens' rows stream through: memory bounds it, with the weights no part of it. A load
// warp, one that issues the products, and two warpgroups that bring results from one of two accumulators in TMEM
// through shared memory to whole boxes of 64 columns, by turns (TMA stores, which end at the last token by
// themselves; one warpgroup instead took 3% more).
//
// Measured (one GB300): 777 tokens of 32 heads in 11.6 us (42 MB, floor 6.2; on mma.sync 15.8 to 18.3), 1000 tokens
// of 128 heads in 46.5 us (213 MB, floor 31); 1000 of 128 heads out 34.7 us (181 MB, floor 26.6; on mma.sync
// 46 to 54). The weights read again for every 64 or 128 tokens, out of L2, held the others back.
#pragma once

#include <cuda.h>

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_paged_device.cuh"
#include "cfa_tensor.cuh"

namespace cfa {

template <bool FOLD>
struct HeadsMma {
    static constexpr int kChunks = (FOLD ? kLatN : kLatC) / 64;        // of 64 dims of x
    static constexpr int kCols = FOLD ? 256 : kLatV;                   // of a job's result
    static constexpr int kSplit = FOLD ? kLatC / kCols : 1;            // jobs of a head's 128 tokens
    static constexpr int kWeights = kChunks * kCols * 128;             // bytes
    static constexpr int kWSlots = FOLD ? 2 : 1, kXSlots = FOLD ? 2 : 4;
    static constexpr int kOutSlots = FOLD ? 2 : 1;                     // of either warpgroup
    static constexpr int kBox = 128 * 128;                             // 128 tokens of 64 dims
    static constexpr int kW = 0, kX = kW + kWSlots * kWeights, kOut = kX + kXSlots * kBox;
    static constexpr int kBars = kOut + 2 * kOutSlots * kBox;
    static constexpr int kFullW = kBars, kEmptyW = kFullW + 8 * kWSlots, kFullX = kEmptyW + 8 * kWSlots,
                         kEmptyX = kFullX + 8 * kXSlots, kFullAcc = kEmptyX + 8 * kXSlots, kEmptyAcc = kFullAcc + 16,
                         kDrain = kEmptyAcc + 16, kBarsEnd = kDrain + 8;
    static constexpr int kMisc = kBarsEnd, kBytes = kMisc + 16;
    static_assert(kBytes <= 227 * 1024, "it fits");
};

__device__ __forceinline__ void tma_store_2d(const void *tmap, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(src) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the last N groups of this thread's stores have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <bool FOLD>
__global__ void __launch_bounds__(kHeadsMmaThreads, 1)
latent_heads_mma_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ LatentHeadsParams p) {
    using S = HeadsMma<FOLD>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    int *misc = reinterpret_cast<int *>(smem + S::kMisc);
    volatile int *timed_out = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);
    if (tid < (S::kBarsEnd - S::kBars) / 8) {
        const int at = S::kBars + 8 * tid;
        mbar_init(base + at, at >= S::kEmptyAcc && at < S::kDrain ? 8 : 1);  // the warps that read an accumulator
        fence_mbar_init();
    }
    if (tid == 0) misc[0] = 0;
    if (warp == 5) tmem_alloc(smem_addr(tmem_slot), 512);
    if (warp == 4 && elect_one()) {
        prefetch_tensor_map(&tm_x);
        prefetch_tensor_map(&tm_w);
        prefetch_tensor_map(&tm_y);
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    grid_dependency_wait();
    grid_dependents_launch();
    const uint32_t tmem = *tmem_slot;
    const int tiles = (p.T + 127) / 128, per_w = tiles;  // jobs with the same weights
    const long long jobs = static_cast<long long>(p.H) * S::kSplit * tiles;
    const long long j0 = jobs * blockIdx.x / gridDim.x, j1 = jobs * (blockIdx.x + 1) / gridDim.x;
    // which weights (head, part of the columns) and tokens the run begins with
    const int w0 = static_cast<int>(j0 / per_w), t0 = static_cast<int>(j0 - static_cast<long long>(w0) * per_w);
    const int n_jobs = static_cast<int>(j1 - j0);
    auto wait = [&](int bar, uint32_t parity, unsigned site) {
        return bounded_wait([&]() { return mbar_try_wait(base + bar, parity); }, p.timeout_ns, timed_out, p.status, site);
    };
    auto wait_warp = [&](int bar, uint32_t parity, unsigned site) { return __all_sync(~0u, wait(bar, parity, site)); };

    if (warp == 4) {
        // -------------------------------------------------------------------- load warp
        uint32_t nw = 0, nx = 0;
        bool ok = true;
        int w = w0, t = t0;
        CFA_ROLLED for (int j = 0; ok && j < n_jobs; ++j) {
            const int h = w / S::kSplit, part = w % S::kSplit;
            if (j == 0 || t == 0) {
                const uint32_t slot = nw % S::kWSlots;
                if (nw >= S::kWSlots) ok = wait_warp(S::kEmptyW + 8 * slot, (nw / S::kWSlots - 1) & 1, kSiteStageEmpty);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t full = base + S::kFullW + 8 * slot, dst = base + S::kW + slot * S::kWeights;
                    mbar_arrive_expect_tx(full, S::kWeights);
                    if (FOLD) {  // [2 dims][256 latent dims][128 bytes]
#pragma unroll 1
                        for (int i = 0; i < 8; ++i)
                            tma_load_2d(dst + i * 8192, &tm_w, h * kLatKv + 64 * (i >> 2), S::kCols * part + 64 * (i & 3), full);
                    } else {     // [8 latent dims][2 dims][64][128 bytes]
#pragma unroll 1
                        for (int i = 0; i < 16; ++i)
                            tma_load_2d(dst + i * 8192, &tm_w, h * kLatKv + kLatN + 64 * (i & 1), 64 * (i >> 1), full);
                    }
                }
                __syncwarp();
                ++nw;
            }
            CFA_ROLLED for (int c = 0; c < S::kChunks; ++c, ++nx) {
                const uint32_t slot = nx % S::kXSlots, full = base + S::kFullX + 8 * slot;
                if (nx >= S::kXSlots) ok = wait_warp(S::kEmptyX + 8 * slot, (nx / S::kXSlots - 1) & 1, kSiteStageEmpty);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, S::kBox);
                    tma_load_2d(base + S::kX + slot * S::kBox, &tm_x, h * (FOLD ? kLatQ : kLatC) + 64 * c, 128 * t, full);
                }
                __syncwarp();
            }
            if (++t == tiles) t = 0, ++w;
        }
        if (lane == 0 && *timed_out) {
            // a wait gave up: the copies in flight land before the block ends
            const uint64_t since = global_timer_ns();
            auto land = [&](uint32_t bar, uint32_t parity) {
                while (!mbar_try_wait(bar, parity) && global_timer_ns() - since < kDrainTimeoutFactor * p.timeout_ns) {
                }
            };
            for (uint32_t k = nx > S::kXSlots ? nx - S::kXSlots : 0; k < nx; ++k)
                land(base + S::kFullX + 8 * (k % S::kXSlots), (k / S::kXSlots) & 1);
            for (uint32_t k = nw > S::kWSlots ? nw - S::kWSlots : 0; k < nw; ++k)
                land(base + S::kFullW + 8 * (k % S::kWSlots), (k / S::kWSlots) & 1);
        }
        __syncwarp();
    } else if (warp == 5) {
        // --------------------------------------------------------------------- products
        const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
        const uint32_t idesc = umma_idesc_bf16(128, S::kCols, false, !FOLD);
        const uint64_t x0 = umma_smem_desc(base + S::kX, 16, 1024), b0 = umma_smem_desc(base + S::kW, FOLD ? 16 : 8192, 1024);
        uint32_t nw = 0, nx = 0;
        bool ok = true;
        int t = t0;
        CFA_ROLLED for (int j = 0; ok && j < n_jobs; ++j) {
            const uint32_t acc = j & 1;
            if (j == 0 || t == 0) {
                ok = wait_warp(S::kFullW + 8 * (nw % S::kWSlots), (nw / S::kWSlots) & 1, kSiteStageFull);
                ++nw;
            }
            const uint32_t slot_w = (nw - 1) % S::kWSlots;
            if (j >= 2) ok = ok && wait_warp(S::kEmptyAcc + 8 * acc, ((j >> 1) - 1) & 1, kSiteKvExchange);
            CFA_ROLLED for (int c = 0; ok && c < S::kChunks; ++c, ++nx) {
                const uint32_t slot = nx % S::kXSlots;
                ok = wait_warp(S::kFullX + 8 * slot, (nx / S::kXSlots) & 1, kSiteStageFull);
                tcgen05_fence_after();
                if (ok && elect_one()) {
                    const uint64_t a = x0 + slot * (S::kBox >> 4);
                    const uint64_t b = b0 + slot_w * (S::kWeights >> 4) + c * ((FOLD ? S::kCols * 128 : 16384) >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)  // 32 bytes a step, or 16 rows of 128
                        umma_bf16(tm + 256 * acc, a + 2 * ks, b + (FOLD ? 2 : 128) * ks, idesc, c > 0 || ks > 0);
                    umma_commit(base + S::kEmptyX + 8 * slot);
                    if (c == S::kChunks - 1) {
                        umma_commit(base + S::kFullAcc + 8 * acc);
                        if (t + 1 == tiles) umma_commit(base + S::kEmptyW + 8 * slot_w);
                    }
                }
                __syncwarp();
            }
            if (++t == tiles) t = 0;
        }
        if (elect_one() && *timed_out) {
            // a wait gave up: the products in flight end before the block does
            umma_commit(base + S::kDrain);
            const uint64_t since = global_timer_ns();
            while (!mbar_try_wait(base + S::kDrain, 0) && global_timer_ns() - since < kDrainTimeoutFactor * p.timeout_ns) {
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------------- results
        const int group = warp >= 4, row = 32 * (warp & 3) + lane;  // of the two warpgroups; token of the tile
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lanes of this warp
        auto meet = [&]() { asm volatile("bar.sync %0, 128;" :: "r"(1 + group) : "memory"); };
        const int out0 = S::kOut + group * S::kOutSlots * S::kBox, thread = 128 * group + row;
        uint32_t n_out = 0;
        int w = w0, t = t0;
        CFA_ROLLED for (int j = 0; j < n_jobs; ++j) {
            const uint32_t acc = j & 1;
            const int h = w / S::kSplit, part = w % S::kSplit;
            uint4 rot[4];  // the rotated dims pass through
            const bool copies = FOLD && part == 0;
            const uint16_t *src = p.x + h * kLatQ + kLatN + 8 * (thread & 7);
            if (copies) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = 128 * t + 32 * i + (thread >> 3);
                    if (tok < p.T) rot[i] = *reinterpret_cast<const uint4 *>(src + tok * p.x_stride);
                }
            }
            wait(S::kFullAcc + 8 * acc, (j >> 1) & 1, kSiteKvExchange);
            __syncwarp();
            tcgen05_fence_after();
#pragma unroll 1
            for (int c = 64 * group; c < S::kCols; c += 128, ++n_out) {
                uint32_t v[64];
                tmem_ld_x32(tmem + lanes + 256 * acc + c, v);
                tmem_ld_x32(tmem + lanes + 256 * acc + c + 32, v + 32);
                tmem_wait_ld();
                if (c + 128 >= S::kCols) {  // the accumulator is read
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(base + S::kEmptyAcc + 8 * acc);
                }
                if (row == 0) bulk_wait_read<S::kOutSlots - 1>();  // the slot's last store has read it
                meet();
                const int slot = out0 + (n_out % S::kOutSlots) * S::kBox;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[k] = pack2_bf16_cvt(__uint_as_float(v[8 * e + 2 * k]), __uint_as_float(v[8 * e + 2 * k + 1]));
                    *reinterpret_cast<uint4 *>(smem + slot + row * 128 + ((e ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
                meet();
                if (row == 0) {
                    tma_store_2d(&tm_y, FOLD ? h * kLatRow + S::kCols * part + c : h * kLatV + c, 128 * t, base + slot);
                    bulk_commit();
                }
            }
            if (copies) {
                uint16_t *dst = p.y + h * kLatRow + kLatC + 8 * (thread & 7);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = 128 * t + 32 * i + (thread >> 3);
                    if (tok < p.T) *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(tok) * p.H * kLatRow) = rot[i];
                }
            }
            if (++t == tiles) t = 0, ++w;
        }
        if (row == 0) bulk_wait_all();
    }
    tcgen05_fence_before();
    __syncthreads();
    if (warp == 5) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace cfa
