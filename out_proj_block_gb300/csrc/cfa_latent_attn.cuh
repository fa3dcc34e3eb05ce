// cfa_latent_attn.cuh -- attention of folded queries over paged latent rows.
//
//   o = sum_j w_j row_j[:512] / sum_j w_j,  w_j = 2^(s_j - m),  s_j = scale log2(e) q . row_j,
//   m = max_j s_j;  lse = (m + log2 sum_j w_j) ln 2
//
// for each of a request's query rows (tokens x heads, which lie one behind the other) over the
// cache rows that its token sees. A row without any is 0 with lse -inf.
//
// Every cache row is key and value at once, 1152 bytes for 2176 operations a query row: with 128 rows to
// a tile the tensor cores need 17 clocks of a pair of SMs for it at their full rate, and the
// memory 25. A tile of 128 rows needs more than one SM, though: its outputs alone, 128 x 512 in
// fp32, fill the whole TMEM. So a cluster of two blocks works on a tile with the instructions that
// span both (cta_group::2, M = 128: 64 rows to each block, twice as many TMEM lanes as rows, so that a
// row's columns stand in two halves):
//   S = Q K^T   128 rows x 128 keys, 576 dims; either block holds its 64 rows of Q and 64 of
//               the keys, in nine 64-dim chunks
//   O += P V    128 rows x 512 dims, 128 keys; either block holds its 64 rows of P and 256 of the
//               dims, for all keys: these come a second time, a block later, out of L2. The
//               keys that a block has for S will not do: the other one's are needed too
// TMEM holds O (256 columns) and two S (64 each), so that the next block's scores run under this
// one's softmax. Warps: four for the softmax (a thread for half the keys of a row), one to issue
// the products, two to load keys and values (TMA boxes of 64 dims with 128-byte swizzle, each
// inside one page), and one that passes on what has landed: the issuing block waits for both blocks'
// copies, and values that some or all rows do not see are cleared before the product, because a masked
// weight is 0 and 0 times NaN is NaN.
//
// Tiles are cut into runs of blocks of keys, one to a cluster (cfa_latent_split.h); what the
// runs' ends cut leaves records, which a second kernel merges in the order of the runs, so results
// are bitwise reproducible. A row's maximum is followed lazily, a published method: O is rescaled
// only when it grew by more than 8 (a factor 2^8, far inside fp32).
//
// Weights are rounded to bf16 for their product with the values (tensor cores take both operands in
// one type; 2^-8 each, the size of the result's own rounding); their sum, the maxima, the outputs
// and the records are fp32.
#pragma once

#include <cuda.h>

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_latent_split.h"
#include "cfa_paged_device.cuh"
#include "cfa_tensor.cuh"
#include "cfa_tile.cuh"

namespace cfa {

constexpr int kLatChunk = 64 * 128;        // 64 rows of 64 dims
// a block of keys takes three slots of three chunks of keys and two slots of four chunks of values
// (both key halves of 128 dims): each wait, arrival and commit costs its warp 100 clocks or more, which slots of
// single chunks could not hide (5000 clocks a block instead of NNNN)
constexpr int kLatKSlots = 3, kLatKSlot = 3 * kLatChunk, kLatVSlots = 2, kLatVSlot = 4 * kLatChunk;
constexpr int kLatQChunks = kLatRow / 64;  // 9
constexpr int kLatShare = 1;                // least units of a run
constexpr int kLatWarps = kLatAttnThreads / 32;

// Shared memory, the same in both blocks of a cluster (an instruction that spans them has one
// offset for both).
struct LatSmem {
    static constexpr int kQ = 0;                                 // [9][64 rows][128 bytes]
    static constexpr int kP = kQ + kLatQChunks * kLatChunk;      // [2 key halves][64 rows][128 bytes]
    static constexpr int kK = kP + 2 * kLatChunk;                // ring of [3][64 keys][128 bytes]
    static constexpr int kV = kK + kLatKSlots * kLatKSlot;       // ring of [2 key halves][2][64 keys][128 bytes]
    static constexpr int kBars = kV + kLatVSlots * kLatVSlot;
    static constexpr int kFullK = kBars, kEmptyK = kFullK + 8 * kLatKSlots, kReadyK = kEmptyK + 8 * kLatKSlots;
    static constexpr int kFullV = kReadyK + 8 * kLatKSlots, kEmptyV = kFullV + 8 * kLatVSlots,
                         kReadyV = kEmptyV + 8 * kLatVSlots;
    static constexpr int kFullQ = kReadyV + 8 * kLatVSlots, kEmptyQ = kFullQ + 8, kReadyQ = kEmptyQ + 8;
    static constexpr int kScores = kReadyQ + 8, kWeights = kScores + 16, kSum = kWeights + 8, kDrain = kSum + 8;
    static constexpr int kBarsEnd = kDrain + 8;
    static constexpr int kMisc = kBarsEnd;                       // flags, TMEM address, run's start
    static constexpr int kSums = kMisc + 64;                     // int [9]: the scan's sums
    static constexpr int kMax = kSums + 64;                      // float [2][2][64]: maxima of a row's halves
    static constexpr int kBytes = kMax + 1024;
};
static_assert(LatSmem::kMisc % 8 == 0 && LatSmem::kBytes <= 227 * 1024, "it fits");

// Arrive on the barrier at this offset in both blocks once all earlier products have ended.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
// D[tmem] (+)= A[smem] . B[smem] of both blocks, issued by one thread of the first.
__device__ __forceinline__ void umma2_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}
// Arrives on a barrier of either block (an address from map_to_rank). What it tells of are writes of the
// asynchronous proxy, or ones that a proxy fence has put in front of it, to the arriving
// block's own shared memory, which that block's own tensor core reads. The form that releases at cluster scope
// takes 1100 clocks each time: 16,000 for a block of keys that should take 3000.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(remote_bar) : "memory");
}
// By one warp of each block.
__device__ __forceinline__ void tmem2_alloc(uint32_t slot_smem_addr, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(slot_smem_addr), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ int latent_length(const LatentAttnParams &p, int b) {
    const int len = __ldcg(p.lens + b);
    return len < 0 || len > static_cast<long long>(p.width) * p.page_size ? 0 : len;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLatAttnThreads, 1)
latent_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_rows,
                        const __grid_constant__ LatentAttnParams p) {
    using S = LatSmem;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    const int rank = static_cast<int>(cluster_ctarank()), run = static_cast<int>(blockIdx.x) >> 1;
    int *misc = reinterpret_cast<int *>(smem + S::kMisc);
    volatile int *timed_out = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);

    // a thread a barrier, with the arrivals it expects
    if (tid < (S::kBarsEnd - S::kBars) / 8) {
        const int at = S::kBars + 8 * tid;
        uint32_t count = 1;
        if ((at >= S::kReadyK && at < S::kFullV) || (at >= S::kReadyV && at < S::kFullQ) || at == S::kReadyQ)
            count = 2;  // the relays of both blocks
        if (at == S::kWeights) count = 8;  // the compute warps of both
        mbar_init(base + at, count);
        fence_mbar_init();
    }
    if (tid == 0) misc[0] = 0;
    if (warp == kLatMmaWarp) tmem2_alloc(smem_addr(tmem_slot), 512);
    if (warp == kLatLoadWarp && elect_one()) {
        prefetch_tensor_map(&tm_q);
        prefetch_tensor_map(&tm_rows);
    }
    __syncwarp();
    tcgen05_fence_before();
    cluster_arrive();  // (the other block's barriers are ready behind the wait below)
    grid_dependency_wait();

    // ---- every block scans the requests, each thread some of them
    LatentWalk walk;
    auto request = [&](int b) {
        const int tok0 = __ldcg(p.cu + b);
        return LatentRequest{tok0, __ldcg(p.cu + b + 1) - tok0, latent_length(p, b)};
    };
    {
        int *sums = reinterpret_cast<int *>(smem + S::kSums);
        const int per = (p.B + kLatAttnThreads - 1) / kLatAttnThreads, first = tid * per, last = min(p.B, first + per);
        auto more = [](int a, int b) { return min(a + b, kLatMaxUnits); };
        int units = 0;
        bool bad = false;
        CFA_ROLLED for (int b = first; b < last; ++b) {
            LatentRequest r = request(b);
            if (r.tok0 < 0 || r.n < 0 || r.n > p.T || r.tok0 > p.T - r.n) bad = true;
            else units = more(units, latent_units(r, p.H, p.by_H));
            if (blockIdx.x == 0) {
                const int len = __ldcg(p.lens + b);
                if (len < 0 || len > static_cast<long long>(p.width) * p.page_size) atomicOr(p.status, kStatusBadLengthBit);
            }
        }
        int scan = units;
        CFA_ROLLED for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, scan, o);
            if (lane >= o) scan = more(scan, v);
        }
        if (lane == 31) sums[warp] = scan;
        if (tid == 0) misc[2] = -1;
        const bool refused = __syncthreads_or(bad) != 0;
        int before = 0, all = 0;
        CFA_ROLLED for (int w = 0; w < kLatWarps; ++w) {
            if (w < warp) before = more(before, sums[w]);
            all = more(all, sums[w]);
        }
        const bool valid = !refused && all < kLatMaxUnits;
        if (blockIdx.x == 0 && tid == 0 && !valid) atomicOr(p.status, kStatusBadLengthBit);
        const int share = max(kLatShare, (all + p.runs - 1) / p.runs);
        const long long from = static_cast<long long>(run) * share;
        const int u0 = valid ? static_cast<int>(min(from, static_cast<long long>(all))) : 0;
        const int u1 = valid ? static_cast<int>(min(from + share, static_cast<long long>(all))) : 0;
        // the thread in whose requests the run begins
        int at = more(before, scan - units);
        if (u0 < u1 && u0 >= at && u0 < at + units) {
            int b = first;
            CFA_ROLLED for (; b < last; ++b) {
                const int c = latent_units(request(b), p.H, p.by_H);
                if (u0 < at + c) break;
                at += c;
            }
            misc[2] = b;
            misc[3] = at;
        }
        if (tid == 0) misc[4] = share;
        __syncthreads();
        tcgen05_fence_after();
        walk.begin(u0, misc[2] < 0 ? u0 : u1, misc[2], misc[3], p.H, p.by_H, request);
    }
    grid_dependents_launch();
    cluster_wait();
    const uint32_t tmem = *tmem_slot;
    auto next = [&]() { return walk.next(p.B, p.H, p.by_H, request); };
    const LatentPiece &x = walk.x;
    auto wait = [&](int bar, uint32_t parity, unsigned site) {
        return bounded_wait([&]() { return mbar_try_wait(base + bar, parity); }, p.timeout_ns, timed_out,
                            p.status, site);
    };
    // The same for a warp as a whole.
    auto wait_warp = [&](int bar, uint32_t parity, unsigned site) { return __all_sync(~0u, wait(bar, parity, site)); };
    // cache rows that the last token of the piece's tile sees, and the first
    auto seen_by_last = [&]() { return latent_visible(x.r, min(x.r.n - 1, (x.tile * kLatTile + kLatTile - 1) / p.by_H)); };
    auto seen_by_first = [&]() { return latent_visible(x.r, (x.tile * kLatTile) / p.by_H); };

    if (warp == kLatLoadWarp || warp == kLatLoadWarp + 1) {
        // ------------------------------------------------ load warps: keys (and queries), values
        const bool values = warp != kLatLoadWarp;
        // boxes of 64 keys: 1, 2 or 4 (shifts: a division takes 150 clocks, and a chunk has no more than 350)
        const int box = p.box_rows, bits = box == 64 ? 0 : box == 32 ? 1 : 2, per_half = 1 << bits;
        const int all_rows = p.n_pages * p.page_size;     // outside: reads as zeros
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        // Where the boxes of the tile's 64-key halves lie is found 32 boxes at a time, a lane a box.
        while (ok && next()) {
            if (x.b0 == x.b1) continue;
            if (!values) {
                if (pieces > 0) ok = wait_warp(S::kEmptyQ, (pieces - 1) & 1, kSiteStageEmpty);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(base + S::kFullQ, kLatQChunks * kLatChunk);
                    const int row = x.r.tok0 * p.H + x.tile * kLatTile + 64 * rank;
#pragma unroll 1
                    for (int c = 0; c < kLatQChunks; ++c)
                        tma_load_2d(base + S::kQ + c * kLatChunk, &tm_q, 64 * c, row, base + S::kFullQ);
                }
                __syncwarp();
            }
            ++pieces;
            const int keys = seen_by_last();
            const int *table = p.tables + static_cast<size_t>(x.req) * p.width;
            int rows = 0, cached = -1;  // this lane's box, of group `cached`
            // cache rows of a half's boxes
            auto boxes = [&](int half, int (&y)[4]) {
                const int group = half >> (5 - bits);
                if (group != cached) {
                    cached = group;
                    const int key = (group * 32 + lane) * box;
                    rows = all_rows;
                    if (key < keys) {
                        const int pg = key / p.by_page, id = __ldcg(table + pg);
                        if (id >= 0 && id < p.n_pages) rows = id * p.page_size + key - pg * p.page_size;
                        else atomicOr(p.status, kStatusBadPageBit);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(~0u, rows, ((half << bits) + i) & 31);
            };
            CFA_ROLLED for (int b = x.b0; ok && b < x.b1; ++b) {
                if (!values) {
                    int y[4];
                    boxes(2 * b + rank, y);
                    CFA_ROLLED for (int c = 0; c < kLatKSlots; ++c, ++n) {
                        const int full = S::kFullK + 8 * c;
                        if (n >= kLatKSlots) ok = wait_warp(S::kEmptyK + 8 * c, (n / kLatKSlots - 1) & 1, kSiteStageEmpty);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(base + full, kLatKSlot);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i >= per_half) break;
#pragma unroll
                                for (int k = 0; k < 3; ++k)
                                    tma_load_2d(base + S::kK + c * kLatKSlot + k * kLatChunk + i * box * 128, &tm_rows,
                                                64 * (3 * c + k), y[i], base + full);
                            }
                        }
                        __syncwarp();
                    }
                } else {
                    int y[2][4];
                    boxes(2 * b, y[0]);
                    boxes(2 * b + 1, y[1]);
                    CFA_ROLLED for (int c = 0; c < kLatVSlots; ++c, ++n) {
                        const int full = S::kFullV + 8 * c, dim = 256 * rank + 128 * c;
                        if (n >= kLatVSlots) ok = wait_warp(S::kEmptyV + 8 * c, (n / kLatVSlots - 1) & 1, kSiteStageEmpty);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(base + full, kLatVSlot);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i >= per_half) break;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tma_load_2d(base + S::kV + c * kLatVSlot + k * kLatChunk + i * box * 128, &tm_rows,
                                                dim + 64 * (k & 1), y[k >> 1][i], base + full);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (lane == 0 && *timed_out) {
            // a wait gave up: the copies in flight land before the block ends
            const uint64_t t0 = global_timer_ns();
            const uint32_t slots = values ? kLatVSlots : kLatKSlots;
            auto land = [&](uint32_t bar, uint32_t parity) {
                while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
            };
            for (uint32_t k = n > slots ? n - slots : 0; k < n; ++k)
                land(base + (values ? S::kFullV : S::kFullK) + 8 * (k % slots), (k / slots) & 1);
            if (!values && pieces > 0) land(base + S::kFullQ, (pieces - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kLatLoadWarp + 2) {
        // ------------------------------------------------------------------- relay warp
        // in the order in which the products take them: queries, keys of a block ahead, values
        uint32_t nk = 0, nv = 0, pieces = 0;  // blocks and pieces so far
        const uint32_t ready_k = map_to_rank(base + S::kReadyK, 0), ready_v = map_to_rank(base + S::kReadyV, 0),
                       ready_q = map_to_rank(base + S::kReadyQ, 0);
        bool ok = true;
        auto keys = [&]() {
            CFA_ROLLED for (int c = 0; ok && c < kLatKSlots; ++c) {
                ok = wait_warp(S::kFullK + 8 * c, nk & 1, kSiteStageFull);
                if (ok && elect_one()) mbar_arrive_pair(ready_k + 8 * c);
                __syncwarp();
            }
            ++nk;
        };
        while (ok && next()) {
            if (x.b0 == x.b1) continue;
            ok = wait_warp(S::kFullQ, pieces++ & 1, kSiteStageFull);
            if (ok && elect_one()) mbar_arrive_pair(ready_q);
            __syncwarp();
            const int all = seen_by_last(), some = seen_by_first();
            keys();
            CFA_ROLLED for (int b = x.b0; ok && b < x.b1; ++b, ++nv) {
                if (b + 1 < x.b1) keys();
                const int begin = max(0, some - b * kLatKeys);
                CFA_ROLLED for (int c = 0; ok && c < kLatVSlots; ++c) {
                    ok = wait_warp(S::kFullV + 8 * c, nv & 1, kSiteStageFull);
                    if (ok && begin < kLatKeys) {
                        // keys from `some` on are not seen by every row, from `all` on by none
                        uint8_t *v = smem + S::kV + c * kLatVSlot;
                        CFA_ROLLED for (int i = lane; i < (kLatKeys - begin) * 16; i += 32) {
                            const int r = begin + (i >> 4);
                            uint4 *at = reinterpret_cast<uint4 *>(v + ((r >> 6) * 2 + ((i >> 3) & 1)) * kLatChunk +
                                                                  (r & 63) * 128 + ((i & 7) << 4));
                            uint4 w = make_uint4(0u, 0u, 0u, 0u);
                            if (b * kLatKeys + r < all) {
                                w = *at;
                                const uint32_t f = odd_bf16x2(w.x), g = odd_bf16x2(w.y), h = odd_bf16x2(w.z), k = odd_bf16x2(w.w);
                                if ((f | g | h | k) == 0u) continue;
                                w = make_uint4(w.x & ~f, w.y & ~g, w.z & ~h, w.w & ~k);
                            }
                            *at = w;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (ok && elect_one()) mbar_arrive_pair(ready_v + 8 * c);
                    __syncwarp();
                }
            }
        }
    } else if (warp == kLatMmaWarp) {
        // --------------------------------------------------------- products, by the first block
        if (rank == 0) {
            const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
            const uint32_t idesc_s = umma_idesc_bf16(128, 128, false, false), idesc_o = umma_idesc_bf16(128, 256, false, true);
            uint32_t g = 0, pieces = 0;  // blocks and pieces so far
            bool ok = true;
            auto scores = [&](uint32_t block, bool last) {
                const uint64_t q0 = umma_smem_desc(base + S::kQ, 16, 1024), k0 = umma_smem_desc(base + S::kK, 16, 1024);
                CFA_ROLLED for (int c = 0; ok && c < kLatKSlots; ++c) {
                    ok = wait_warp(S::kReadyK + 8 * c, block & 1, kSiteStageFull);
                    tcgen05_fence_after();
                    if (ok && elect_one()) {
                        const uint64_t a = q0 + c * (kLatKSlot >> 4), b = k0 + c * (kLatKSlot >> 4);
#pragma unroll
                        for (int ks = 0; ks < 12; ++ks)  // 32 bytes a step
                            umma2_bf16(tm + 64 * (block & 1), a + (ks >> 2) * (kLatChunk >> 4) + 2 * (ks & 3),
                                       b + (ks >> 2) * (kLatChunk >> 4) + 2 * (ks & 3), idesc_s, c > 0 || ks > 0);
                        umma2_commit(base + S::kEmptyK + 8 * c);
                        if (c == kLatKSlots - 1) {
                            umma2_commit(base + S::kScores + 8 * (block & 1));
                            if (last) umma2_commit(base + S::kEmptyQ);
                        }
                    }
                    __syncwarp();
                }
            };
            while (ok && next()) {
                const int nb = x.b1 - x.b0;
                if (nb == 0) continue;
                ok = wait_warp(S::kReadyQ, pieces++ & 1, kSiteQExchange);
                scores(g, nb == 1);
                CFA_ROLLED for (int j = 0; ok && j < nb; ++j, ++g) {
                    if (j + 1 < nb) scores(g + 1, j + 2 == nb);
                    ok = ok && wait_warp(S::kWeights, g & 1, kSiteSoftmaxExchange);
                    const uint64_t p0 = umma_smem_desc(base + S::kP, 16, 1024), v0 = umma_smem_desc(base + S::kV, kLatChunk, 1024);
                    CFA_ROLLED for (int c = 0; ok && c < kLatVSlots; ++c) {
                        ok = wait_warp(S::kReadyV + 8 * c, g & 1, kSiteStageFull);
                        tcgen05_fence_after();
                        if (ok && elect_one()) {
                            const uint64_t v = v0 + c * (kLatVSlot >> 4);
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)  // 16 keys of 128 bytes a step
                                umma2_bf16(tm + 128 + 128 * c, p0 + (ks >> 2) * (kLatChunk >> 4) + 2 * (ks & 3),
                                           v + (ks >> 2) * (2 * kLatChunk >> 4) + 128 * (ks & 3), idesc_o, j > 0 || ks > 0);
                            umma2_commit(base + S::kEmptyV + 8 * c);
                            if (c == kLatVSlots - 1) umma2_commit(base + S::kSum);
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one() && *timed_out) {
                // a wait gave up: the products in flight end before the blocks do
                umma2_commit(base + S::kDrain);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait_cluster(base + S::kDrain, 0) &&
                       global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
            }
            __syncwarp();
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------ compute warps
        const int half = warp >> 1, row = (warp & 1) * 32 + lane;  // of the block's 64
        const uint32_t lanes = static_cast<uint32_t>(warp) << 21;   // TMEM lanes of this warp
        float *maxima = reinterpret_cast<float *>(smem + S::kMax);
        const uint32_t weights = map_to_rank(base + S::kWeights, 0);
        uint32_t g = 0;
        int4 cut = make_int4(0, 0, 0, 0);  // the tile that the run's end cuts, for the merge
        // the other half of a row's thread, 64 threads on
        auto meet = [&]() { compute_bar<128>(); };
        while (next()) {
            const int in_request = x.tile * kLatTile + 64 * rank + row;  // the query row
            const int all = x.r.n * p.H;
            const bool live = in_request < all;
            const bool warp_live = in_request - lane < all;
            const int see = live ? latent_visible(x.r, in_request / p.by_H) : 0;
            float m = -INFINITY, l = 0.f;
            CFA_ROLLED for (int b = x.b0; b < x.b1; ++b, ++g) {
                wait(S::kScores + 8 * (g & 1), (g >> 1) & 1, kSiteSoftmaxExchange);
                __syncwarp();
                tcgen05_fence_after();
                uint32_t s[64];
                float top = -INFINITY;
                if (warp_live) {
                    tmem_ld_x32(tmem + lanes + 64 * (g & 1), s);
                    tmem_ld_x32(tmem + lanes + 64 * (g & 1) + 32, s + 32);
                    tmem_wait_ld();
                    const int lim = see - b * kLatKeys - 64 * half;
                    if (!__all_sync(~0u, lim >= 64)) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) s[c] = c < lim ? s[c] : 0xff800000u;
                    }
                    float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        a[(c >> 1) & 3] = fmaxf(fmaxf(a[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                    top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * p.scale_log2;
                }
                float *mx = maxima + 128 * (g & 1);
                mx[64 * half + row] = top;
                meet();
                top = fmaxf(top, mx[64 * (half ^ 1) + row]);
                // both halves of a row come to the same answer
                const bool raise = __any_sync(~0u, top > m + 8.f);
                float scale = 1.f;
                if (raise) {
                    const float mn = fmaxf(m, top);
                    scale = m == mn ? 1.f : exp2_ftz(m - mn);
                    m = mn;
                    l *= scale;
                }
                uint32_t w[32];
                if (warp_live) {
                    const float f = m == -INFINITY ? 0.f : -m;
                    const uint64_t scale2 = pair_f32(p.scale_log2, p.scale_log2), f2 = pair_f32(f, f);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 y = unpair_f32(fma_f32x2(
                            pair_f32(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, f2));
                        const float x0 = exp2_ftz(y.x), x1 = exp2_ftz(y.y);
                        sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(x0, x1));
                        w[e] = pack2_bf16_cvt(x0, x1);
                    }
                    const float2 both = unpair_f32(add_f32x2(sum[0], sum[1]));
                    l += both.x + both.y;
                }
                // the last block's sum is done: O and P are free
                if (g > 0) wait(S::kSum, (g - 1) & 1, kSiteKvExchange);
                __syncwarp();
                tcgen05_fence_after();
                if (warp_live) {
                    if (raise && b > x.b0) {
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            uint32_t v[32];
                            tmem_ld_x32(tmem + lanes + 128 + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * scale);
                            tmem_st_x16(tmem + lanes + 128 + c, v);
                            tmem_st_x16(tmem + lanes + 128 + c + 16, v + 16);
                        }
                        tmem_wait_st();
                    }
                    uint8_t *to = smem + S::kP + half * kLatChunk + row * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4 *>(to + ((c ^ (row & 7)) << 4)) =
                            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                }
                fence_proxy_async_smem();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(weights);
            }
            // ---- the tile's results, or its record
            const bool any = x.b1 > x.b0, final = x.b0 == 0 && x.b1 == x.blocks, begins = x.b0 == 0;
            if (any) wait(S::kSum, (g - 1) & 1, kSiteKvExchange);
            __syncwarp();
            tcgen05_fence_after();
            float *sums = maxima + 128 * (g & 1);  // (the other buffer may still be read)
            sums[64 * half + row] = l;
            meet();
            l += sums[64 * (half ^ 1) + row];
            meet();  // the next block's maxima go to the same place
            const long long out_row = static_cast<long long>(x.r.tok0) * p.H + in_request;
            const int rec = 2 * run + (begins ? 1 : 0);
            float *rec_o = p.rec_o + static_cast<size_t>(rec) * kLatTile * kLatC;
            if (!final && begins && rank == 0 && tid == 0) {
                const int share = misc[4], tile_rows = min(kLatTile, all - x.tile * kLatTile);
                cut = make_int4(tile_rows, static_cast<int>(out_row), (x.unit + x.blocks + kLatItem - 1) / share, 0);
            }
            if (warp_live) {
                if (half == 0 && live) {
                    if (!final) p.rec_ml[rec * kLatTile + 64 * rank + row] = make_float2(m, l);
                    else if (p.lse) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t v[32];
                    __syncwarp();
                    if (any) {
                        tmem_ld_x32(tmem + lanes + 128 + c, v);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0u;
                    }
                    if (!live) continue;
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
                    const int dim = 256 * half + c;
                    if (final) {
                        if (see == 0) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = 0.f;
                        }
                        uint16_t *out = p.out + static_cast<size_t>(out_row) * kLatC + dim;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4 *>(out + 8 * e) =
                                make_uint4(pack2_bf16_cvt(f[8 * e] * inv, f[8 * e + 1] * inv),
                                           pack2_bf16_cvt(f[8 * e + 2] * inv, f[8 * e + 3] * inv),
                                           pack2_bf16_cvt(f[8 * e + 4] * inv, f[8 * e + 5] * inv),
                                           pack2_bf16_cvt(f[8 * e + 6] * inv, f[8 * e + 7] * inv));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(rec_o + (static_cast<size_t>(dim / 4 + e) * kLatTile + 64 * rank + row) * 4) =
                                make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
            }
            tcgen05_fence_before();
        }
        if (rank == 0 && tid == 0) p.cuts[run] = cut;
    }
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();  // nothing of either block reaches into the other any more
    if (warp == kLatMmaWarp) {
        tcgen05_fence_after();
        tmem2_dealloc(tmem, 512);
    }
}

// Merges the records of the tiles that runs' ends cut: blockIdx.y is the run in which such a tile
// begins; a warp takes 32 rows (a lane a row) and 8 of their dims, eight records at a time, so that their loads
// are on their way together.
__global__ void __launch_bounds__(kLatMergeThreads) latent_merge_kernel(const __grid_constant__ LatentAttnParams p) {
    constexpr int N = 8, CH = 2;
    grid_dependency_wait();
    const int run = blockIdx.y, lane = threadIdx.x & 31;
    const int4 cut = __ldcg(p.cuts + run);  // rows, the first one's place, the tile's last run
    const int task = blockIdx.x * (kLatMergeThreads / 32) + (threadIdx.x >> 5);
    const int row = task % (kLatTile / 32) * 32 + lane, chunk = task / (kLatTile / 32) * CH;
    if (row < cut.x) {
        const float2 *ml = p.rec_ml + row;
        const float4 *o = reinterpret_cast<const float4 *>(p.rec_o) + static_cast<size_t>(chunk) * kLatTile + row;
        constexpr int kRec = kLatTile * (kLatC / 4);
        float m = -INFINITY, l = 0.f;
        float a[4 * CH] = {};
        CFA_ROLLED for (int k = run; k <= cut.z; k += N) {
            float2 s[N];
            float4 v[N][CH];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int c = 0; c < CH; ++c) v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k + i <= cut.z) {
                    const int rec = 2 * (k + i) + (k + i == run);  // the first run's second record, the others' first
                    s[i] = __ldcg(ml + rec * kLatTile);
#pragma unroll
                    for (int c = 0; c < CH; ++c) v[i][c] = __ldcg(o + static_cast<size_t>(rec) * kRec + c * kLatTile);
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < N; ++i) top = fmaxf(top, s[i].x);
            const float f = top == -INFINITY ? 0.f : top, g0 = exp2_ftz(m - f);
            m = top;
            l *= g0;
#pragma unroll
            for (int e = 0; e < 4 * CH; ++e) a[e] *= g0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = exp2_ftz(s[i].x - f);
                l += g * s[i].y;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    a[4 * c] += g * v[i][c].x; a[4 * c + 1] += g * v[i][c].y;
                    a[4 * c + 2] += g * v[i][c].z; a[4 * c + 3] += g * v[i][c].w;
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t *out = p.out + (static_cast<size_t>(cut.y) + row) * kLatC + 4 * chunk;
        static_assert(CH == 2, "16 bytes");
        *reinterpret_cast<uint4 *>(out) = l == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                                   : make_uint4(pack2_bf16_cvt(a[0] * inv, a[1] * inv), pack2_bf16_cvt(a[2] * inv, a[3] * inv),
                                                                pack2_bf16_cvt(a[4] * inv, a[5] * inv), pack2_bf16_cvt(a[6] * inv, a[7] * inv));
        if (p.lse && chunk == 0) p.lse[static_cast<size_t>(cut.y) + row] = (m + log2f(l)) * 0.69314718055994531f;
    }
    grid_dependents_launch();
}

}  // namespace cfa
