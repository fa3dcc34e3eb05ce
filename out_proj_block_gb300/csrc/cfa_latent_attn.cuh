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
// inside one page), and one that passes on what has landed, as the issuing block waits for both blocks' copies.
// Values that some or all rows do not see are cleared before the product, by the compute warps: a masked
// weight is 0, and 0 times NaN is NaN.
//
// Tiles are cut into runs of blocks of keys, one to a cluster (cfa_latent_split.h); what the
// runs' ends cut leaves records, which a second kernel merges in the order of the runs, so results
// are bitwise reproducible. A row's maximum is followed lazily: o is the same quotient whatever m is, as both of
// its sums carry 2^-m, so O is rescaled only when the maximum grew by more than 8 (weights up to 2^8, far
// inside fp32).
//
// Measured, with the merge (one GB300): 64 requests of some 8K rows, 128 heads 87 us (385 MB read once;
// floor 57); 200 of some 2K, 32 heads 72 us (floor 47); 16 with up to four drafted tokens, 20 heads 24 us; one of 4K
// rows 15.5 us. In the middle of a run memory bounds it, at 6.2 TB/s (products take 2490 clocks of a block of keys,
// the rows 2900); beside that stand the start (scan, first queries and keys: 8 us), the cut tiles' records (1 to 6 us,
// and 5 to 10 to merge them, 2 of which the launch takes) and, with short requests, a tile's end, some 8000 clocks.
// Merging in the block that ends last instead of in a second kernel took 16 us more for the first of these; merging by
// all blocks behind a wait for one another wants a cooperative launch, which costs 2 us by itself.
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
#include "cfa_tensor_pair.cuh"
#include "cfa_tile.cuh"

namespace cfa {

constexpr int kLatChunk = 64 * 128;        // 64 rows of 64 dims
// a block of keys takes three slots of three chunks of keys and two slots of four chunks of values
// (both key halves of 128 dims): each wait, arrival and commit costs its warp 100 clocks or more, which slots of
// single chunks could not hide (5000 clocks a block instead of 2500)
constexpr int kLatKSlots = 3, kLatKSlot = 3 * kLatChunk, kLatVSlots = 2, kLatVSlot = 4 * kLatChunk;
constexpr int kLatQChunks = kLatRow / 64;  // 9
// Measured with three sets of inputs in turn, which come out 1 to 4% apart from the figures above:
constexpr int kLatAhead = 1;                // blocks of keys that are asked for in L2 ahead of their copies (64 requests of
                                            // some 8K rows, 128 heads: with 1, 2, 3, 4, 6 84, 87, 91, 98, 113 us)
constexpr int kLatPeek = 3;                 // blocks before a tile's end that the next one's first data are asked for
constexpr int kLatShare = 2;                // least units of a run (1, 2, 4: one request of 4K rows 18.0, 16.0, 17.8 us)
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

// Asks for contiguous bytes in L2 (address and size multiples of 16).
__device__ __forceinline__ void bulk_prefetch_l2(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(src), "r"(bytes) : "memory");
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
    if (warp == kLatLoadWarp + 1 && elect_one()) {
        // every block asks for its share of the queries in L2 before the plan says whose they are (0.5 to 0.8 us of 25 to
        // 90 where they are not there yet; more than this many would push one another out)
        const long long rows = static_cast<long long>(p.T) * p.H, share = (rows + gridDim.x - 1) / gridDim.x, at = share * blockIdx.x;
        if (share <= 96 && at < rows) bulk_prefetch_l2(p.q + at * kLatRow, static_cast<uint32_t>(min(share, rows - at)) * kLatRow * 2);
    }
    __syncwarp();
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
        int units = 0;
        bool bad = false;
        LatentRequest r{};  // (with no more requests than threads read once)
        CFA_ROLLED for (int b = first; b < last; ++b) {
            r = request(b);
            if (r.tok0 < 0 || r.n < 0 || r.n > p.T || r.tok0 > p.T - r.n) bad = true;
            else units = latent_more(units, latent_units(r, p.H, p.by_H));
            if (blockIdx.x == 0) {
                const int len = __ldcg(p.lens + b);
                if (len < 0 || len > static_cast<long long>(p.width) * p.page_size) atomicOr(p.status, kStatusBadLengthBit);
            }
        }
        int scan = units;
        CFA_ROLLED for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, scan, o);
            if (lane >= o) scan = latent_more(scan, v);
        }
        if (lane == 31) sums[warp] = scan;
        if (tid == 0) misc[2] = -1;
        const bool refused = __syncthreads_or(bad) != 0;
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kLatWarps; ++w) {
            if (w < warp) before = latent_more(before, sums[w]);
            all = latent_more(all, sums[w]);
        }
        const bool valid = !refused && latent_fits(all);
        if (blockIdx.x == 0 && tid == 0 && !valid) atomicOr(p.status, kStatusBadLengthBit);
        const int share = max(kLatShare, (all + p.runs - 1) / p.runs);
        const long long from = static_cast<long long>(run) * share;
        const int u0 = valid ? static_cast<int>(min(from, static_cast<long long>(all))) : 0;
        const int u1 = valid ? static_cast<int>(min(from + share, static_cast<long long>(all))) : 0;
        // the thread in whose requests the run begins
        int at = latent_more(before, scan - units);
        if (u0 < u1 && u0 >= at && u0 < at + units) {
            int b = first;
            CFA_ROLLED for (; per > 1 && b < last; ++b) {
                r = request(b);
                const int c = latent_units(r, p.H, p.by_H);
                if (u0 < at + c) break;
                at += c;
            }
            misc[2] = b;
            misc[3] = at;
            misc[5] = r.tok0;
            misc[6] = r.n;
            misc[7] = r.len;
        }
        if (tid == 0) misc[4] = share;
        __syncthreads();
        tcgen05_fence_after();
        walk.begin(u0, misc[2] < 0 ? u0 : u1, misc[2], LatentRequest{misc[5], misc[6], misc[7]}, misc[3], p.H, p.by_H);
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
    // cache rows that the last token of the piece's tile sees
    auto seen_by_last = [&]() { return latent_visible(x.r, min(x.r.n - 1, (x.tile * kLatTile + kLatTile - 1) / p.by_H)); };

    if (warp == kLatLoadWarp || warp == kLatLoadWarp + 1) {
        // ------------------------------------------------ load warps: keys (and queries), values
        const bool values = warp != kLatLoadWarp;
        // boxes of 64 keys: 1, 2 or 4 (shifts: a division takes 150 clocks, and a chunk has no more than 350)
        const int box = p.box_rows, bits = box == 64 ? 0 : box == 32 ? 1 : 2, per_half = 1 << bits;
        const int all_rows = p.n_pages * p.page_size;     // outside: reads as zeros
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        auto first_row = [&](const LatentPiece &z) {  // of this block's queries
            return z.r.tok0 * p.H + z.tile * kLatTile + rank * latent_split(latent_rows(z.r, p.H, z.tile));
        };
        // Where the boxes of the tile's 64-key halves lie is found 32 boxes at a time, a lane a box.
        while (ok && next()) {
            if (x.b0 == x.b1) continue;
            const int keys = seen_by_last();
            const int *table = p.tables + static_cast<size_t>(x.req) * p.width;
            // cache rows of a 64-key half's boxes; `at` and `ahead` hold this lane's box of a group of 32
            struct Boxes {
                int group = -1, row;
            } at, ahead;
            auto find = [&](Boxes &f, int half) {
                const int group = half >> (5 - bits);
                if (group == f.group) return;
                const int found = at.group;
                f.group = group;
                if (group == found) {  // (the copies' group, already found)
                    f.row = at.row;
                    return;
                }
                const int key = (group * 32 + lane) * box;
                f.row = all_rows;
                if (key < keys) {
                    const int pg = key / p.by_page, id = __ldcg(table + pg);
                    if (id >= 0 && id < p.n_pages) f.row = id * p.page_size + key - pg * p.page_size;
                    else atomicOr(p.status, kStatusBadPageBit);
                }
            };
            auto boxes = [&](int half, int (&y)[4]) {
                find(at, half);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(~0u, at.row, ((half << bits) + i) & 31);
            };
            // asks for a half's rows in L2, a lane a box
            auto prefetch = [&](int half) {
                find(ahead, half);
                if (lane >> bits == (half & ((32 >> bits) - 1)) && ahead.row < all_rows)
                    bulk_prefetch_l2(p.pages + static_cast<size_t>(ahead.row) * kLatRow, static_cast<uint32_t>(box) * kLatRow * 2);
                __syncwarp();
            };
            int asked = x.b0;  // the last block that L2 has been asked for
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
                    if (b == x.b0 && ok) {  // (behind the keys: the last tile's scores free them first)
                        if (pieces > 0) ok = wait_warp(S::kEmptyQ, (pieces - 1) & 1, kSiteStageEmpty);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(base + S::kFullQ, kLatQChunks * kLatChunk);
#pragma unroll 1
                            for (int c = 0; c < kLatQChunks; ++c)
                                tma_load_2d(base + S::kQ + c * kLatChunk, &tm_q, 64 * c, first_row(x), base + S::kFullQ);
                        }
                        __syncwarp();
                        ++pieces;
                    }
                    CFA_ROLLED for (int k = 0; ok && k < 2 && asked < min(b + kLatAhead, x.b1 - 1); ++k) prefetch(2 * ++asked + rank);
                    if (b == max(x.b0, x.b1 - kLatPeek)) {
                        // the next tile's queries and first keys, in L2 by the time they are loaded
                        LatentWalk peek = walk;
                        if (peek.next(p.B, p.H, p.by_H, request) && peek.x.b0 < peek.x.b1) {
                            const LatentPiece &z = peek.x;
                            const int key = (2 * z.b0 + rank) * 64 + lane * box;
                            if (lane < per_half && key < latent_visible(z.r, z.r.n - 1)) {
                                const int pg = key / p.by_page, id = __ldcg(p.tables + static_cast<size_t>(z.req) * p.width + pg);
                                if (id >= 0 && id < p.n_pages)
                                    bulk_prefetch_l2(p.pages + (static_cast<size_t>(id) * p.page_size + key - pg * p.page_size) * kLatRow,
                                                     static_cast<uint32_t>(box) * kLatRow * 2);
                            }
                            const int rows = min(64, latent_rows(z.r, p.H, z.tile) - rank * latent_split(latent_rows(z.r, p.H, z.tile)));
                            if (lane == 31 && rows > 0)
                                bulk_prefetch_l2(p.q + static_cast<size_t>(first_row(z)) * kLatRow, static_cast<uint32_t>(rows) * kLatRow * 2);
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
            keys();
            CFA_ROLLED for (int b = x.b0; ok && b < x.b1; ++b, ++nv) {
                if (b + 1 < x.b1) keys();
                CFA_ROLLED for (int c = 0; ok && c < kLatVSlots; ++c) {
                    ok = wait_warp(S::kFullV + 8 * c, nv & 1, kSiteStageFull);
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
        bool more = next();
        while (more) {
            const LatentPiece z = x;
            const int tile_rows = latent_rows(z.r, p.H, z.tile), split = latent_split(tile_rows);
            const int here = rank ? tile_rows - split : split;         // rows of this block
            const int in_tile = rank * split + row;
            const bool live = row < here, warp_live = row - lane < here;
            // (rows past the last see what that one sees, so that their warp takes no masked blocks for them)
            const int see = latent_visible(z.r, (z.tile * kLatTile + rank * split + min(row, max(here, 1) - 1)) / p.by_H);
            const int some = latent_visible(z.r, (z.tile * kLatTile) / p.by_H);  // keys that every row sees
            const int all = latent_visible(z.r, (z.tile * kLatTile + tile_rows - 1) / p.by_H);  // and any
            float m = -INFINITY, l = 0.f;
            CFA_ROLLED for (int b = z.b0; b < z.b1; ++b, ++g) {
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
                    const float mn = top > m + 8.f ? top : m;  // (each row by itself: others must not change it)
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
                    if (raise && b > z.b0) {
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
                if (some < (b + 1) * kLatKeys) {
                    // keys from `some` on are not seen by every row, from `all` on by none: what is not
                    // finite of the first, and all of the others, becomes 0
                    const int begin = max(0, some - b * kLatKeys), end = min(kLatKeys, all - b * kLatKeys);
                    CFA_ROLLED for (int c = 0; c < kLatVSlots; ++c) {
                        wait(S::kFullV + 8 * c, g & 1, kSiteStageFull);
                        __syncwarp();
                        uint8_t *v = smem + S::kV + c * kLatVSlot + ((tid >> 3) & 1) * kLatChunk + ((tid & 7) << 4);
                        // (of a row's 16-byte chunks any order will do; the key halves lie 2 chunks apart)
                        auto at = [&](int r) { return reinterpret_cast<uint4 *>(v + r * 128 + (r >> 6) * kLatChunk); };
                        CFA_ROLLED for (int r = begin + (tid >> 4); r < end; r += 8) {
                            const uint4 d = *at(r);
                            const uint32_t f = odd_bf16x2(d.x), h = odd_bf16x2(d.y), i = odd_bf16x2(d.z), k = odd_bf16x2(d.w);
                            if ((f | h | i | k) != 0u) *at(r) = make_uint4(d.x & ~f, d.y & ~h, d.z & ~i, d.w & ~k);
                        }
#pragma unroll
                        for (int i = 0; i < kLatKeys / 8; ++i) {
                            const int r = 8 * i + (tid >> 4);
                            if (r >= end) *at(r) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                fence_proxy_async_smem();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(weights);
            }
            // ---- the tile's results, or its record
            const bool any = z.b1 > z.b0, final = z.b0 == 0 && z.b1 == z.blocks, begins = z.b0 == 0;
            more = next();  // (its loads are on their way meanwhile)
            if (any) wait(S::kSum, (g - 1) & 1, kSiteKvExchange);
            __syncwarp();
            tcgen05_fence_after();
            float *sums = maxima + 128 * (g & 1);  // (the other buffer may still be read)
            sums[64 * half + row] = l;
            meet();
            l += sums[64 * (half ^ 1) + row];
            meet();  // the next block's maxima go to the same place
            const long long tile_row = static_cast<long long>(z.r.tok0) * p.H + z.tile * kLatTile;
            const long long out_row = tile_row + in_tile;
            const int row_group = row - lane;  // the warp's first row
            if (!final && begins && rank == 0 && tid == 0)
                cut = make_int4(tile_rows, static_cast<int>(tile_row), (z.unit + z.blocks + kLatItem - 1) / misc[4], 0);
            if (!warp_live) continue;
            if (!final) {
                // a piece's record: the run's second where the tile begins in it, else its first
                const int rec = 2 * run + (begins ? 1 : 0);
                if (half == 0 && live) p.rec_ml[rec * kLatTile + in_tile] = make_float2(m, l);
                float *rec_o = p.rec_o + static_cast<size_t>(rec) * kLatTile * kLatC + 4 * in_tile;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_x32(tmem + lanes + 128 + c, v);
                    tmem_wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(rec_o + static_cast<size_t>(64 * half + c / 4 + e) * (4 * kLatTile)) =
                            make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
            } else {
                if (p.lse && half == 0 && live) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int odd = lane & 1;
                uint16_t *out = p.out + (out_row - odd) * kLatC + 256 * half + 8 * odd;
                const bool even_live = row - odd < here, odd_live = row - odd + 1 < here;
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
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack2_bf16_cvt(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
#pragma unroll
                    for (int h = 0; h < 2; ++h) write_rows_in_pairs(out + c + 16 * h, kLatC, w + 8 * h, even_live, odd_live);
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

// A warp's part of the merge of a tile: 32 rows, a lane a row, and kChunks times 4 dims; the records of its pieces are
// read kMost at a time.
template <int kChunks, int kMost>
__device__ __forceinline__ void latent_merge_rows(const LatentAttnParams &p, int4 cut, int run, int row0, int chunk) {
    constexpr int kRec = kLatTile * (kLatC / 4);
    const int lane = threadIdx.x & 31, row = row0 + lane, from = min(row, cut.x - 1), last = cut.z;
    const float2 *ml = p.rec_ml + from;
    const float4 *o = reinterpret_cast<const float4 *>(p.rec_o) + static_cast<size_t>(chunk) * kLatTile + from;
    float m = -INFINITY, l = 0.f, a[kChunks][4] = {};
    CFA_ROLLED for (int k = run; k <= last; k += kMost) {
        float2 s[kMost];
        float4 v[kMost][kChunks];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            s[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k + i <= last) {
                const int rec = 2 * (k + i) + (k + i == run);  // the first run's second record, the others' first
                s[i] = __ldcg(ml + rec * kLatTile);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) v[i][c] = __ldcg(o + static_cast<size_t>(rec) * kRec + c * kLatTile);
            }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kMost; ++i) top = fmaxf(top, s[i].x);
        const float f = top == -INFINITY ? 0.f : top, g0 = exp2_ftz(m - f);
        m = top;
        l *= g0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[c][e] *= g0;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const float g = exp2_ftz(s[i].x - f);
            l += g * s[i].y;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                a[c][0] += g * v[i][c].x; a[c][1] += g * v[i][c].y; a[c][2] += g * v[i][c].z; a[c][3] += g * v[i][c].w;
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[2 * kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        w[2 * c] = pack2_bf16_cvt(a[c][0] * inv, a[c][1] * inv);
        w[2 * c + 1] = pack2_bf16_cvt(a[c][2] * inv, a[c][3] * inv);
    }
    uint16_t *out = p.out + (static_cast<size_t>(cut.y) + row) * kLatC + 4 * chunk;
    if constexpr (kChunks >= 4) {
        const int odd = lane & 1;
#pragma unroll
        for (int h = 0; h < kChunks / 4; ++h)
            write_rows_in_pairs(out - odd * kLatC + 8 * odd + 16 * h, kLatC, w + 8 * h, row - odd < cut.x, row + 1 - odd < cut.x);
    } else if (row < cut.x) {
        if constexpr (kChunks == 2) *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    }
    if (p.lse && row < cut.x && chunk == 0) p.lse[static_cast<size_t>(cut.y) + row] = (m + log2f(l)) * 0.69314718055994531f;
}

// Merges the records of the tiles that runs' ends cut. What counts is that enough loads are on their way: a warp has
// 16 of 16 bytes a lane, of as many dims as that is for the tile's pieces.
__global__ void __launch_bounds__(kLatMergeThreads, 2) latent_merge_kernel(const __grid_constant__ LatentAttnParams p) {
    constexpr int kWarps = kLatMergeThreads / 32;
    __shared__ int4 cuts[kLatMergeThreads];
    __shared__ int before[kLatMergeThreads + 1], sums[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_dependents_launch();
    // every block lists the tasks: a run's tile, by rows and dims
    auto chunks_of = [](int pieces) { return pieces <= 2 ? 8 : pieces <= 4 ? 4 : pieces <= 8 ? 2 : 1; };
    int4 cut = make_int4(0, 0, 0, 0);  // rows, the first one's place, the tile's last run
    if (tid < p.runs) cut = __ldcg(p.cuts + tid);
    int scan = (cut.x + 31) / 32 * (kLatC / 4 / chunks_of(cut.z - tid + 1));
    CFA_ROLLED for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    cuts[tid] = cut;
    __syncthreads();
    CFA_ROLLED for (int w = 0; w < warp; ++w) scan += sums[w];
    before[tid + 1] = scan;
    if (tid == 0) before[0] = 0;
    __syncthreads();
    const int all = before[kLatMergeThreads];
    CFA_ROLLED for (int task = static_cast<int>(blockIdx.x) * kWarps + warp; task < all; task += static_cast<int>(gridDim.x) * kWarps) {
        int lo = 0, hi = kLatMergeThreads;  // the last run whose tasks begin no later
        CFA_ROLLED while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before[mid] <= task) lo = mid;
            else hi = mid;
        }
        cut = cuts[lo];
        const int groups = (cut.x + 31) / 32, at = task - before[lo], row = at % groups * 32;
        const int chunks = chunks_of(cut.z - lo + 1), chunk = at / groups * chunks;
        if (chunks == 8) latent_merge_rows<8, 2>(p, cut, lo, row, chunk);
        else if (chunks == 4) latent_merge_rows<4, 4>(p, cut, lo, row, chunk);
        else if (chunks == 2) latent_merge_rows<2, 8>(p, cut, lo, row, chunk);
        else latent_merge_rows<1, 16>(p, cut, lo, row, chunk);
    }
}

}  // namespace cfa
