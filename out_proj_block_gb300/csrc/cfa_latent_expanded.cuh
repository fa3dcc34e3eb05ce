// cfa_latent_expanded.cuh -- attention of prompts over expanded keys and values.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  m = max_j s_j,
//   s_j = scale log2(e) (q_nope . k_j + q_rope . k_rope_j);  lse = (m + log2 sum_j w_j) ln 2
//
// for each query token and head over the keys that the token sees. A row without any is 0 with lse -inf.
//
// A task is a head of a request and 512 of its tokens; 192 dims of scores and 128 of values are 640
// operations a query and key, so products bound it. A cluster of two blocks takes a task as two tiles of
// 256 rows (128 to either block) with the tcgen05 instructions that span both: a block of 128 keys is S = Q K^T
// (12 instructions of 256 x 128 x 16) and O += P V (8) for either tile, and either block holds half of it, 64 keys
// for the scores and 64 dims for the values. In one block's own instructions (128 x 128 x 16) the
// scores' two operands kept shared memory busy for 92 clocks each, where the arithmetic takes 64, and left room
// for little more than one block of keys. TMEM holds S and O of both tiles (4 x 128 columns), the weights P as
// bf16 in place of the scores. A tile's next scores need its weights' product to have ended, so while one tile's
// softmax runs (a thread a row), the other's products do: the tiles take turns. The last commit that a
// tile's scores wait for covers the product before them, so O may be rescaled then; that is done lazily, when a
// row's maximum grew by more than 8 (a factor 2^8, far inside fp32), a published method.
//
// Tasks are dealt out in turn to one cluster per pair of SMs, those of most keys first and each round in
// the other direction; in the order of requests instead, five prompts of 763 to 1500 tokens took the last cluster
// 20% longer than the mean. What does not fill the last round is split along the keys; its parts leave records,
// which a second kernel merges in order, so results are bitwise reproducible.
//
// Measured, with the merge (one GB300): 1024 tokens behind 2500 keys, 128 heads: 192 us (1.32 PFLOP/s); five
// prompts of up to 1500 tokens, 32 heads: 114 us (0.65). A block of keys takes 2950 clocks of 512 rows, of
// which products are 2560; a task's begin and end 7000, its last blocks, which one tile alone sees or
// whose keys are masked, 5000 each. Tiles that go through the tasks each by itself, so that one's last
// blocks run beside the other's next task, took more in the middle (3200 to 3500 clocks a block) than they saved.
//
// Weights are rounded to bf16 for their product with the values (2^-8 each, the size of the result's own
// rounding); their sum, the maxima, the outputs and the records are fp32.
#pragma once

#include <cuda.h>

#include "cfa_device.cuh"
#include "cfa_latent.h"
#include "cfa_paged.h"
#include "cfa_paged_device.cuh"
#include "cfa_tensor.cuh"
#include "cfa_tensor_pair.cuh"
#include "cfa_tile.cuh"

namespace cfa {

constexpr int kExpChunk = 128 * 128;   // 128 rows of 64 dims
constexpr int kExpSlots = 3;           // blocks of keys and of values in flight
constexpr int kExpKSlot = 3 * 64 * 128, kExpVSlot = 128 * 128;
constexpr int kExpPeek = 3;            // blocks before an item's end that the next one's queries are asked for in L2
constexpr int kExpTile = 256;          // tokens of a tile, half of them to either block
constexpr int kExpRows = 2 * kExpTile; // tokens of a task

// Shared memory, the same in both blocks of a cluster.
struct ExpSmem {
    static constexpr int kQ = 0;                              // [2 tiles][3][128 rows][128 bytes]
    static constexpr int kK = kQ + 6 * kExpChunk;             // ring of [3][64 keys][128 bytes]
    static constexpr int kV = kK + kExpSlots * kExpKSlot;     // ring of [128 keys][128 bytes]
    static constexpr int kBars = kV + kExpSlots * kExpVSlot;
    static constexpr int kFullK = kBars, kEmptyK = kFullK + 8 * kExpSlots, kReadyK = kEmptyK + 8 * kExpSlots;
    static constexpr int kFullV = kReadyK + 8 * kExpSlots, kEmptyV = kFullV + 8 * kExpSlots, kReadyV = kEmptyV + 8 * kExpSlots;
    static constexpr int kFullQ = kReadyV + 8 * kExpSlots, kEmptyQ = kFullQ + 16, kReadyQ = kEmptyQ + 16;  // a tile each
    static constexpr int kScores = kReadyQ + 16, kWeights = kScores + 16, kDrain = kWeights + 16;
    static constexpr int kBarsEnd = kDrain + 8;
    static constexpr int kMisc = kBarsEnd;                    // flags, TMEM address
    static constexpr int kSums = kMisc + 16;                  // int [12]: the scan's sums
    static constexpr int kTasks = kSums + 64;                 // int [kExpMaxTasks]: a head's tasks, the dearest first
    static constexpr int kBytes = kTasks + 4 * (kPagedMaxTokens / kExpRows + kPagedMaxSeqs);
};
static_assert(ExpSmem::kBytes <= 227 * 1024, "it fits");
// Tasks of a head at most, and how the list names one.
constexpr int kExpMaxTasks = kPagedMaxTokens / kExpRows + kPagedMaxSeqs;
constexpr int kExpTaskBits = 12;
static_assert(kPagedMaxTokens / kExpRows < 1 << kExpTaskBits, "a request's task fits its bits");

// Tasks and how they are dealt out to `grid` clusters, from what a scan over the requests finds.
struct ExpPlan {
    int full;   // rounds in which every cluster has a task
    int rest;   // tasks behind them
    int parts;  // that each of those is split into at most
};
CFA_HD ExpPlan latent_expanded_plan(int tasks, int grid) {
    ExpPlan p;
    p.full = tasks / grid;
    p.rest = tasks - p.full * grid;
    p.parts = p.rest > 0 ? paged_min(kExpMaxParts, grid / p.rest) : 1;
    return p;
}

// A task's part.
struct ExpItem {
    int req, h, tile;          // request, head, which 512 of its tokens
    int tok0, n, k0, len;      // the request's tokens and keys
    int part, parts;           // which of how many parts of its blocks
    int b0, end0, end1;        // first block of keys, and behind the last one that each tile sees
    int rec;                   // its record's number
    __device__ __forceinline__ int end(int t) const { return t ? end1 : end0; }
    __device__ __forceinline__ int last() const { return max(end0, end1); }
    __device__ __forceinline__ int rows(int t) const { return max(0, min(kExpTile, n - tile * kExpRows - kExpTile * t)); }
    // keys that token i of the request sees
    __device__ __forceinline__ int visible(int i) const { return max(0, min(len, len - n + i + 1)); }
};

// Lists a head's tasks in smem, (request << 12 | which 512 tokens), those of most blocks first: dealt out in turn
// and back, they come out even, and what is left for the last round is cheap. The number of all
// heads', or -1 where the offsets are not in order. `work` holds 8 kExpMaxTasks bytes. By all threads of the block.
template <int kThreads>
__device__ __forceinline__ int latent_expanded_list(const LatentExpandedParams &p, int *list, int2 *work, int *sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads, first = tid * per, last = min(p.B, first + per);
    int mine = 0;
    bool bad = false;
    CFA_ROLLED for (int b = first; b < last; ++b) {
        const int a = __ldcg(p.cu + b), e = __ldcg(p.cu + b + 1), ka = __ldcg(p.cu_k + b), ke = __ldcg(p.cu_k + b + 1);
        if (a < 0 || e < a || e > p.T || ka < 0 || ke < ka || ke > p.S) bad = true;
        else mine += (e - a + kExpRows - 1) / kExpRows;
    }
    int scan = mine;
    CFA_ROLLED for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    const bool refused = __syncthreads_or(bad) != 0;
    int at = scan - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += sums[w];
        all += sums[w];
    }
    if (refused) return -1;
    CFA_ROLLED for (int b = first; b < last; ++b) {
        const int tok0 = __ldcg(p.cu + b), n = __ldcg(p.cu + b + 1) - tok0;
        const int len = __ldcg(p.cu_k + b + 1) - __ldcg(p.cu_k + b);
        CFA_ROLLED for (int i = 0; i * kExpRows < n; ++i)  // (named by its keys: half of them more or less is no matter)
            work[at++] = make_int2(min(len, max(0, len - n + (i + 1) * kExpRows)), b << kExpTaskBits | i);
    }
    __syncthreads();
    CFA_ROLLED for (int i = tid; i < all; i += kThreads) {
        const int2 x = work[i];
        int rank = 0;
        CFA_ROLLED for (int j = 0; j < all; ++j) rank += work[j].x > x.x || (work[j].x == x.x && j < i);
        list[rank] = x.y;
    }
    __syncthreads();
    return all * p.H;
}

// Task number `task`, part `part` of at most `parts`; false where it has fewer.
__device__ __forceinline__ bool latent_expanded_item(const LatentExpandedParams &p, const int *list, int task, int part,
                                                     int parts, ExpItem &x) {
    const int at = task / p.by_H, lo = list[at] >> kExpTaskBits;
    x.req = lo;
    x.h = task - at * p.H;
    x.tile = list[at] & ((1 << kExpTaskBits) - 1);
    x.tok0 = __ldcg(p.cu + lo);
    x.n = __ldcg(p.cu + lo + 1) - x.tok0;
    x.k0 = __ldcg(p.cu_k + lo);
    x.len = __ldcg(p.cu_k + lo + 1) - x.k0;
    auto blocks_of = [&](int t) {
        const int rows = x.rows(t);
        return rows > 0 ? (x.visible(x.tile * kExpRows + kExpTile * t + rows - 1) + 127) / 128 : 0;
    };
    const int e0 = blocks_of(0), e1 = blocks_of(1), blocks = max(e0, e1);
    x.part = part;
    x.parts = max(1, min(parts, blocks / kExpLeast));
    if (part >= x.parts) return false;
    x.b0 = blocks * part / x.parts;
    const int b1 = blocks * (part + 1) / x.parts;
    x.end0 = max(x.b0, min(b1, e0));
    x.end1 = max(x.b0, min(b1, e1));
    return true;
}

__device__ __forceinline__ void registers_of_softmax() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;"); }
__device__ __forceinline__ void registers_of_loads() { asm volatile("setmaxnreg.dec.sync.aligned.u32 88;"); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpThreads, 1)
latent_expanded_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                       const __grid_constant__ CUtensorMap tm_rope, const __grid_constant__ LatentExpandedParams p) {
    using S = ExpSmem;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    const int rank = static_cast<int>(cluster_ctarank()), cluster = static_cast<int>(blockIdx.x) >> 1;
    int *misc = reinterpret_cast<int *>(smem + S::kMisc);
    volatile int *timed_out = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);
    int *list = reinterpret_cast<int *>(smem + S::kTasks);

    // a thread a barrier, with the arrivals it expects
    if (tid < (S::kBarsEnd - S::kBars) / 8) {
        const int at = S::kBars + 8 * tid;
        uint32_t count = 1;
        if ((at >= S::kReadyK && at < S::kFullV) || (at >= S::kReadyV && at < S::kFullQ) || (at >= S::kReadyQ && at < S::kScores))
            count = 2;  // the relays of both blocks
        if (at >= S::kEmptyQ && at < S::kReadyQ) count = 4;   // a tile's warps
        if (at >= S::kWeights && at < S::kDrain) count = 8;   // and those of both blocks
        mbar_init(base + at, count);
        fence_mbar_init();
    }
    if (tid == 0) misc[0] = 0;
    if (warp == kExpMmaWarp) tmem2_alloc(smem_addr(tmem_slot), 512);
    if (warp == kExpLoadWarp && elect_one()) {
        prefetch_tensor_map(&tm_q);
        prefetch_tensor_map(&tm_kv);
        prefetch_tensor_map(&tm_rope);
    }
    __syncwarp();
    tcgen05_fence_before();
    cluster_arrive();  // (the other block's barriers are ready behind the wait below)
    grid_dependency_wait();
    const int tasks = latent_expanded_list<kExpThreads>(p, list, reinterpret_cast<int2 *>(smem + S::kQ),  // (free yet)
                                                        reinterpret_cast<int *>(smem + S::kSums));
    tcgen05_fence_after();
    if (blockIdx.x == 0 && tid == 0 && tasks < 0) atomicOr(p.status, kStatusBadLengthBit);
    grid_dependents_launch();
    fence_proxy_async_smem();  // (the queries go where the list was made)
    __syncthreads();
    cluster_wait();
    const uint32_t tmem = *tmem_slot;
    const int grid = static_cast<int>(gridDim.x) >> 1;
    const ExpPlan plan = latent_expanded_plan(max(0, tasks), grid);
    if (blockIdx.x == 0 && tid == 0) *p.rest = plan.parts > 1 ? plan.rest : 0;
    // The cluster's item of round r; false where it has none.
    auto item = [&](int r, ExpItem &x) {
        const int at = r & 1 ? grid - 1 - cluster : cluster;
        if (r < plan.full) return latent_expanded_item(p, list, r * grid + at, 0, 1, x);
        const int task = at / plan.parts, part = at - task * plan.parts;
        x.rec = at;
        return task < plan.rest && latent_expanded_item(p, list, plan.full * grid + task, part, plan.parts, x);
    };
    const int rounds = plan.full + (plan.rest > 0);
    // The first item from round r on, r becomes the round behind it; false at the end.
    auto next = [&](int &r, ExpItem &x) {
        CFA_ROLLED while (r < rounds)
            if (item(r++, x)) return true;
        return false;
    };
    auto wait = [&](int bar, uint32_t parity, unsigned site) {
        return bounded_wait([&]() { return mbar_try_wait(base + bar, parity); }, p.timeout_ns, timed_out, p.status, site);
    };
    // The same for a warp as a whole.
    auto wait_warp = [&](int bar, uint32_t parity, unsigned site) { return __all_sync(~0u, wait(bar, parity, site)); };

    if (warp >= kExpLoadWarp) {
        registers_of_loads();
        if (warp == kExpLoadWarp || warp == kExpLoadWarp + 1) {
            // -------------------------------------- load warps: keys and queries, values
            const bool values = warp != kExpLoadWarp;
            uint32_t n = 0, queried = 0, queries = 0;  // blocks; tiles whose queries were ever loaded, and phases, a bit a tile
            bool ok = true;
            int r = 0;
            ExpItem x, ahead;
            bool have = next(r, x);
            for (; ok && have; x = ahead) {
                const int last = x.last();
                have = next(r, ahead);
                CFA_ROLLED for (int b = x.b0; ok && b < last; ++b, ++n) {
                    const uint32_t slot = n % kExpSlots, again = n / kExpSlots;
                    const int full = (values ? S::kFullV : S::kFullK) + 8 * slot;
                    if (again > 0) ok = wait_warp((values ? S::kEmptyV : S::kEmptyK) + 8 * slot, (again - 1) & 1, kSiteStageEmpty);
                    if (!ok) break;
                    if (elect_one()) {
                        if (!values) {  // 64 of the keys
                            const uint32_t dst = base + S::kK + slot * kExpKSlot;
                            const int y = x.k0 + 128 * b + 64 * rank;
                            mbar_arrive_expect_tx(base + full, kExpKSlot);
                            tma_load_2d(dst, &tm_kv, x.h * kLatKv, y, base + full);
                            tma_load_2d(dst + 64 * 128, &tm_kv, x.h * kLatKv + 64, y, base + full);
                            tma_load_2d(dst + 2 * 64 * 128, &tm_rope, 0, y, base + full);
                        } else {        // 64 of the dims
                            const uint32_t dst = base + S::kV + slot * kExpVSlot;
                            const int dim = x.h * kLatKv + kLatN + 64 * rank, y = x.k0 + 128 * b;
                            mbar_arrive_expect_tx(base + full, kExpVSlot);
                            tma_load_2d(dst, &tm_kv, dim, y, base + full);
                            tma_load_2d(dst + 64 * 128, &tm_kv, dim, y + 64, base + full);
                            if (have && b == max(x.b0, last - kExpPeek)) {
                                // the next item's queries, in L2 by the time they are loaded
#pragma unroll 1
                                for (int i = 0; i < 6; ++i)
                                    if (ahead.end(i / 3) > ahead.b0)
                                        tma_prefetch_2d(&tm_q, ahead.h * kLatQ + 64 * (i % 3),
                                                        ahead.tok0 + ahead.tile * kExpRows + kExpTile * (i / 3) + 128 * rank);
                            }
                        }
                    }
                    __syncwarp();
                    if (values || b > x.b0) continue;
                    // the queries behind the first keys, which find room earlier
                    CFA_ROLLED for (int t = 0; ok && t < 2; ++t) {
                        if (x.end(t) == x.b0) continue;
                        if (queried >> t & 1) ok = wait_warp(S::kEmptyQ + 8 * t, ~queries >> t & 1, kSiteStageEmpty);
                        if (!ok) break;
                        if (elect_one()) {
                            const uint32_t full_q = base + S::kFullQ + 8 * t;
                            mbar_arrive_expect_tx(full_q, 3 * kExpChunk);
#pragma unroll
                            for (int c = 0; c < 3; ++c)
                                tma_load_2d(base + S::kQ + (3 * t + c) * kExpChunk, &tm_q, x.h * kLatQ + 64 * c,
                                            x.tok0 + x.tile * kExpRows + kExpTile * t + 128 * rank, full_q);
                        }
                        __syncwarp();
                        queried |= 1u << t;
                        queries ^= 1u << t;
                    }
                }
            }
            if (lane == 0 && *timed_out) {
                // a wait gave up: the copies in flight land before the block ends
                const uint64_t t0 = global_timer_ns();
                auto land = [&](uint32_t bar, uint32_t parity) {
                    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                    }
                };
                for (uint32_t k = n > kExpSlots ? n - kExpSlots : 0; k < n; ++k)
                    land(base + (values ? S::kFullV : S::kFullK) + 8 * (k % kExpSlots), (k / kExpSlots) & 1);
                for (int t = 0; !values && t < 2; ++t)
                    if (queried >> t & 1) land(base + S::kFullQ + 8 * t, ~queries >> t & 1);
            }
            __syncwarp();
        } else if (warp == kExpRelayWarp) {
            // ----------------------------------------------------------------- relay warp
            // tells the issuing block what has landed, in the order in which the products take it: keys of a
            // block ahead, values
            uint32_t nk = 0, nv = 0, queries = 0;
            const uint32_t ready_k = map_to_rank(base + S::kReadyK, 0), ready_v = map_to_rank(base + S::kReadyV, 0),
                           ready_q = map_to_rank(base + S::kReadyQ, 0);
            bool ok = true;
            auto pass_on = [&](int full, uint32_t ready, uint32_t parity) {
                ok = ok && wait_warp(full, parity, kSiteStageFull);
                if (ok && elect_one()) mbar_arrive_pair(ready);
                __syncwarp();
            };
            auto keys = [&]() {
                pass_on(S::kFullK + 8 * (nk % kExpSlots), ready_k + 8 * (nk % kExpSlots), (nk / kExpSlots) & 1);
                ++nk;
            };
            int r = 0;
            ExpItem x;
            while (ok && next(r, x)) {
                if (x.last() == x.b0) continue;
                // keys that every row of a tile sees, and that any row of the task does
                const int some0 = x.visible(x.tile * kExpRows), some1 = x.visible(x.tile * kExpRows + kExpTile);
                const int all = x.visible(min(x.n, x.tile * kExpRows + kExpRows) - 1);
                keys();
                CFA_ROLLED for (int t = 0; t < 2; ++t) {
                    if (x.end(t) == x.b0) continue;
                    pass_on(S::kFullQ + 8 * t, ready_q + 8 * t, queries >> t & 1);
                    queries ^= 1u << t;
                }
                CFA_ROLLED for (int b = x.b0; ok && b < x.last(); ++b, ++nv) {
                    if (b + 1 < x.last()) keys();
                    const uint32_t slot = nv % kExpSlots;
                    ok = ok && wait_warp(S::kFullV + 8 * slot, (nv / kExpSlots) & 1, kSiteStageFull);
                    const int begin = (b < x.end0 ? some0 : some1) - 128 * b, end = all - 128 * b;
                    if (ok && begin < 128) {
                        // Keys from `begin` on are not seen by every row, from `end` on by none. A masked weight is 0, and 0
                        // times NaN is NaN: what is not finite of the first becomes 0, and the merge adds it to the rows that
                        // see it; the others become 0. (A lane 16 bytes of every fourth row; of a row's chunks any order will do.)
                        uint8_t *v = smem + S::kV + slot * kExpVSlot + (lane >> 3) * 128 + ((lane & 7) << 4);
                        CFA_ROLLED for (int k0 = max(0, begin) & ~31; k0 < 128; k0 += 32) {
                            uint4 d[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) d[i] = *reinterpret_cast<const uint4 *>(v + k0 * 128 + i * 512);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int k = k0 + 4 * i + (lane >> 3);
                                // an exponent of ones and the 1 added to it carry into the sign's place
                                auto carry = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
                                const uint32_t odd = (carry(d[i].x) | carry(d[i].y) | carry(d[i].z) | carry(d[i].w)) & 0x80008000u;
                                if (k < begin || (k < end && odd == 0u)) continue;
                                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                                if (k < end) {
                                    *p.odd = 1u;
                                    w = make_uint4(d[i].x & ~odd_bf16x2(d[i].x), d[i].y & ~odd_bf16x2(d[i].y),
                                                   d[i].z & ~odd_bf16x2(d[i].z), d[i].w & ~odd_bf16x2(d[i].w));
                                }
                                *reinterpret_cast<uint4 *>(v + k0 * 128 + i * 512) = w;
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (ok && elect_one()) mbar_arrive_pair(ready_v + 8 * slot);
                    __syncwarp();
                }
            }
        } else if (warp == kExpMmaWarp && rank == 0) {
            // -------------------------------------------------- products, by the first block
            const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
            const uint32_t idesc_s = umma_idesc_bf16(256, 128, false, false), idesc_o = umma_idesc_bf16(256, 128, false, true);
            const uint64_t q0 = umma_smem_desc(base + S::kQ, 16, 1024), k0 = umma_smem_desc(base + S::kK, 16, 1024),
                           v0 = umma_smem_desc(base + S::kV, kExpVSlot, 1024);
            uint32_t n = 0, queries = 0, weights = 0;  // blocks before the item's; phases, a bit a tile
            bool ok = true;
            int r = 0;
            ExpItem x, ahead;
            bool have = next(r, x);
            for (; ok && have; x = ahead) {
                const int last = x.last(), b0 = x.b0;
                // By one thread: scores of tile t and block b. `frees`: nobody reads the keys after.
                auto scores = [&](int t, int b, bool frees) {
                    const uint32_t slot = (n + b - b0) % kExpSlots;
                    const uint64_t a = q0 + 3 * t * (kExpChunk >> 4), bd = k0 + slot * (kExpKSlot >> 4);
#pragma unroll
                    for (int ks = 0; ks < 12; ++ks)  // 32 bytes a step
                        umma2_bf16(tm + 128 * t, a + (ks >> 2) * (kExpChunk >> 4) + 2 * (ks & 3),
                                   bd + (ks >> 2) * (64 * 128 >> 4) + 2 * (ks & 3), idesc_s, ks > 0);
                    if (frees) umma2_commit(base + S::kEmptyK + 8 * slot);
                    umma2_commit(base + S::kScores + 8 * t);
                };
                auto keys = [&](int b) {
                    const uint32_t k = n + b - b0;
                    ok = ok && wait_warp(S::kReadyK + 8 * (k % kExpSlots), (k / kExpSlots) & 1, kSiteStageFull);
                };
                if (last > b0) keys(b0);
                CFA_ROLLED for (int t = 0; ok && t < 2; ++t) {
                    if (x.end(t) == b0) continue;
                    ok = wait_warp(S::kReadyQ + 8 * t, queries >> t & 1, kSiteQExchange);
                    queries ^= 1u << t;
                    tcgen05_fence_after();
                    if (ok && elect_one()) scores(t, b0, t == 1 || x.end1 == b0);
                    __syncwarp();
                }
                have = next(r, ahead);  // (beside the first softmax)
                CFA_ROLLED for (int b = b0; ok && b < last; ++b) {
                    const uint32_t slot = (n + b - b0) % kExpSlots;
                    if (b + 1 < last) keys(b + 1);
                    ok = ok && wait_warp(S::kReadyV + 8 * slot, ((n + b - b0) / kExpSlots) & 1, kSiteStageFull);
                    CFA_ROLLED for (int t = 0; ok && t < 2; ++t) {
                        if (b >= x.end(t)) continue;
                        ok = wait_warp(S::kWeights + 8 * t, weights >> t & 1, kSiteSoftmaxExchange);
                        weights ^= 1u << t;
                        tcgen05_fence_after();
                        // the product and the next scores in one go: between two goes the tensor core runs dry for some 400 clocks
                        if (ok && elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)  // 16 keys of 128 bytes a step
                                umma2_bf16_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * ks, v0 + slot * (kExpVSlot >> 4) + 128 * ks,
                                              idesc_o, b > b0 || ks > 0);
                            if (t == 1 || b >= x.end1) umma2_commit(base + S::kEmptyV + 8 * slot);
                            // behind the last product there are no more scores, but the tile's warps learn that it ended
                            if (b + 1 < x.end(t)) scores(t, b + 1, t == 1 || b + 1 >= x.end1);
                            else umma2_commit(base + S::kScores + 8 * t);
                        }
                        __syncwarp();
                    }
                }
                n += last - b0;
            }
            if (elect_one() && *timed_out) {
                // a wait gave up: the products in flight end before the blocks do
                umma2_commit(base + S::kDrain);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(base + S::kDrain, 0) && global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------- softmax warps, a warpgroup a tile
        registers_of_softmax();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lanes of this warp
        const uint32_t t_s = tmem + lanes + 128 * t, t_o = tmem + lanes + 256 + 128 * t;
        const int scores = S::kScores + 8 * t;
        const uint32_t weights = map_to_rank(base + S::kWeights, 0) + 8 * t;
        uint32_t scored = 0;  // phases
        int r = 0;
        ExpItem x, ahead;
        bool have = next(r, x);
        for (; have; x = ahead) {
            // of a split task, for the merge: where its rows are and how many parts it has
            if (r > plan.full && plan.parts > 1 && x.part == 0 && rank == 0 && tid == 0)
                p.splits[x.rec / plan.parts] = make_int4((x.tok0 + x.tile * kExpRows) * p.H + x.h, min(kExpRows, x.n - x.tile * kExpRows),
                                                         x.parts, x.rec);
            const int first = x.tile * kExpRows + kExpTile * t + 128 * rank;  // this block's first token of the tile
            const int rows = max(0, min(128, x.rows(t) - 128 * rank));
            const bool live = row < rows, warp_live = row - lane < rows;
            // (rows past the last see what that one sees, so that their warp takes no masked blocks for them: they took 20%
            // of the time of a prompt that ends inside a warp's rows)
            const int see = x.visible(first + min(row, max(rows, 1) - 1));
            float m = -INFINITY, l = 0.f;
            CFA_ROLLED for (int b = x.b0; b < x.end(t); ++b, ++scored) {
                wait(scores, scored & 1, kSiteSoftmaxExchange);
                __syncwarp();
                tcgen05_fence_after();
                if (warp_live) {
                    uint32_t s[128];
#pragma unroll
                    for (int c = 0; c < 128; c += 32) tmem_ld_x32(t_s + c, s + c);
                    tmem_wait_ld();
                    const int lim = see - 128 * b;
                    if (!__all_sync(~0u, lim >= 128)) {
                        const int least = __reduce_min_sync(~0u, lim);
#pragma unroll
                        for (int g = 0; g < 128; g += 32)
                            if (least < g + 32) {
#pragma unroll
                                for (int c = g; c < g + 32; ++c) s[c] = c < lim ? s[c] : 0xff800000u;
                            }
                    }
                    float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 2)
                        a[(c >> 1) & 3] = fmaxf(fmaxf(a[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                    const float top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * p.scale_log2;
                    if (__any_sync(~0u, top > m + 8.f)) {
                        // rescale to the new maximum (m = -inf: nothing is there yet)
                        const float mn = top > m + 8.f ? top : m;  // (each row by itself: others must not change it)
                        const float g = m == mn ? 1.f : exp2_ftz(m - mn);
                        m = mn;
                        l *= g;
                        if (b > x.b0) {
#pragma unroll 1
                            for (int c = 0; c < kLatV; c += 32) {
                                uint32_t v[32];
                                tmem_ld_x32(t_o + c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * g);
                                tmem_st_x16(t_o + c, v);
                                tmem_st_x16(t_o + c + 16, v + 16);
                            }
                        }
                    }
                    const float f = m == -INFINITY ? 0.f : -m;
                    const uint64_t scale2 = pair_f32(p.scale_log2, p.scale_log2), f2 = pair_f32(f, f);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = unpair_f32(fma_f32x2(
                                pair_f32(__uint_as_float(s[32 * c + 2 * e]), __uint_as_float(s[32 * c + 2 * e + 1])), scale2, f2));
                            const float x0 = exp2_ftz(y.x), x1 = exp2_ftz(y.y);
                            sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(x0, x1));
                            w[e] = pack2_bf16_cvt(x0, x1);
                        }
                        tmem_st_x16(t_s + 16 * c, w);
                    }
                    const float2 both = unpair_f32(add_f32x2(sum[0], sum[1]));
                    l += both.x + both.y;
                    tmem_wait_st();
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(weights);
            }
            const bool any = x.end(t) > x.b0;
            have = next(r, ahead);  // (its loads are on their way meanwhile)
            if (any) {
                wait(scores, scored & 1, kSiteKvExchange);
                ++scored;
            }
            __syncwarp();
            tcgen05_fence_after();
            // ---- the tile's results, or its record
            if (warp_live) {
                const int in_task = kExpTile * t + 128 * rank + row;
                const size_t tok = static_cast<size_t>(x.tok0 + first + row);
                if (x.parts > 1) {
                    if (live) p.rec_ml[x.rec * kExpRows + in_task] = make_float2(m, l);
                    float *rec_o = p.rec_o + static_cast<size_t>(x.rec) * kExpRows * kLatV + 4 * in_task;
#pragma unroll 1
                    for (int c = 0; any && c < kLatV; c += 32) {  // (without keys: m says that nothing is there)
                        uint32_t v[32];
                        __syncwarp();
                        tmem_ld_x32(t_o + c, v);
                        tmem_wait_ld();
                        if (!live) continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<uint4 *>(rec_o + static_cast<size_t>(c / 4 + e) * (4 * kExpRows)) =
                                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                } else {
                    if (p.lse && live) p.lse[tok * p.H + x.h] = (m + log2f(l)) * 0.69314718055994531f;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    // through the tile's first chunk of queries, which nobody reads any more, so that a row's 128 bytes
                    // are written together
                    uint8_t *stage = smem + S::kQ + 3 * t * kExpChunk + (row - lane) * 128;
#pragma unroll 1
                    for (int c = 0; c < kLatV; c += 64) {
                        __syncwarp();
                        uint4 y[8];
                        if (any) {
                            uint32_t v[64];
                            tmem_ld_x32(t_o + c, v);
                            tmem_ld_x32(t_o + c + 32, v + 32);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = pack2_bf16_cvt(__uint_as_float(v[8 * e + 2 * k]) * inv, __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
                                *reinterpret_cast<uint4 *>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int k = 4 * e + (lane >> 3);
                                y[e] = *reinterpret_cast<const uint4 *>(stage + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
                            }
                        } else {  // (without keys the tile has no queries: the next item's may be landing there)
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = make_uint4(0u, 0u, 0u, 0u);
                        }
                        uint16_t *out = p.out + ((tok - lane) * p.H + x.h) * kLatV + c + 8 * (lane & 7);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int k = 4 * e + (lane >> 3);
                            if (row - lane + k < rows) *reinterpret_cast<uint4 *>(out + static_cast<size_t>(k) * p.H * kLatV) = y[e];
                        }
                    }
                    fence_proxy_async_smem();  // (the next queries come by the asynchronous proxy)
                }
            }
            tcgen05_fence_before();
            __syncwarp();
            if (any && lane == 0) mbar_arrive(base + S::kEmptyQ + 8 * t);
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    cluster_sync_all();  // nothing of either block reaches into the other any more
    if (warp == kExpMmaWarp) {
        tcgen05_fence_after();
        tmem2_dealloc(tmem, 512);
    }
}

// Adds the values that are not finite to the rows that see them, where the attention has met one that some rows
// see and others do not (rows that have them already do not change). The last block does it, when
// all rows are written: a thread goes through a request's new tokens with 8 dims of a head and holds what they
// have seen so far. Rare, so it need only end in time: a load a token.
__device__ __noinline__ void latent_expanded_add_odd(const LatentExpandedParams &p) {
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomic_add_acq_rel_gpu(p.odd + 1, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    if (threadIdx.x < 2) p.odd[threadIdx.x] = 0;
    constexpr int C = kLatV / 8;
    for (int task = threadIdx.x; task < p.B * p.H * C; task += kLatMergeThreads) {
        const int c = task % C, b = task / C / p.H, h = task / C - b * p.H;
        const int tok0 = p.cu[b], n = p.cu[b + 1] - tok0, k0 = p.cu_k[b], len = p.cu_k[b + 1] - k0;
        bool some = false;
        float seen[8] = {};
        // token i is the first that sees key len - n + i (the first token's keys all see)
        for (int i = max(1, n - len); i < n; ++i) {
            float v[8];
            unpack8_bf16(*reinterpret_cast<const uint4 *>(p.kv + (k0 + len - n + i) * p.kv_stride + h * kLatKv + kLatN + 8 * c), v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!(fabsf(v[e]) < INFINITY)) seen[e] += v[e], some = true;
            if (!some) continue;
            uint4 *at = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(tok0 + i) * p.H + h) * kLatV + 8 * c);
            float y[8];
            unpack8_bf16(*at, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = seen[e] == 0.f ? y[e] : y[e] + seen[e];
            *at = make_uint4(pack2_bf16_cvt(y[0], y[1]), pack2_bf16_cvt(y[2], y[3]), pack2_bf16_cvt(y[4], y[5]), pack2_bf16_cvt(y[6], y[7]));
        }
    }
}

// Merges the records of the split tasks, a warp for 32 rows (a lane a row) and 16 dims.
__global__ void __launch_bounds__(kLatMergeThreads, 3) latent_expanded_merge_kernel(const __grid_constant__ LatentExpandedParams p) {
    grid_dependency_wait();
    const unsigned odd = __ldcg(p.odd);
    const int rest = __ldcg(p.rest);
    const int lane = threadIdx.x & 31, warps = static_cast<int>(gridDim.x) * (kLatMergeThreads / 32);
    constexpr int kRec = kExpRows * (kLatV / 4);
    CFA_ROLLED for (int i = static_cast<int>(blockIdx.x) * (kLatMergeThreads / 32) + (threadIdx.x >> 5); i < rest * 128; i += warps) {
        const int4 x = __ldcg(p.splits + (i >> 7));  // the first row's place, rows, parts, the first record
        const int row = (i & 15) * 32 + lane, chunk = (i >> 4 & 7) * 4, parts = x.z;
        if (parts == 1 || row >= x.y) continue;
        const float2 *ml = p.rec_ml + x.w * kExpRows + row;
        const float4 *o = reinterpret_cast<const float4 *>(p.rec_o) + static_cast<size_t>(x.w) * kRec + chunk * kExpRows + row;
        float m = -INFINITY, l = 0.f;
        float2 s[kExpMaxParts];
#pragma unroll
        for (int k = 0; k < kExpMaxParts; ++k) {
            s[k] = k < parts ? __ldcg(ml + k * kExpRows) : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, s[k].x);
        }
        const float f = m == -INFINITY ? 0.f : m;
        float a[16] = {};
#pragma unroll
        for (int k = 0; k < kExpMaxParts; ++k) {
            if (k >= parts) break;
            const float g = exp2_ftz(s[k].x - f);
            l += g * s[k].y;
            if (s[k].x == -INFINITY && s[k].y == 0.f) continue;  // no keys: there may be no outputs
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 v = __ldcg(o + static_cast<size_t>(k) * kRec + c * kExpRows);
                a[4 * c] += g * v.x; a[4 * c + 1] += g * v.y; a[4 * c + 2] += g * v.z; a[4 * c + 3] += g * v.w;
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = static_cast<size_t>(x.x) + static_cast<size_t>(row) * p.H;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4 *>(p.out + at * kLatV + 4 * chunk + 8 * c) =
                make_uint4(pack2_bf16_cvt(a[8 * c] * inv, a[8 * c + 1] * inv), pack2_bf16_cvt(a[8 * c + 2] * inv, a[8 * c + 3] * inv),
                           pack2_bf16_cvt(a[8 * c + 4] * inv, a[8 * c + 5] * inv), pack2_bf16_cvt(a[8 * c + 6] * inv, a[8 * c + 7] * inv));
        if (p.lse && chunk == 0) p.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
    }
    if (odd) latent_expanded_add_odd(p);
    grid_dependents_launch();
}

}  // namespace cfa
