// cfa_latent_expanded.cuh -- attention of prompts over expanded keys and values.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  m = max_j s_j,
//   s_j = scale log2(e) (q_nope . k_j + q_rope . k_rope_j);  lse = (m + log2 sum_j w_j) ln 2
//
// for each query token and head over the keys that the token sees. A row without any is 0 with lse -inf.
//
// A task is two tiles of 256 tokens of a request and head, 128 rows to either block of a cluster; 192 dims of scores
// and 128 of values are 640 operations a query and key, so products bound it. They are the tcgen05 instructions that
// span both blocks: a block of 128 keys is S = Q K^T (12 instructions of 256 x 128 x 16) and O += P V (8) for a
// tile, and either block holds half of it, 64 keys for the scores and 64 dims for the values. In one block's own
// instructions (128 x 128 x 16) the scores' two operands kept shared memory busy for 92 clocks each, where the
// arithmetic takes 64, and left room for little more than one block of keys. TMEM holds S and O of both tiles (4 x 128
// columns), the weights P as bf16 in place of the scores. A tile's next scores need its weights' product to have
// ended, so while one tile's softmax runs (a thread a row), the other's products do: the tiles take turns. The last
// commit that a tile's scores wait for covers the product before them, so O may be rescaled then; that is done
// lazily, when a row's maximum grew by more than 8: o is the same quotient whatever m is, as both of its sums carry
// 2^-m (weights up to 2^8, far inside fp32).
//
// Which tiles make a task: two heads' of the same tokens, or two in a row of one head (kExpShared). Tasks are dealt out
// in turn to one cluster per pair of SMs, those of most keys first and each round in the other direction; in the order
// of requests instead, five prompts of 763 to 1500 tokens took the last cluster 20% longer than the mean. What does
// not fill the last round is split along the keys; its parts leave records, which a second kernel merges in order, so
// results are bitwise reproducible.
//
// Measured, with the merge (one GB300): 1024 tokens behind 2500 keys, 128 heads: 192 us (1.32 PFLOP/s); five
// prompts of up to 1500 tokens, 32 heads: 92 us (0.82). A block of keys takes 2820 clocks of 512 rows, of which
// products are 2560: the softmax of a tile, 1070, and the two hand-overs, 400, take as long as the other's products. A
// task's begin, end and masked blocks take some 7000 beside that. Values are looked over for what is not finite by the
// warps of the softmax: the warp that relays took 4300 clocks for a block, at the end of every tile two of them. Tiles
// that go through the tasks each by itself, so that one's last blocks run beside the other's next task, took more in the
// middle (3200 to 3500 clocks a block) than they saved.
//
// Weights are rounded to bf16 for their product with the values (2^-8 each, the size of the result's own
// rounding); their sum, the maxima, the outputs and the records are fp32.
#pragma once

#include <type_traits>

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
// Keys from which on two tiles in a row of a head make a task, and blocks of keys are loaded once for both. Below, two
// heads' tiles do, which end together: of two in a row the first sees two blocks fewer. Two in a row always and never, in
// us, by keys 1024, 1500, 2200, 2600, 3600, 4500: 1024 tokens of 128 heads 69 and 62, 93 and 92, 126 and 126, 142 and 144,
// 187 and 191, 225 and 234; 512 tokens of 128 heads 47 and 46, 60 and 59, 78 and 77, 87 and 86, 111 and 111, 132 and 133;
// of four requests of 512 tokens and 128 heads (to 2200) 136 and 134, 179 and 180, 243 and 258; 2048 tokens of 32 heads
// (from 2200) 59 and 55, 68 and 64, 92 and 88, 113 and 109. So where the two cross goes by the number of tasks too, from
// 1400 keys on to beyond 4500; of 108 shapes any switch from 1600 to 4000 is in the mean within 0.2% of any other.
// Short prompts want one below: five of 763 to 1500, 32 heads 105 and 91; 300 tokens 16 times 81 and 69.
constexpr int kExpShared = 2560;
constexpr int kExpPeek = 3;            // blocks before an item's end that the next one's queries are asked for in L2
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
    static constexpr int kScores = kReadyQ + 16, kEnded = kScores + 16, kWeights = kEnded + 16, kDrain = kWeights + 16;
    static constexpr int kBarsEnd = kDrain + 8;
    static constexpr int kMisc = kBarsEnd;                    // flags, TMEM address
    static constexpr int kSums = kMisc + 16;                  // int [12]: the scan's sums
    static constexpr int kList = kSums + 64;                  // int [kExpMaxEntries]: what tasks are made of, the dearest first
    static constexpr int kBytes = kList + 4 * (kPagedMaxTokens / kExpTile + kPagedMaxSeqs);
};
static_assert(ExpSmem::kBytes <= 227 * 1024, "it fits");
// An entry of the list: a request, a tile of it by its 256 tokens, whether the next tile belongs to it too, and
// how many entries before it are of two tiles.
constexpr int kExpMaxEntries = kPagedMaxTokens / kExpTile + kPagedMaxSeqs;
constexpr int kExpNameBits = 20, kExpReqBits = 10;
static_assert(kPagedMaxSeqs <= 1 << kExpReqBits && 2 * kPagedMaxTokens / kExpTile <= 1 << (kExpNameBits - kExpReqBits) &&
              kExpMaxEntries <= 1 << (31 - kExpNameBits) && kExpMaxEntries <= 1 << 11, "they fit their bits");
static_assert(8 * kExpMaxEntries <= ExpSmem::kK, "the list is made where the queries go");

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

// A tile's part: 256 tokens of a request and head, and some of its blocks of keys.
struct ExpPart {
    int h, first;              // head, first token of the tile in the request
    int tok0, n, k0, len;      // the request's tokens and keys
    int b0, end;               // blocks of keys
    __device__ __forceinline__ int rows() const { return max(0, min(kExpTile, n - first)); }
    // keys that token i of the request sees
    __device__ __forceinline__ int visible(int i) const { return max(0, min(len, len - n + i + 1)); }
};
// A task's part.
struct ExpItem {
    ExpPart a, b;              // of either tile
    bool shared;               // of the same keys: blocks are loaded once for both
    int part, parts;           // which of how many parts
    int rec;                   // its record's number
    __device__ __forceinline__ int blocks() const { return max(a.end - a.b0, b.end - b.b0); }
    // Blocks that are loaded; and the place among them of tile t's j-th (they go by turns).
    __device__ __forceinline__ int loaded() const { return shared ? blocks() : a.end - a.b0 + b.end - b.b0; }
    __device__ __forceinline__ int place(int t, int j) const {
        return shared ? j : j + (t ? min(j + 1, a.end - a.b0) : min(j, b.end - b.b0));
    }
};

// The entries of a request: fn(name, keys) for every one.
template <typename Fn>
__device__ __forceinline__ int latent_expanded_entries(int b, int n, int len, const Fn &fn) {
    int entries = 0;
    CFA_ROLLED for (int i = 0; i * kExpTile < n; ++entries) {
        const int keys = min(len, max(0, len - n + (i + 2) * kExpTile));  // (half a block more or less is no matter)
        const bool two = keys > kExpShared && (i + 1) * kExpTile < n;
        fn(b << (kExpNameBits - kExpReqBits) | i << 1 | (two ? 1 : 0), keys);
        i += two ? 2 : 1;
    }
    return entries;
}
// Tasks of the entries before entry `at`: an entry of two tiles makes a task for every head, one of a single tile for
// every two heads.
__device__ __forceinline__ int latent_expanded_start(const LatentExpandedParams &p, int at, int twos) {
    return twos * p.H + (at - twos) * ((p.H + 1) / 2);
}
// Lists the entries in smem, those of most blocks first: dealt out in turn and back, tasks come out even, and
// what is left for the last round is cheap. The number of tasks, or -1 where the offsets are not in order, and of
// entries. `work` holds 8 bytes an entry. By all threads of the block.
template <int kThreads>
__device__ __forceinline__ int latent_expanded_list(const LatentExpandedParams &p, int *list, int2 *work, int *sums, int &entries) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads, first = tid * per, last = min(p.B, first + per);
    int mine = 0;
    bool bad = false;
    CFA_ROLLED for (int b = first; b < last; ++b) {
        const int a = __ldcg(p.cu + b), e = __ldcg(p.cu + b + 1), ka = __ldcg(p.cu_k + b), ke = __ldcg(p.cu_k + b + 1);
        if (a < 0 || e < a || e > p.T || ka < 0 || ke < ka || ke > p.S) bad = true;
        else mine += latent_expanded_entries(b, e - a, ke - ka, [](int, int) {});
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
    entries = refused ? 0 : all;
    if (refused) return -1;
    CFA_ROLLED for (int b = first; b < last; ++b)
        latent_expanded_entries(b, __ldcg(p.cu + b + 1) - __ldcg(p.cu + b), __ldcg(p.cu_k + b + 1) - __ldcg(p.cu_k + b),
                                [&](int name, int keys) {
                                    // (a key that no other entry has: blocks, then the order of requests)
                                    work[at] = make_int2(min((keys + 127) / 128, (1 << 20) - 1) << 11 | (kExpMaxEntries - 1 - at), name);
                                    ++at;
                                });
    __syncthreads();
    int twos = 0;
    CFA_ROLLED for (int i = tid; i < all; i += kThreads) {
        const int2 x = work[i];
        int ahead = 0;
        twos = 0;
#pragma unroll 8
        for (int j = 0; j < all; ++j) {
            const int2 y = work[j];
            twos += y.y & 1;
            ahead += y.x > x.x ? (y.y & 1) << 16 | 1 : 0;  // entries, and from bit 16 on those of two tiles
        }
        const int rank = ahead & 0xffff, before = ahead >> 16;
        list[rank] = before << kExpNameBits | x.y;
    }
    if (tid == 0) sums[0] = twos;  // (the first thread has an entry if anyone has)
    __syncthreads();
    return latent_expanded_start(p, all, sums[0]);
}

// Task number `task`, part `part` of at most `parts`; false where it has fewer.
__device__ __forceinline__ bool latent_expanded_item(const LatentExpandedParams &p, const int *list, int entries, int task, int part,
                                                     int parts, ExpItem &x) {
    int lo = 0, hi = entries;  // the last entry whose tasks begin no later
    CFA_ROLLED while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (latent_expanded_start(p, mid, list[mid] >> kExpNameBits) <= task) lo = mid;
        else hi = mid;
    }
    const int name = list[lo], k = task - latent_expanded_start(p, lo, name >> kExpNameBits);
    const int req = name >> (kExpNameBits - kExpReqBits) & ((1 << kExpReqBits) - 1);
    const int first = (name >> 1 & ((1 << (kExpNameBits - kExpReqBits - 1)) - 1)) * kExpTile;
    const int tok0 = __ldcg(p.cu + req), tok1 = __ldcg(p.cu + req + 1), k0 = __ldcg(p.cu_k + req), k1 = __ldcg(p.cu_k + req + 1);
    x.shared = name & 1;
    x.a = ExpPart{x.shared ? k : 2 * k, first, tok0, tok1 - tok0, k0, k1 - k0, 0, 0};
    x.b = x.a;
    if (x.shared) x.b.first += kExpTile;
    else if (++x.b.h >= p.H) x.b.n = 0;  // (the last of an odd number of heads is alone)
    auto blocks_of = [](const ExpPart &z) { return z.rows() > 0 ? (z.visible(z.first + z.rows() - 1) + 127) / 128 : 0; };
    const int na = blocks_of(x.a), nb = blocks_of(x.b), blocks = max(na, nb);
    x.part = part;
    x.parts = max(1, min(parts, blocks / kExpLeast));
    if (part >= x.parts) return false;
    int from = 0, to = blocks;
    if (x.parts > 1) {  // (a division takes 150 clocks)
        from = blocks * part / x.parts;
        to = blocks * (part + 1) / x.parts;
    }
    x.a.b0 = from;
    x.a.end = max(from, min(to, na));
    x.b.b0 = from;
    x.b.end = max(from, min(to, nb));
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
    int *list = reinterpret_cast<int *>(smem + S::kList);

    // a thread a barrier, with the arrivals it expects
    if (tid < (S::kBarsEnd - S::kBars) / 8) {
        const int at = S::kBars + 8 * tid;
        uint32_t count = 1;
        if ((at >= S::kReadyK && at < S::kFullV) || (at >= S::kReadyV && at < S::kFullQ) || (at >= S::kReadyQ && at < S::kScores))
            count = 2;  // the relays of both blocks
        if (at >= S::kWeights && at < S::kDrain) count = 8;   // a tile's warps of both blocks
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
    int entries;
    const int tasks = latent_expanded_list<kExpThreads>(p, list, reinterpret_cast<int2 *>(smem + S::kQ),  // (free yet)
                                                        reinterpret_cast<int *>(smem + S::kSums), entries);
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
        if (r < plan.full) return latent_expanded_item(p, list, entries, r * grid + at, 0, 1, x);
        const int task = at / plan.parts, part = at - task * plan.parts;
        x.rec = at;
        return task < plan.rest && latent_expanded_item(p, list, entries, plan.full * grid + task, part, plan.parts, x);
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
                const int blocks = x.blocks();
                auto load = [&](const ExpPart &z, int j) {  // a block's keys or values
                    if (!ok || j >= z.end - z.b0) return;
                    const uint32_t slot = n % kExpSlots, again = n / kExpSlots;
                    const int full = (values ? S::kFullV : S::kFullK) + 8 * slot;
                    if (again > 0) ok = wait_warp((values ? S::kEmptyV : S::kEmptyK) + 8 * slot, (again - 1) & 1, kSiteStageEmpty);
                    if (!ok) return;
                    if (elect_one()) {
                        if (!values) {  // 64 of the keys
                            const uint32_t dst = base + S::kK + slot * kExpKSlot;
                            const int y = z.k0 + 128 * (z.b0 + j) + 64 * rank;
                            mbar_arrive_expect_tx(base + full, kExpKSlot);
                            tma_load_2d(dst, &tm_kv, z.h * kLatKv, y, base + full);
                            tma_load_2d(dst + 64 * 128, &tm_kv, z.h * kLatKv + 64, y, base + full);
                            tma_load_2d(dst + 2 * 64 * 128, &tm_rope, 0, y, base + full);
                        } else {        // 64 of the dims
                            const uint32_t dst = base + S::kV + slot * kExpVSlot;
                            const int dim = z.h * kLatKv + kLatN + 64 * rank, y = z.k0 + 128 * (z.b0 + j);
                            mbar_arrive_expect_tx(base + full, kExpVSlot);
                            tma_load_2d(dst, &tm_kv, dim, y, base + full);
                            tma_load_2d(dst + 64 * 128, &tm_kv, dim, y + 64, base + full);
                        }
                    }
                    __syncwarp();
                    ++n;
                };
                auto query = [&](const ExpPart &z, int t) {
                    if (!ok || z.end == z.b0) return;
                    if (queried >> t & 1) ok = wait_warp(S::kEmptyQ + 8 * t, ~queries >> t & 1, kSiteStageEmpty);
                    if (!ok) return;
                    if (elect_one()) {
                        const uint32_t full_q = base + S::kFullQ + 8 * t;
                        mbar_arrive_expect_tx(full_q, 3 * kExpChunk);
#pragma unroll
                        for (int c = 0; c < 3; ++c)
                            tma_load_2d(base + S::kQ + (3 * t + c) * kExpChunk, &tm_q, z.h * kLatQ + 64 * c, z.tok0 + z.first + 128 * rank,
                                        full_q);
                    }
                    __syncwarp();
                    queried |= 1u << t;
                    queries ^= 1u << t;
                };
                // the next item's queries, in L2 by the time they are loaded
                auto ask = [&](const ExpPart &z) {
                    if (z.end == z.b0 || !elect_one()) return;
#pragma unroll
                    for (int c = 0; c < 3; ++c) tma_prefetch_2d(&tm_q, z.h * kLatQ + 64 * c, z.tok0 + z.first + 128 * rank);
                };
                if (blocks == 0) have = next(r, ahead);
                CFA_ROLLED for (int j = 0; ok && j < blocks; ++j) {
                    if (!x.shared) load(x.a, j);
                    load(x.b, j);
                    if (!values && j == 0) {  // the queries behind the first keys, which find room earlier
                        query(x.a, 0);
                        query(x.b, 1);
                    }
                    if (j == 0) have = next(r, ahead);  // (behind the first copies)
                    if (values && have && j == max(0, blocks - kExpPeek)) {
                        ask(ahead.a);
                        __syncwarp();
                        ask(ahead.b);
                        __syncwarp();
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
            // tells the issuing block what has landed, in the order in which the products take it: by turns of a tile,
            // keys of a block ahead, values
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
                auto begin = [&](const ExpPart &z, int t) {
                    if (z.end == z.b0) return;
                    if (t == 1 || !x.shared) keys();
                };
                auto query = [&](const ExpPart &z, int t) {
                    if (z.end == z.b0) return;
                    pass_on(S::kFullQ + 8 * t, ready_q + 8 * t, queries >> t & 1);
                    queries ^= 1u << t;
                };
                auto block = [&](const ExpPart &z, int j) {
                    const int b = z.b0 + j;
                    if (b + 1 < z.end) keys();
                    if (b >= z.end) return;
                    pass_on(S::kFullV + 8 * (nv % kExpSlots), ready_v + 8 * (nv % kExpSlots), (nv / kExpSlots) & 1);
                    ++nv;
                };
                begin(x.a, 0);
                begin(x.b, 1);
                query(x.a, 0);
                query(x.b, 1);
                CFA_ROLLED for (int j = 0; ok && j < x.blocks(); ++j) {
                    if (!x.shared) block(x.a, j);
                    block(x.b, j);
                }
            }
        } else if (warp == kExpMmaWarp && rank == 0) {
            // -------------------------------------------------- products, by the first block
            const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
            const uint32_t idesc_s = umma_idesc_bf16(256, 128, false, false), idesc_o = umma_idesc_bf16(256, 128, false, true);
            const uint64_t q0 = umma_smem_desc(base + S::kQ, 16, 1024), k0 = umma_smem_desc(base + S::kK, 16, 1024),
                           v0 = umma_smem_desc(base + S::kV, kExpVSlot, 1024);
            uint32_t n = 0, queries = 0, weights = 0;  // blocks loaded before the item's; phases, a bit a tile
            bool ok = true;
            int r = 0;
            ExpItem x, ahead;
            bool have = next(r, x);
            for (; ok && have; x = ahead) {
                const int na = x.a.end - x.a.b0, nb = x.b.end - x.b.b0, blocks = max(na, nb);
                // By one thread: the scores of tile t from loaded block k.
                auto scores = [&](int t, uint32_t k, bool last) {
                    const uint32_t slot = k % kExpSlots;
                    const uint64_t a = q0 + 3 * t * (kExpChunk >> 4), bd = k0 + slot * (kExpKSlot >> 4);
#pragma unroll
                    for (int ks = 0; ks < 12; ++ks)  // 32 bytes a step
                        umma2_bf16(tm + 128 * t, a + (ks >> 2) * (kExpChunk >> 4) + 2 * (ks & 3),
                                   bd + (ks >> 2) * (64 * 128 >> 4) + 2 * (ks & 3), idesc_s, ks > 0);
                    if (t == 1 || !x.shared) umma2_commit(base + S::kEmptyK + 8 * slot);
                    umma2_commit(base + S::kScores + 8 * t);
                    if (last) umma2_commit(base + S::kEmptyQ + 8 * t);
                };
                // Keys or values of tile t's block j have landed (with shared ones the first tile waits for both).
                auto landed = [&](int ready, int t, int j, uint32_t k) {
                    if (x.shared && t == 1 && j < na) return;
                    ok = ok && wait_warp(ready + 8 * (k % kExpSlots), (k / kExpSlots) & 1, kSiteStageFull);
                };
                CFA_ROLLED for (int t = 0; ok && t < 2; ++t) {
                    if ((t ? nb : na) == 0) continue;
                    const uint32_t k = n + x.place(t, 0);
                    landed(S::kReadyK, t, 0, k);
                    ok = ok && wait_warp(S::kReadyQ + 8 * t, queries >> t & 1, kSiteQExchange);
                    queries ^= 1u << t;
                    tcgen05_fence_after();
                    if (ok && elect_one()) scores(t, k, (t ? nb : na) == 1);
                    __syncwarp();
                }
                have = next(r, ahead);  // (beside the first softmax)
                CFA_ROLLED for (int j = 0; ok && j < blocks; ++j) {
                    CFA_ROLLED for (int t = 0; ok && t < 2; ++t) {
                        const int end = t ? nb : na;
                        if (j >= end) continue;
                        const bool more = j + 1 < end;
                        const uint32_t k = n + x.place(t, j + 1), v = n + x.place(t, j), slot = v % kExpSlots;
                        if (more) landed(S::kReadyK, t, j + 1, k);
                        landed(S::kReadyV, t, j, v);
                        ok = ok && wait_warp(S::kWeights + 8 * t, weights >> t & 1, kSiteSoftmaxExchange);
                        weights ^= 1u << t;
                        tcgen05_fence_after();
                        // the product and the next scores in one go: between two goes the tensor core runs dry for some 400 clocks
                        if (ok && elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)  // 16 keys of 128 bytes a step
                                umma2_bf16_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * ks, v0 + slot * (kExpVSlot >> 4) + 128 * ks,
                                              idesc_o, j > 0 || ks > 0);
                            if (t == 1 || !x.shared) umma2_commit(base + S::kEmptyV + 8 * slot);
                            if (more) scores(t, k, j + 2 == end);
                            else umma2_commit(base + S::kEnded + 8 * t);
                        }
                        __syncwarp();
                    }
                }
                n += x.loaded();
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
        uint32_t ended = 0;  // phase
        const uint32_t weights = map_to_rank(base + S::kWeights, 0) + 8 * t;
        uint32_t scored = 0, nv = 0;  // phases; both tiles' blocks before the item's
        int r = 0;
        ExpItem x, ahead;
        bool have = next(r, x);
        for (; have; x = ahead) {
            const ExpPart z = t ? x.b : x.a;
            // of a split task, for the merge: where a tile's rows are and how many parts it has
            if (r > plan.full && plan.parts > 1 && x.part == 0 && rank == 0 && row == 0)
                p.splits[2 * (x.rec / plan.parts) + t] = make_int4((z.tok0 + z.first) * p.H + z.h, z.rows(), x.parts, x.rec);
            const int first = z.first + 128 * rank;  // this block's first token of the tile
            const int rows = max(0, min(128, z.rows() - 128 * rank));
            const bool live = row < rows, warp_live = row - lane < rows;
            // (rows past the last see what that one sees, so that their warp takes no masked blocks for them: they took 20%
            // of the time of a prompt that ends inside a warp's rows)
            const int see = z.visible(first + min(row, max(rows, 1) - 1));
            // keys that every row of the tile sees, and that any does to whom they belong; blocks whose values it looks over
            const int some = z.visible(z.first), all = t || x.shared ? x.b.visible(x.b.first + x.b.rows() - 1) : z.visible(z.first + z.rows() - 1);
            const int look = x.shared && t ? x.a.end : z.b0;
            float m = -INFINITY, l = 0.f;
            auto block = [&](auto masked, int b) {  // of keys; masked: that not every row sees as a whole
                wait(scores, scored & 1, kSiteSoftmaxExchange);
                __syncwarp();
                tcgen05_fence_after();
                if (warp_live) {
                    uint32_t s[128];
#pragma unroll
                    for (int c = 0; c < 128; c += 32) tmem_ld_x32(t_s + c, s + c);
                    tmem_wait_ld();
                    const int lim = see - 128 * b;
                    if (masked.value && !__all_sync(~0u, lim >= 128)) {
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
                        if (b > z.b0) {
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
                if (masked.value && b >= look) {
                    // Keys from `some` on are not seen by every row, from `all` on by none. A masked weight is 0, and 0
                    // times NaN is NaN: what is not finite becomes 0, and the merge adds it to the rows that see it. (A
                    // thread 16 bytes of every 16th row; of a row's chunks any order will do.)
                    const uint32_t at = nv + x.place(t, b - z.b0);
                    wait(S::kFullV + 8 * (at % kExpSlots), (at / kExpSlots) & 1, kSiteStageFull);
                    __syncwarp();
                    uint8_t *v = smem + S::kV + at % kExpSlots * kExpVSlot + (row >> 3) * 128 + ((row & 7) << 4);
                    const int k0 = 128 * b + (row >> 3);
                    uint32_t most = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t m2 = max_abs_bf16x8(most, *reinterpret_cast<const uint4 *>(v + i * 2048));
                        most = k0 + 16 * i < some ? most : m2;
                    }
                    if (odd_bf16x2(most) != 0u) {
                        CFA_ROLLED for (int i = 0; i < 8; ++i) {
                            const int k = k0 + 16 * i;
                            if (k < some) continue;
                            uint4 w = *reinterpret_cast<const uint4 *>(v + i * 2048);
                            const uint32_t f = odd_bf16x2(w.x), h = odd_bf16x2(w.y), o = odd_bf16x2(w.z), q = odd_bf16x2(w.w);
                            if ((f | h | o | q) != 0u && k < all) {
                                p.odd_tiles[static_cast<unsigned>(z.tok0 + z.first) / kExpTile] = 1;
                                *p.odd = 1u;
                            }
                            *reinterpret_cast<uint4 *>(v + i * 2048) = make_uint4(w.x & ~f, w.y & ~h, w.z & ~o, w.w & ~q);
                        }
                        fence_proxy_async_smem();
                    }
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(weights);
                ++scored;
            };
            // (a loop for each: what few blocks need, in one loop with the others, made theirs 100 clocks longer)
            const int whole = max(z.b0, min(z.end, some / 128));
            CFA_ROLLED for (int b = z.b0; b < whole; ++b) block(std::false_type{}, b);
            CFA_ROLLED for (int b = whole; b < z.end; ++b) block(std::true_type{}, b);
            nv += x.loaded();
            const bool any = z.end > z.b0;
            have = next(r, ahead);  // (its loads are on their way meanwhile)
            if (any) wait(S::kEnded + 8 * t, ended++ & 1, kSiteKvExchange);
            __syncwarp();
            tcgen05_fence_after();
            // ---- the tile's results, or its record
            if (warp_live) {
                const int in_task = kExpTile * t + 128 * rank + row;
                const size_t tok = static_cast<size_t>(z.tok0 + first + row);
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
                    if (p.lse && live) p.lse[tok * p.H + z.h] = (m + log2f(l)) * 0.69314718055994531f;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const int odd = lane & 1;
                    const size_t next_row = static_cast<size_t>(p.H) * kLatV;
                    uint16_t *out = p.out + ((tok - odd) * p.H + z.h) * kLatV + 8 * odd;
                    const bool even_live = row - odd < rows, odd_live = row - odd + 1 < rows;
#pragma unroll 1
                    for (int c = 0; c < kLatV; c += 32) {
                        uint32_t v[32];
                        __syncwarp();
                        if (any) {
                            tmem_ld_x32(t_o + c, v);
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
                        for (int h = 0; h < 2; ++h) write_rows_in_pairs(out + c + 16 * h, next_row, w + 8 * h, even_live, odd_live);
                    }
                }
            }
            tcgen05_fence_before();
            __syncwarp();
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

// Values that are not finite, where the attention has cleared them as only some of a tile's rows see them, are added to
// the rows that do (rows that have them already do not change): inf + inf = inf, and what was NaN stays NaN. A tile clears
// them from the key on that its first row does not see, or that the tile before it did not where both were one task.
// So a tile's rows want the keys that its own and the tile before's tokens are the first to see, 512 at most, whatever
// the request's length. Who wrote a row adds to it: the merge's warps to the rows that they merge, and then all
// warps of the grid to the tiles that were not split, of which only those are visited that cleared something, with
// those of other heads and requests whose tokens lie beside theirs.
//
// Measured (one GB300), one infinity in the call: five prompts of up to 1500 tokens, 32 heads 116 us instead of 90;
// 1024 tokens behind 2500, 128 heads 247 instead of 180; 64 prompts of 100 tokens, 32 heads 146 instead of 97. One
// block that went through all tokens of the batch took 5700, 4400 and 6600.

// By a warp: tokens [32 from, 32 to) of a request's tile, head h and 8 dims. A lane reads a token's key, looks for what is
// not finite, and gives it to the lanes behind it.
__device__ __noinline__ void latent_expanded_add_odd(const LatentExpandedParams &p, int b, int tile, int h, int chunk, int from, int to) {
    const int lane = threadIdx.x & 31;
    const int tok0 = p.cu[b], n = p.cu[b + 1] - tok0, k0 = p.cu_k[b], len = p.cu_k[b + 1] - k0;
    const int first = kExpTile * tile, end = min(n, first + 32 * to);
    const uint16_t *values = p.kv + h * kLatKv + kLatN + 8 * chunk;
    float seen[8] = {};
    bool some = false;
    CFA_ROLLED for (int t0 = max(0, first - kExpTile); t0 < end; t0 += 32) {
        const int t = t0 + lane;
        float v[8] = {};
        bool mine = false;
        if (t >= max(1, n - len) && t < end) {  // token t is the first that sees key len - n + t (the first token's keys all see)
            unpack8_bf16(*reinterpret_cast<const uint4 *>(values + (k0 + len - n + t) * p.kv_stride), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool odd = !(fabsf(v[e]) < INFINITY);
                v[e] = odd ? v[e] : 0.f;
                mine |= odd;
            }
        }
        const unsigned odd = __ballot_sync(~0u, mine);
        float add[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) add[e] = seen[e];
        CFA_ROLLED for (unsigned left = odd; left; left &= left - 1) {
            const int src = __ffs(left) - 1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = __shfl_sync(~0u, v[e], src);
                seen[e] += x;
                if (lane >= src) add[e] += x;
            }
        }
        some |= odd != 0;
        if (!some || t0 < first + 32 * from || t >= end) continue;
        uint4 *at = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(tok0 + t) * p.H + h) * kLatV + 8 * chunk);
        float y[8];
        unpack8_bf16(*at, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = add[e] == 0.f ? y[e] : y[e] + add[e];
        *at = make_uint4(pack2_bf16_cvt(y[0], y[1]), pack2_bf16_cvt(y[2], y[3]), pack2_bf16_cvt(y[4], y[5]), pack2_bf16_cvt(y[6], y[7]));
    }
}

// By all warps of the grid: the rows that each has merged, then the tiles that were not split. The last block clears the marks.
__device__ __noinline__ void latent_expanded_add_odd_all(const LatentExpandedParams &p, int rest) {
    const int tid = threadIdx.x, lane = tid & 31, warps = static_cast<int>(gridDim.x) * (kLatMergeThreads / 32);
    int i = static_cast<int>(blockIdx.x) * (kLatMergeThreads / 32) + (tid >> 5);
    CFA_ROLLED for (int k = i; k < rest * 128; k += warps) {  // the merge's own loop
        const int4 x = __ldcg(p.splits + 2 * (k >> 7) + (k >> 3 & 1));
        if (x.z == 1 || x.y == 0) continue;
        const int tok = x.x / p.H;
        int b = p.B - 1;  // the request that it belongs to
        CFA_ROLLED while (p.cu[b] > tok) --b;
        CFA_ROLLED for (int c = 0; c < 2; ++c)  // (16 dims)
            latent_expanded_add_odd(p, b, (tok - p.cu[b]) / kExpTile, x.x - tok * p.H, 2 * (k >> 4 & 7) + c, k & 7, (k & 7) + 1);
    }
    constexpr int kChunks = kLatV / 8;
    auto marked = [&](int tok) { return __ldcg(p.odd_tiles + tok / kExpTile) != 0; };
    CFA_ROLLED for (int b = 0; b < p.B; ++b) {  // i goes through all requests' units in turn
        const int tok0 = p.cu[b], units = (p.cu[b + 1] - tok0 + kExpTile - 1) / kExpTile * p.H * kChunks;
        CFA_ROLLED for (; i < units; i += warps) {
            const int tile = i / (p.H * kChunks), at = i - tile * p.H * kChunks, h = at / kChunks, tok = tok0 + tile * kExpTile;
            bool skip = !marked(tok) && (tile == 0 || !marked(tok - kExpTile));
            CFA_ROLLED for (int k = lane; k < 2 * rest; k += 32) {  // (its rows were the merge's)
                const int4 x = __ldcg(p.splits + k);
                skip |= x.x == tok * p.H + h && x.y > 0 && x.z > 1;
            }
            if (!__any_sync(~0u, skip)) latent_expanded_add_odd(p, b, tile, h, at - h * kChunks, 0, kExpTile / 32);
        }
        i -= units;
    }
    __shared__ bool last;
    __syncthreads();
    if (tid == 0) last = atomic_add_acq_rel_gpu(p.odd + 1, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;  // others may still read them
    if (tid < 2) p.odd[tid] = 0;
    CFA_ROLLED for (int i = tid; i < kExpMarks; i += kLatMergeThreads) p.odd_tiles[i] = 0;
}

// Merges the records of the split tasks, a warp for 32 rows (a lane a row) and 16 dims.
__global__ void __launch_bounds__(kLatMergeThreads, 3) latent_expanded_merge_kernel(const __grid_constant__ LatentExpandedParams p) {
    grid_dependency_wait();
    const unsigned odd = __ldcg(p.odd);
    const int rest = __ldcg(p.rest);
    const int lane = threadIdx.x & 31, warps = static_cast<int>(gridDim.x) * (kLatMergeThreads / 32);
    constexpr int kRec = kExpRows * (kLatV / 4);
    CFA_ROLLED for (int i = static_cast<int>(blockIdx.x) * (kLatMergeThreads / 32) + (threadIdx.x >> 5); i < rest * 128; i += warps) {
        const int4 x = __ldcg(p.splits + 2 * (i >> 7) + (i >> 3 & 1));  // the tile's first row's place, rows, parts, the first record
        const int row = (i & 15) * 32 + lane, in_tile = row % kExpTile, chunk = (i >> 4 & 7) * 4, parts = x.z;
        if (parts == 1 || in_tile >= x.y) continue;
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
        const size_t at = static_cast<size_t>(x.x) + static_cast<size_t>(in_tile) * p.H;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4 *>(p.out + at * kLatV + 4 * chunk + 8 * c) =
                make_uint4(pack2_bf16_cvt(a[8 * c] * inv, a[8 * c + 1] * inv), pack2_bf16_cvt(a[8 * c + 2] * inv, a[8 * c + 3] * inv),
                           pack2_bf16_cvt(a[8 * c + 4] * inv, a[8 * c + 5] * inv), pack2_bf16_cvt(a[8 * c + 6] * inv, a[8 * c + 7] * inv));
        if (p.lse && chunk == 0) p.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
    }
    if (odd) latent_expanded_add_odd_all(p, rest);
    grid_dependents_launch();
}

}  // namespace cfa
