// cfa_paged_attn.cuh -- attention of a ragged batch over a prefix that all its
// requests share and each request's own pages.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = scale log2(e) q . k_j,
//   m = max_j s_j;  lse = (m + log2 sum_j w_j) ln 2
//
// over the prefix's keys and, of request b's own len_b keys, those up to
// len_b - n_b + i for its i-th of n_b query tokens. A row without keys is 0
// with lse -inf.
//
// One launch of one block per SM works through the runs of cfa_paged_split.h,
// and a second one merges the records of rows whose keys several pieces hold.
// Two load warps stream K and V through rings of 128-key stages (TMA boxes of
// 64 dims with 128-byte swizzle, each inside one page); what the two compute
// warpgroups do with a stage depends on how many query rows the piece has:
//   up to 16 rows   the piece goes to one warpgroup, the next one to the other, so
//                   that one streams while the other begins or ends a piece: four
//                   warps, 32 keys of a block each, on mma.sync with a running max
//                   and sum per warp, joined in shared memory at the piece's end.
//                   The bytes of the keys bound it, and the 16-row instruction wastes
//                   least on a few rows
//   up to 128 rows  tcgen05, one tile of queries; even blocks of keys go to one
//                   warpgroup and odd ones to the other, each with its own
//                   scores and outputs in TMEM
//   up to 256 rows  tcgen05, two tiles of queries, one to a warpgroup, on the
//                   same keys
// On tcgen05 a block's keys go in two halves: S = Q K^T (M = 128 rows, N = 64
// keys) of the next half runs while a thread per row takes this half's scores from
// TMEM and writes the weights back over them as bf16; O += P V reads them there. A
// warpgroup has an MMA warp of its own. A row's maximum is followed lazily: the result
// is the same quotient whatever reference its two sums carry, so O is rescaled only when
// the maximum grew by more than 8 (weights up to 2^8, far inside fp32), which is rare.
//
// Weights are rounded to bf16 for the product with V (tensor cores take both
// operands in one type; 2^-8 each, the size of the result's own rounding); their
// sum, the maxima, the outputs and the records are fp32.
//
// Measured, with the merge (one GB300, 32 heads x 128 where not said):
//   16 requests, 4096 shared keys and some 1024 own ones, no groups: 46.2 us, 213 MB (4.6 TB/s)
//   64 requests, 32768 and 2048, 8 key heads: 85 us, 431 MB (5.1 TB/s)
//   256 requests, 8192 and 512, 8 key heads, pages of 16: 92 us, 315 MB
//   8 requests of up to 512 new tokens, 4096 and 1500, 8 key heads: 228 us (1.14 PFLOP/s)
//   one request, 64 and 64 keys: 10.7 us
// What bounds it: many keys, the memory, with some 4 us before the first copy (the plan, and
// instructions that arrive one line after the other) and 4 us of the merge; small pieces over
// small pages, the copies' issue (80 clocks a box) on two stages of K and of V; many rows, the
// products and the softmax alike: a half of 64 keys and 256 rows takes 1500 clocks of products
// (the 64-key scores read their 128 query rows from shared memory for 59 clocks where the
// arithmetic takes 34) and 1575 of softmax with its waits. Scores of 128 keys at once spend
// fewer clocks but find no second buffer in TMEM: 249 us instead of 229 then. The loops' code has to
// stay in the instruction cache: versions above some 7600 instructions lost 5%.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "cfa_device.cuh"
#include "cfa_paged.h"
#include "cfa_paged_device.cuh"
#include "cfa_paged_split.h"
#include "cfa_tensor.cuh"
#include "cfa_tile.cuh"

namespace cfa {

// Register share of the calling warpgroup. The block is launched with 512 x 128 =
// 65,536; the two compute warpgroups take 176 a thread and the others keep 80:
// 128 x (176 + 176 + 80 + 80) = 65,536.
__device__ __forceinline__ void registers_for_compute() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
}
__device__ __forceinline__ void registers_for_issue() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
}

// Blocks of keys whose cache rows the address warp finds ahead of the load warps, four
// at a time: entries of 12 ints (up to 8 boxes' rows, their number, and whether the run
// ends here), groups of 4 entries.
constexpr int kPagedGroups = 4;
constexpr int kPagedEntry = 12;
// Pieces that the prep warp has laid out at most.
constexpr int kPagedSlots = 3;

// Shared memory of the attention kernel for head_dim D.
template <int D>
struct PagedSmem {
    static constexpr int kStage = kPagedKeys * D * 2;           // one block of K or V
    static constexpr int kHalf = kPagedKeys * 128;              // its 64-dim column halves
    static constexpr int kStages = D == 128 ? 2 : 4;            // of K, and as many of V
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kQ = 0;                                // two query tiles; scratch otherwise
    static constexpr int kRing = 2 * kQTile;
    // a piece: its numbers, where its rows lie (int [256]: token and head of the group), then
    // up to 16 query rows, [D / 64][16][64] swizzled
    static constexpr int kSlots = kRing + 2 * kStages * kStage;
    static constexpr int kSlotRows = 128, kSlotQ = kSlotRows + 256 * 4, kSlot = kSlotQ + 16 * D * 2;
    static constexpr int kMl = kSlots + kPagedSlots * kSlot;    // float2 [128]: max and sum
    static constexpr int kBars = kMl + 128 * 8;
    static constexpr int kMisc = kBars + 48 * 8;                // flags, TMEM address, scan sums
    static constexpr int kFifo = kMisc + 256;                   // the address warp's entries
    static constexpr int kArrays = kFifo + 4 * kPagedGroups * kPagedEntry * 4;  // PagedEntry [B + 1]
    static int bytes(int B) { return kArrays + 16 * (B + 1) + 1024; }
};
static_assert(sizeof(PagedPiece) <= 128, "a piece fits its slot");
constexpr int kPagedBars = 48;

// A count that one thread raises and others wait for, within the same bound as a barrier.
__device__ __forceinline__ void paged_publish(int *count, uint32_t v) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" :: "r"(smem_addr(count)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t paged_count(const int *count) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_addr(count)) : "memory");
    return v;
}
// A row's entry in a piece's table: its token, and its head within the group above that.
constexpr int kPagedTokenBits = 18;
constexpr int kPagedTokenMask = (1 << kPagedTokenBits) - 1;
static_assert(kPagedMaxTokens <= kPagedTokenMask, "a token fits its bits");
template <int D>
__device__ __forceinline__ const uint16_t *paged_query(const PagedAttnParams &p, int at, int h) {
    return p.q + (at & kPagedTokenMask) * p.q_stride + (h * p.shape.G + (at >> kPagedTokenBits)) * D;
}

// What of a stage's values must not meet masked weights, which are 0, and 0 times NaN is NaN: rows
// [keys, end), past the keys, may hold anything and become 0; of rows [begin, keys), which some
// query rows see and others do not, what is not finite becomes 0, and the merge is told to add
// it to the rows that see it. By `threads` threads, of which this is the t-th.
template <int D>
__device__ __forceinline__ void paged_clear(const PagedAttnParams &p, uint8_t *rows, int begin, int keys, int end, int t,
                                            int threads) {
    CFA_ROLLED for (int i = t; i < (end - begin) * (D / 8); i += threads) {
        const int r = begin + i / (D / 8), c = i % (D / 8);  // (of a row's chunks any order will do)
        uint4 *at = reinterpret_cast<uint4 *>(rows + (c >> 3) * PagedSmem<D>::kHalf + r * 128 + ((c & 7) << 4));
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < keys) {
            v = *at;
            const uint32_t a = odd_bf16x2(v.x), b = odd_bf16x2(v.y), d = odd_bf16x2(v.z), e = odd_bf16x2(v.w);
            if ((a | b | d | e) == 0u) continue;
            *p.odd = 1u;
            v = make_uint4(v.x & ~a, v.y & ~b, v.z & ~d, v.w & ~e);
        }
        *at = v;
        if (r < keys) fence_proxy_async_smem();  // (the stage's next copy comes after)
    }
}

template <bool V>
struct PagedFlag {
    static constexpr bool value = V;
};

template <int D>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedAttnParams p) {
    using S = PagedSmem<D>;
    constexpr int NS = S::kStages;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    const uint32_t ring = base + S::kRing;
    const uint32_t bar_full = base + S::kBars, bar_empty = bar_full + 16 * NS;  // K's stages, then V's
    const uint32_t bar_both = bar_empty + 16 * NS, bar_q = bar_both + 8, bar_s = bar_q + 8, bar_p = bar_s + 32,
                   bar_drain = bar_p + 32, bar_piece = bar_drain + 16, bar_piece_free = bar_piece + 8 * kPagedSlots,
                   bar_entry = bar_piece_free + 8 * kPagedSlots, bar_entry_free = bar_entry + 8 * kPagedGroups;
    int *misc = reinterpret_cast<int *>(smem + S::kMisc);
    volatile int *timed_out = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);
    PagedEntry *req = reinterpret_cast<PagedEntry *>(smem + S::kArrays);
    int *entries = reinterpret_cast<int *>(smem + S::kFifo);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kMl);

    // a thread a barrier, with the arrivals it expects
    if (tid < kPagedBars) {
        const uint32_t bar = base + S::kBars + 8 * tid;
        uint32_t count = 1;
        if (bar >= bar_empty && bar < bar_both) count = 4;  // warps of a warpgroup, or arrivals and commits
        if (bar == bar_both || bar == bar_q) count = kComputeThreads;
        if (bar >= bar_p && bar < bar_drain) count = 4;
        if (bar >= bar_piece && bar < bar_piece_free) count = 33;  // the prep warp's lanes, and their word
        if (bar >= bar_piece_free && bar < bar_entry) count = kComputeWarps + 2;
        if (bar >= bar_entry_free) count = 2;
        mbar_init(bar, count);
        if (tid < 8 && tid != 1) misc[tid] = 0;  // (misc[1]: the TMEM address)
        fence_mbar_init();
    }
    if (warp == kComputeWarps) tmem_alloc(smem_addr(tmem_slot), 512);
    if (warp == kComputeWarps + 1 && elect_one()) {
        prefetch_tensor_map(&tm_k);
        prefetch_tensor_map(&tm_v);
    }
    tcgen05_fence_before();
    grid_dependency_wait();

    // ---- every block scans the requests, a thread a request
    const PagedShape &shape = p.shape;
    const int B = p.B, G = shape.G;
    PagedPlan plan;
    {
        // sums of each warp: units of blocks, items, tokens that share; sums of units and items
        // stop at the limit, which makes the plan invalid
        int *sums = reinterpret_cast<int *>(smem + S::kQ), *items_before = sums + 64;  // (free until the first piece)
        int units = 0, items = 0, tokens = 0;
        bool bad = false, refused = false;
        const int cu_first = __ldcg(p.cu), cu_end = __ldcg(p.cu + B);
        auto more = [](int a, int b) { return min(a + b, kPagedMaxUnits); };
        CFA_ROLLED for (int first = 0; first < B; first += kPagedThreads) {
            const int b = first + tid;
            PagedRequest r{0, 0, 0};
            int u = 0, k = 0, t = 0;
            if (b < B) {
                r.tok0 = __ldcg(p.cu + b);
                r.n = __ldcg(p.cu + b + 1) - r.tok0;
                r.len = __ldcg(p.lens + b);
                if (r.len < 0 || r.len > static_cast<long long>(p.width) * p.page_size) {
                    r.len = 0;
                    if (blockIdx.x == 0) atomicOr(p.status, kStatusBadLengthBit);
                }
                if (r.tok0 < 0 || r.n < 0 || r.n > p.T || r.tok0 > p.T - r.n) {
                    bad = true;
                } else {
                    const PagedCost cost = paged_request_cost(shape, r);
                    u = static_cast<int>(min(cost.blocks, static_cast<long long>(kPagedMaxUnits)));
                    k = static_cast<int>(min(cost.items, static_cast<long long>(kPagedMaxUnits)));
                    t = paged_alone(shape, r.n) ? 0 : r.n;
                }
            }
            int su = u, sk = k, st = t;
            CFA_ROLLED for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(~0u, su, o), c = __shfl_up_sync(~0u, sk, o), d = __shfl_up_sync(~0u, st, o);
                if (lane >= o) su = more(su, a), sk = more(sk, c), st += d;
            }
            if (lane == 31) sums[warp] = su, sums[16 + warp] = sk, sums[32 + warp] = st;
            refused |= __syncthreads_or(bad) != 0;
            int wu = 0, wk = 0, wt = 0;
            if (lane < 16) wu = sums[lane], wk = sums[16 + lane], wt = sums[32 + lane];
            CFA_ROLLED for (int o = 1; o < 16; o <<= 1) {
                const int a = __shfl_up_sync(~0u, wu, o), c = __shfl_up_sync(~0u, wk, o), d = __shfl_up_sync(~0u, wt, o);
                if (lane >= o) wu = more(wu, a), wk = more(wk, c), wt += d;
            }
            const int left = (warp + 31) & 31;
            const int bu = __shfl_sync(~0u, wu, left), bk = __shfl_sync(~0u, wk, left), bt = __shfl_sync(~0u, wt, left);
            if (b < B) {
                req[b] = PagedEntry{more(units, su - u + (warp ? bu : 0)), tokens + st - t + (warp ? bt : 0), r.tok0, r.len};
                items_before[b] = more(items, sk - k + (warp ? bk : 0));
            }
            units = more(units, __shfl_sync(~0u, wu, 15));
            items = more(items, __shfl_sync(~0u, wk, 15));
            tokens += __shfl_sync(~0u, wt, 15);
            if (first + kPagedThreads < B) __syncthreads();  // the sums are read
        }
        if (tid == 0) req[B] = PagedEntry{units, tokens, cu_end, 0};
        const int all_tokens = cu_end - cu_first;
        plan = paged_plan(shape, PagedCost{units, items}, tokens, all_tokens - tokens, p.block_clocks, !refused);
        CFA_ROLLED for (int b = tid; b < B; b += kPagedThreads) req[b].unit += items_before[b] * plan.item_units;
        if (tid == 0) req[B].unit += items * plan.item_units;
        __syncthreads();
        tcgen05_fence_after();
        if (blockIdx.x == 0 && tid == 0) {
            PagedPlan told = plan;
            told.by_share = FastDiv(static_cast<uint32_t>(plan.share));
            *reinterpret_cast<PagedPlan *>(p.plan_ws) = told;
            if (!plan.valid) atomicOr(p.status, kStatusBadLengthBit);
        }
    }
    grid_dependents_launch();
    const uint32_t tmem = *tmem_slot;
    const int run = blockIdx.x;
    const long long first = static_cast<long long>(run) * plan.share;
    const int u0 = static_cast<int>(min(first, static_cast<long long>(plan.units)));
    const int u1 = static_cast<int>(min(first + plan.share, static_cast<long long>(plan.units)));
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned site) {
        return bounded_wait([&]() { return mbar_try_wait(bar, parity); }, p.timeout_ns, timed_out, p.status, site);
    };
    // The same for a warp as a whole.
    auto wait_warp = [&](uint32_t bar, uint32_t parity, unsigned site) {
        return __all_sync(~0u, wait(bar, parity, site));
    };
    // Block n of the run lies in stage n % NS of each ring (K: 0, V: 1), in its n / NS-th pass.
    auto slot_of = [&](int v, uint32_t n) { return v * NS + n % NS; };
    auto stage_at = [&](int v, uint32_t n) { return ring + slot_of(v, n) * S::kStage; };
    auto wait_full = [&](int v, uint32_t n) { wait(bar_full + 8 * slot_of(v, n), (n / NS) & 1, kSiteStageFull); };
    // Keys of block j of a piece's item: where they lie and how many there are.
    auto block_keys = [&](const PagedPiece &x, int j, int *key0) {
        const bool pre = j < x.prefix_blocks;
        *key0 = (pre ? j : j - x.prefix_blocks) * kPagedKeys;
        return min(kPagedKeys, (pre ? p.prefix_len : x.own_limit) - *key0);
    };
    // Where a row of a piece's tile lies: its token and its head of the group.
    auto find_row = [&](const PagedPiece &x, int r) {
        const int i = (x.row0 + r) / shape.by_G;
        int t = x.r.tok0 + i;
        if (x.req < 0) {
            const int b = paged_find(B, i, [&](int k) { return req[k].tok; });
            t = req[b].tok0 + i - req[b].tok;
        }
        return t | (x.row0 + r - i * G) << kPagedTokenBits;
    };
    if (warp >= kComputeWarps) {
        registers_for_issue();
        if (warp < kComputeWarps + 2) {
            // -------------------------------------------- load warps: one for K, one for V
            const int v = warp - kComputeWarps;
            uint32_t n = 0;
            const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * 128;
            for (;; ++n) {
                const uint32_t group = n / 4;
                if (n % 4 == 0 && !wait_warp(bar_entry + 8 * (group % kPagedGroups), (group / kPagedGroups) & 1, kSiteStageFull))
                    break;
                const int *e = entries + n % (4 * kPagedGroups) * kPagedEntry;
                const int mine = lane < 10 ? e[lane] : 0;
                if (__shfl_sync(~0u, mine, 9)) break;  // the run's end
                const uint32_t full = bar_full + 8 * slot_of(v, n);
                if (n >= NS && !wait_warp(bar_empty + 8 * slot_of(v, n), (n / NS - 1) & 1, kSiteStageEmpty)) break;
                const int boxes = __shfl_sync(~0u, mine, 8);
                const uint32_t dst = stage_at(v, n);
                if (elect_one()) {
                    mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes) * box_bytes * (D / 64));
                    paged_publish(misc + 4 + v, n + 1);
                }
                __syncwarp();
                CFA_ROLLED for (int k = 0; k < boxes; ++k) {
                    const int y = __shfl_sync(~0u, mine, k);
                    if (elect_one()) {
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_2d(dst + k * box_bytes + h * S::kHalf, v ? &tm_v : &tm_k, 64 * h, y, full);
                    }
                    __syncwarp();
                }
                if (n % 4 == 3 && elect_one()) mbar_arrive(bar_entry_free + 8 * (group % kPagedGroups));
                __syncwarp();
            }
            if (lane == 0 && *timed_out) {
                // a wait gave up: the copies in flight land before the block ends
                const uint64_t t0 = global_timer_ns();
                for (uint32_t k = n > NS ? n - NS : 0; k < n; ++k)
                    while (!mbar_try_wait(bar_full + 8 * slot_of(v, k), (k / NS) & 1) &&
                           global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                    }
            }
            __syncwarp();
        } else if (warp == kComputeWarps + 2) {
            // ------------------------------------------------------- address warp
            // Finds the cache rows of the run's blocks, four at a time (8 lanes each, a lane a
            // box), ahead of the load warps: a table entry takes as long to arrive as the keys.
            const int box = p.box_rows, sub = lane >> 3, i = lane & 7;
            const int all_rows = p.n_pages * p.n_kv * p.page_size;
            PagedPiece x;
            int u = u0, j = 0;  // the next piece, the next block of this one
            x.b1 = 0;
            bool more = true;
            for (uint32_t g = 0; more; ++g) {
                const int *id_at = nullptr;
                int boxes = 0, add = 0;
                bool mine = false, end = false;
                CFA_ROLLED for (int k = 0; k < 4 && more; ++k, ++j) {
                    if (j == x.b1) {
                        more = paged_next(shape, plan, req, B, u, u1, x);
                        j = x.b0;
                    }
                    if (sub == k) {
                        mine = true;
                        if (more) {
                            int key0;
                            const int keys = block_keys(x, j, &key0);
                            boxes = keys > 0 ? (keys + box - 1) / box : 0;
                            const int key = key0 + i * box, pg = key / p.by_page;
                            if (i < boxes)
                                id_at = (j < x.prefix_blocks ? p.prefix_table
                                                             : p.tables + static_cast<size_t>(x.req) * p.width) + pg;
                            add = x.h * p.page_size + key - pg * p.page_size;
                        }
                        end = !more;
                    }
                }
                int y = all_rows;  // outside: reads as zeros
                if (id_at) {
                    const int id = __ldcg(id_at);
                    if (id >= 0 && id < p.n_pages) y = id * p.n_kv * p.page_size + add;
                    else atomicOr(p.status, kStatusBadPageBit);
                }
                if (__any_sync(~0u, g >= kPagedGroups && !wait(bar_entry_free + 8 * (g % kPagedGroups),
                                                               (g / kPagedGroups - 1) & 1, kSiteStageEmpty)))
                    break;
                int *e = entries + (4 * (g % kPagedGroups) + sub) * kPagedEntry;
                if (mine) {
                    e[i] = y;
                    if (i == 0) e[8] = boxes, e[9] = end;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_entry + 8 * (g % kPagedGroups));
            }
        } else if (warp == kComputeWarps + 3) {
            // ---------------------------------------------------------- prep warp
            // Lays pieces out ahead: their numbers, where each row's query and result lie,
            // and the queries themselves where they are few. A piece without blocks ends the run.
            bool more = true;
            int u = u0;
            PagedCut cut{};  // the tile that the run's end cuts, for the merge
            PagedPiece x;
            for (uint32_t k = 0; more; ++k) {
                more = paged_next(shape, plan, req, B, u, u1, x);
                if (!more) x.b0 = x.b1 = x.rows = 0;
                else if (x.req >= 0 && paged_alone(shape, x.r.n) && x.b0 == 0 && x.b1 < x.blocks)
                    cut = PagedCut{x.rows, x.row0, x.r.tok0, x.h, paged_last_run(plan, x.first_unit, x.blocks, x.cost), {0, 0, 0}};
                x.final = more && paged_final(shape, x);
                if (more) paged_record(shape, plan, x.req < 0 ? 0 : req[x.req].tok, run, x);
                if (__any_sync(~0u, k >= kPagedSlots && !wait(bar_piece_free + 8 * (k % kPagedSlots),
                                                              (k / kPagedSlots - 1) & 1, kSiteStageEmpty)))
                    break;
                uint8_t *slot = smem + S::kSlots + k % kPagedSlots * S::kSlot;
                if (lane == 0) *reinterpret_cast<PagedPiece *>(slot) = x;
                const bool few = x.rows <= kPagedSmallRows;
                int *row_at = reinterpret_cast<int *>(slot + S::kSlotRows);
                if (few) {  // (of a tile the compute warps do it, a thread a row)
                    if (lane < x.rows) row_at[lane] = find_row(x, lane);
                    __syncwarp();
                    CFA_ROLLED for (int c = lane; c < 16 * (D / 8); c += 32) {
                        const int r = c / (D / 8), ch = c % (D / 8);
                        uint8_t *dst = slot + S::kSlotQ + (ch >> 3) * 2048 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                        if (r < x.rows)
                            cp_async_16(smem_addr(dst), paged_query<D>(p, row_at[r], x.h) + 8 * ch);
                        else
                            *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                // every lane's arrival follows its copies; the next piece need not wait for them
                cp_async_arrive(bar_piece + 8 * (k % kPagedSlots));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_piece + 8 * (k % kPagedSlots));
            }
            cp_async_wait_all();
            if (lane == 0) *reinterpret_cast<PagedCut *>(p.plan_ws + kPagedPlanInts + 8 * run) = cut;
        } else if (warp < kComputeWarps + 6) {
            // ------------------------------------------- MMA warps, one for a warpgroup
            const int w = warp - (kComputeWarps + 4);
            const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
            const uint32_t d_s = tm + 128 * w, d_o = tm + 256 + D * w, bs = bar_s + 16 * w, bp = bar_p + 16 * w;
            uint32_t n = 0, queries = 0, weights = 0;  // the piece's first block; phases
            for (uint32_t k_piece = 0;; ++k_piece) {
                const uint32_t at_slot = k_piece % kPagedSlots;
                if (!wait_warp(bar_piece + 8 * at_slot, (k_piece / kPagedSlots) & 1, kSiteStageFull)) break;
                const PagedPiece *x = reinterpret_cast<const PagedPiece *>(smem + S::kSlots + at_slot * S::kSlot);
                const int nb = uniform(x->b1 - x->b0), rows = uniform(x->rows);
                __syncwarp();
                if (elect_one()) mbar_arrive(bar_piece_free + 8 * at_slot);
                __syncwarp();
                if (nb == 0) break;
                if (rows > kPagedSmallRows) {
                    wait_warp(bar_q, queries++ & 1, kSiteQExchange);
                    tcgen05_fence_after();
                    const bool split = rows <= 128;
                    const int step = split ? 2 : 1, first_block = split ? w : 0;
                    const uint32_t q = base + S::kQ + (split ? 0 : w * S::kQTile), arrivals = split ? 3 : 1;
                    // scores of half h of block j (64 of the stage's rows: 8192 bytes on)
                    auto scores = [&](int j, int h) {
                        const uint32_t k = stage_at(0, n + j) + 8192 * h;
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)  // 32 bytes a step
                                umma_bf16(d_s + 64 * h, umma_smem_desc(q + (ks >> 2) * S::kHalf, 16, 1024) + 2 * (ks & 3),
                                          umma_smem_desc(k + (ks >> 2) * S::kHalf, 16, 1024) + 2 * (ks & 3),
                                          umma_idesc_bf16(128, 64, false, false), ks > 0);
                            umma_commit(bs + 8 * h);
                            if (h == 1) {  // the keys are read
                                mbar_arrive_n(bar_empty + 8 * slot_of(0, n + j), arrivals);
                                umma_commit(bar_empty + 8 * slot_of(0, n + j));
                            }
                        }
                        __syncwarp();
                    };
                    auto ready = [&](int v, int j) {
                        wait_warp(bar_full + 8 * slot_of(v, n + j), ((n + j) / NS) & 1, kSiteStageFull);
                        tcgen05_fence_after();
                    };
                    if (first_block < nb) {
                        ready(0, first_block);
                        scores(first_block, 0);
                        scores(first_block, 1);
                    }
                    CFA_ROLLED for (int j = first_block; j < nb; j += step, ++weights) {
                        ready(1, j);
                        const bool more = j + step < nb;
                        CFA_ROLLED for (int h = 0; h < 2; ++h) {
                            wait_warp(bp + 8 * h, weights & 1, kSiteSoftmaxExchange);
                            tcgen05_fence_after();
                            const uint64_t vd = umma_smem_desc(stage_at(1, n + j) + 8192 * h, S::kHalf, 1024);
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)  // 16 rows of 128 bytes a step
                                    umma_bf16_ts(d_o, d_s + 64 * h + 8 * ks, vd + 128 * ks, umma_idesc_bf16(128, D, false, true),
                                                 j > first_block || h > 0 || ks > 0);
                                if (h == 1) {  // the values are read
                                    mbar_arrive_n(bar_empty + 8 * slot_of(1, n + j), arrivals);
                                    umma_commit(bar_empty + 8 * slot_of(1, n + j));
                                }
                                // behind the last blocks' values there are no more scores, but the
                                // warpgroup still learns that the products are done
                                if (!more) umma_commit(bs + 8 * h);
                            }
                            __syncwarp();
                            if (more) {
                                if (h == 0) ready(0, j + step);
                                scores(j + step, h);
                            }
                        }
                    }
                }
                n += nb;
            }
            if (elect_one() && *timed_out) {
                // a wait gave up: the products in flight end before the block does
                umma_commit(bar_drain + 8 * w);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar_drain + 8 * w, 0) &&
                       global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
            }
            __syncwarp();
        } else if (warp == kComputeWarps + 6) {
            // --------------------------------------------------------- merge-rows warp
            // For the merge: where each shared row's result goes and its own keys' item.
            for (int r = run * 32 + lane; r < plan.shared_rows; r += shape.grid * 32) {
                const int tok = r / shape.by_G, b = paged_find(B, tok, [&](int k) { return req[k].tok; });
                const PagedRequest q = paged_request_at(req, b);
                const int all = q.n * G, mine = r - req[b].tok * G, tile = paged_own_tile(all);
                const int own = all > tile ? mine / tile : 0, row0 = own * tile, blocks = paged_cdiv(q.len, kPagedKeys);
                PagedRow d;
                d.out_row = (q.tok0 + tok - req[b].tok) * p.n_heads + r - tok * G;
                d.unit = plan.prefix_units + req[b].unit + own * paged_item_units(plan, tile, paged_cost(tile), blocks);
                d.head_units = (req[b + 1].unit - req[b].unit) / shape.by_nkv;
                d.blocks = blocks;
                d.rows = min(tile, all - row0);
                d.row = mine - row0;
                reinterpret_cast<PagedRow *>(p.plan_ws + kPagedPlanInts + 8 * shape.grid)[r] = d;
            }
        }
    } else {
        // ---------------------------------------------------------- compute warps
        registers_for_compute();
        const int wg = warp >> 2, wtid = tid & 127;
        uint32_t n = 0, scored = 0, met = 0;  // the piece's first block; phases
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lanes of this warp
        auto wg_bar = [&]() { asm volatile("bar.sync %0, 128;" :: "r"(2 + wg) : "memory"); };
        // Both warpgroups meet; bounded, as one of them may have given up.
        auto meet = [&]() {
            mbar_arrive(bar_both);
            wait(bar_both, met++ & 1, kSiteKvExchange);
        };
        for (uint32_t k_piece = 0;; ++k_piece) {
            // one thread's word for its warpgroup: where its wait gave up, no warp goes on alone
            const uint32_t at_slot = k_piece % kPagedSlots;
            const bool there = wait(bar_piece + 8 * at_slot, (k_piece / kPagedSlots) & 1, kSiteStageFull);
            volatile int *word = misc + 8 + 2 * wg + (k_piece & 1);  // (read before the next but one is written)
            if (wtid == 0) *word = there;
            wg_bar();
            if (!*word) break;
            const uint8_t *slot = smem + S::kSlots + at_slot * S::kSlot;
            const PagedPiece &x = *reinterpret_cast<const PagedPiece *>(slot);
            const int nb = x.b1 - x.b0;
            if (nb == 0) break;
            const bool few = x.rows <= kPagedSmallRows;
            auto piece_done = [&]() {
                n += nb;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_piece_free + 8 * at_slot);
            };
            if (few && static_cast<int>(k_piece & 1) != wg) {  // the other warpgroup's
                piece_done();
                continue;
            }
            int *row_at = reinterpret_cast<int *>(smem + S::kSlots + at_slot * S::kSlot + S::kSlotRows);
            const bool final = x.final;
            float *rec_o = p.rec_o + x.rec * D + x.rec_row * 4;
            float2 *rec_ml = p.rec_ml + x.rec + x.rec_row;
            const int rec_stride = x.rec_stride;
            auto result_row = [&](int row) {
                const int at = row_at[row];
                return (at & kPagedTokenMask) * p.n_heads + x.h * G + (at >> kPagedTokenBits);
            };
            auto write_lse = [&](int row, float m, float l) {
                if (p.lse) p.lse[result_row(row)] = (m + log2f(l)) * 0.69314718055994531f;
            };

            if (few) {
                // ---- mma.sync: this warp's 32 keys of every block
                const int r0 = lane >> 2, c2 = (lane & 3) * 2, kw = 32 * (warp & 3);
                uint32_t q[D / 16][4];
                {
                    const uint32_t qs = smem_addr(slot + S::kSlotQ) + (lane & 15) * 128;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t c = 2 * k + (lane >> 4);
                        ldmatrix_x4(q[k], qs + (c >> 3) * 2048 + (((c & 7) ^ (lane & 7)) << 4));
                    }
                }
                float o[D / 8][4];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
                float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
                // The other warpgroup's blocks may lie between this one's last and these: a
                // parity says nothing about a stage that is not yet this block's, so the load
                // warps' counts come first.
                uint32_t issued[2] = {0, 0};
                auto wait_issued = [&](int v, uint32_t block) {
                    if (issued[v] <= block)
                        bounded_wait([&]() { return (issued[v] = paged_count(misc + 4 + v)) > block; }, p.timeout_ns,
                                   timed_out, p.status, kSiteStageFull);
                };
                // own keys that rows r0 and r0 + 8 see
                const int see0 = paged_visible(x.r, (x.row0 + r0) / shape.by_G);
                const int see1 = paged_visible(x.r, (x.row0 + r0 + 8) / shape.by_G);
                const uint32_t kkey = kw + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
                const uint32_t vkey = kw + (lane & 15), vc = lane >> 4;
                CFA_ROLLED for (int j = 0; j < nb; ++j) {
                    const uint32_t block = n + j;
                    int key0;
                    const int keys = block_keys(x, x.b0 + j, &key0) - kw;
                    key0 += kw;
                    wait_issued(0, block);
                    wait_full(0, block);
                    __syncwarp();
                    float s[4][4] = {};
                    if (keys > 0) {
                        // chunk 2 k + kc of the row, swizzled: bits 5 and 6 of its address turn with k
                        const uint32_t st = stage_at(0, block) + kkey * 128 + ((kc ^ (kkey & 7)) << 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            uint32_t b[4], d[4];
                            const uint32_t at = (st ^ ((k & 3) << 5)) + (k >> 2) * S::kHalf;
                            ldmatrix_x4(b, at);
                            ldmatrix_x4(d, at + 16 * 128);
                            mma_16x8x16(s[0], q[k], b[0], b[1]);
                            mma_16x8x16(s[1], q[k], b[2], b[3]);
                            mma_16x8x16(s[2], q[k], d[0], d[1]);
                            mma_16x8x16(s[3], q[k], d[2], d[3]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_empty + 8 * slot_of(0, block));
                    uint32_t pr[2][4];
                    int seen = 32;  // of the warp's keys, by every row
                    if (keys > 0) {
                        const bool own = x.b0 + j >= x.prefix_blocks;
                        const int lim0 = own ? min(keys, see0 - key0) : keys;
                        const int lim1 = own ? min(keys, see1 - key0) : keys;
                        seen = uniform(lim0);  // (lane 0 has the first row)
                        float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int col = 8 * t + c2 + e;
                                s[t][e] = col < lim0 ? s[t][e] * p.scale_log2 : -INFINITY;
                                s[t][2 + e] = col < lim1 ? s[t][2 + e] * p.scale_log2 : -INFINITY;
                                a0 = fmaxf(a0, s[t][e]);
                                a1 = fmaxf(a1, s[t][2 + e]);
                            }
#pragma unroll
                        for (int d = 1; d < 4; d <<= 1) {
                            a0 = fmaxf(a0, __shfl_xor_sync(~0u, a0, d));
                            a1 = fmaxf(a1, __shfl_xor_sync(~0u, a1, d));
                        }
                        const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
                        const float f0 = n0 == -INFINITY ? 0.f : n0, f1 = n1 == -INFINITY ? 0.f : n1;
                        if (__any_sync(~0u, n0 != m0 || n1 != m1)) {
                            const float g0 = exp2_ftz(m0 - f0), g1 = exp2_ftz(m1 - f1);
                            l0 *= g0;
                            l1 *= g1;
#pragma unroll
                            for (int i = 0; i < D / 8; ++i) {
                                o[i][0] *= g0; o[i][1] *= g0; o[i][2] *= g1; o[i][3] *= g1;
                            }
                            m0 = n0;
                            m1 = n1;
                        }
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                s[t][e] = exp2_ftz(s[t][e] - f0);
                                s[t][2 + e] = exp2_ftz(s[t][2 + e] - f1);
                                l0 += s[t][e];
                                l1 += s[t][2 + e];
                            }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            pr[t][0] = pack2_bf16_cvt(s[2 * t][0], s[2 * t][1]);
                            pr[t][1] = pack2_bf16_cvt(s[2 * t][2], s[2 * t][3]);
                            pr[t][2] = pack2_bf16_cvt(s[2 * t + 1][0], s[2 * t + 1][1]);
                            pr[t][3] = pack2_bf16_cvt(s[2 * t + 1][2], s[2 * t + 1][3]);
                        }
                    }
                    wait_issued(1, block);
                    wait_full(1, block);
                    __syncwarp();
                    if (keys > 0) {
                        const uint32_t st = stage_at(1, block) + vkey * 128 + ((vc ^ (vkey & 7)) << 4);
                        auto values = [&](auto whole) {
                            // rows past the keys may hold anything, and 0 times NaN is NaN
                            auto keep = [&](int k) {
                                return (k < keys ? 0xffffu : 0u) | (k + 1 < keys ? 0xffff0000u : 0u);
                            };
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                uint32_t b[4], d[4];
                                const uint32_t at = (st ^ ((i & 3) << 5)) + (i >> 2) * S::kHalf;
                                ldmatrix_x4_trans(b, at);
                                ldmatrix_x4_trans(d, at + 16 * 128);
                                if constexpr (!decltype(whole)::value) {
                                    b[0] &= keep(c2); b[1] &= keep(c2 + 8); b[2] &= keep(c2); b[3] &= keep(c2 + 8);
                                    d[0] &= keep(c2 + 16); d[1] &= keep(c2 + 24); d[2] &= keep(c2 + 16); d[3] &= keep(c2 + 24);
                                }
                                mma_16x8x16(o[2 * i], pr[0], b[0], b[1]);
                                mma_16x8x16(o[2 * i + 1], pr[0], b[2], b[3]);
                                mma_16x8x16(o[2 * i], pr[1], d[0], d[1]);
                                mma_16x8x16(o[2 * i + 1], pr[1], d[2], d[3]);
                            }
                        };
                        if (seen >= 32) {
                            values(PagedFlag<true>{});
                        } else {
                            if (seen < min(keys, 32)) {
                                paged_clear<D>(p, smem + S::kRing + slot_of(1, block) * S::kStage + kw * 128, max(seen, 0),
                                               min(keys, 32), min(keys, 32), lane, 32);
                                __syncwarp();
                            }
                            values(PagedFlag<false>{});
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_empty + 8 * slot_of(1, block));
                }
                // ---- join the warpgroup's four warps
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    l0 += __shfl_xor_sync(~0u, l0, d);
                    l1 += __shfl_xor_sync(~0u, l1, d);
                }
                float *scr = reinterpret_cast<float *>(smem + S::kQ + wg * S::kQTile);  // [4][16][D]
                float2 *wml = ml + 64 * wg;                                             // [4][16]
                // column of a row in the scratch: rows 8 floats apart in the banks
                auto col = [&](int row, int c) { return c ^ ((row & 7) << 3); };
                auto leave = [&](int row, float m, float l, int e) {
                    if (row >= x.rows) return;
                    const int at = (warp & 3) * 16 + row;
                    if (c2 == 0) wml[at] = make_float2(m, l);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2 *>(scr + at * D + col(row, 8 * i + c2)) = make_float2(o[i][e], o[i][e + 1]);
                };
                leave(r0, m0, l0, 0);
                leave(r0 + 8, m1, l1, 2);
                wg_bar();
                // (threads for 2, 4, 8 or 16 rows)
                const int bits = x.rows <= 2 ? 1 : x.rows <= 4 ? 2 : x.rows <= 8 ? 3 : 4, row = wtid & ((1 << bits) - 1);
                CFA_ROLLED for (int c = wtid >> bits; c < D / 4 && row < x.rows; c += 128 >> bits) {
                    float2 w[4];
                    float4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[k] = wml[k * 16 + row];
                        v[k] = *reinterpret_cast<const float4 *>(scr + (k * 16 + row) * D + col(row, 4 * c));
                    }
                    const float m = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
                    const float f = m == -INFINITY ? 0.f : m;
                    float l = 0.f;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float g = exp2_ftz(w[k].x - f);
                        l += g * w[k].y;
                        a.x += g * v[k].x; a.y += g * v[k].y; a.z += g * v[k].z; a.w += g * v[k].w;
                    }
                    if (final) {
                        const float inv = l > 0.f ? 1.f / l : 0.f;
                        *reinterpret_cast<uint2 *>(p.out + static_cast<size_t>(result_row(row)) * D + 4 * c) =
                            make_uint2(pack2_bf16(a.x * inv, a.y * inv), pack2_bf16(a.z * inv, a.w * inv));
                        if (c == 0) write_lse(row, m, l);
                    } else {
                        *reinterpret_cast<float4 *>(rec_o + (static_cast<size_t>(c) * rec_stride + row) * 4) = a;
                        if (c == 0) rec_ml[row] = make_float2(m, l);
                    }
                }
                piece_done();
                continue;
            }

            // ---- tcgen05
            const bool split = x.rows <= 128;
            if (tid < x.rows) row_at[tid] = find_row(x, tid);
            meet();  // the scratch and the query tiles are free
            // asynchronous copies: all of them on their way before the first has landed
#pragma unroll 4
            for (int i = tid; i < (split ? 128 : 256) * (D / 8); i += kComputeThreads) {
                const int row = i / (D / 8), c = i % (D / 8);
                uint8_t *dst = smem + S::kQ + (row >> 7) * S::kQTile + (c >> 3) * S::kHalf + (row & 127) * 128 +
                               (((c & 7) ^ (row & 7)) << 4);
                if (row < x.rows) cp_async_16(smem_addr(dst), paged_query<D>(p, row_at[row], x.h) + 8 * c);
                else *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            tcgen05_fence_before();
            mbar_arrive(bar_q);

            const int step = split ? 2 : 1, first_block = split ? wg : 0;
            const int row = (split ? 0 : 128 * wg) + 32 * (warp & 3) + lane;
            const bool live = row < x.rows;
            const bool warp_live = (row & ~31) < x.rows;
            const int see = x.req < 0 ? 0 : paged_visible(x.r, (x.row0 + min(row, x.rows - 1)) / shape.by_G);
            const int all_see = paged_visible(x.r, x.row0 / shape.by_G);  // what the first row sees, every row does
            const uint32_t t_s = tmem + lanes + 128 * wg, t_o = tmem + lanes + 256 + D * wg;
            const uint32_t bs = bar_s + 16 * wg, bp = bar_p + 16 * wg;
            float m = -INFINITY, l = 0.f;
            bool begun = false;
            CFA_ROLLED for (int j = first_block; j < nb; j += step, ++scored) {
                int key0;
                const int keys = block_keys(x, x.b0 + j, &key0);
                const bool own = x.b0 + j >= x.prefix_blocks;
                const int lim = own ? min(keys, see - key0) : keys;
                const int some = own ? max(0, all_see - key0) : kPagedKeys;  // keys from here on some rows do not see
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(bs + 8 * h, scored & 1, kSiteSoftmaxExchange);
                    __syncwarp();
                    tcgen05_fence_after();
                    if (h == 0 && (keys < kPagedKeys || some < keys)) {
                        // (not before these scores: with them the stage's last values are known to
                        // have landed, and its barrier's parity to speak of these)
                        wait_full(1, n + j);
                        paged_clear<D>(p, smem + S::kRing + slot_of(1, n + j) * S::kStage, min(some, max(keys, 0)),
                                       max(keys, 0), kPagedKeys, wtid, 128);
                        fence_proxy_async_smem();
                    }
                    if (warp_live) {
                        uint32_t s[64];
                        tmem_ld_x32(t_s + 64 * h, s);
                        tmem_ld_x32(t_s + 64 * h + 32, s + 32);
                        tmem_wait_ld();
                        if (!__all_sync(~0u, lim - 64 * h >= 64)) {
#pragma unroll
                            for (int c = 0; c < 64; ++c) s[c] = c < lim - 64 * h ? s[c] : 0xff800000u;
                        }
                        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 64; c += 2)
                            a[(c >> 1) & 3] = fmaxf(fmaxf(a[(c >> 1) & 3], __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
                        const float top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * p.scale_log2;
                        if (__any_sync(~0u, top > m + 8.f)) {
                            // rescale to the new maximum (m = -inf: nothing is there yet)
                            const float mn = fmaxf(m, top);
                            const float g = m == mn ? 1.f : exp2_ftz(m - mn);
                            m = mn;
                            l *= g;
                            if (begun) {
                                // the other half's signal says that the last values' product is done
                                wait(bs + 8 * (h ^ 1), (scored + h) & 1, kSiteSoftmaxExchange);
                                __syncwarp();
                                tcgen05_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D; c += 32) {
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
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 y = unpair_f32(fma_f32x2(
                                    pair_f32(__uint_as_float(s[32 * c + 2 * e]), __uint_as_float(s[32 * c + 2 * e + 1])),
                                    scale2, f2));
                                const float x0 = exp2_ftz(y.x), x1 = exp2_ftz(y.y);
                                sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(x0, x1));
                                w[e] = pack2_bf16_cvt(x0, x1);
                            }
                            tmem_st_x16(t_s + 64 * h + 16 * c, w);
                        }
                        const float2 both_sums = unpair_f32(add_f32x2(sum[0], sum[1]));
                        l += both_sums.x + both_sums.y;
                        tmem_wait_st();
                    }
                    begun = true;
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bp + 8 * h);
                }
            }
            if (begun) {
                wait(bs, scored & 1, kSiteKvExchange);
                wait(bs + 8, scored & 1, kSiteKvExchange);
                ++scored;
            }
            __syncwarp();
            tcgen05_fence_after();
            // ---- the tile's results, or its record
            float mb = -INFINITY, lb = 0.f, ga = 1.f, gb = 0.f;
            // the other half's outputs
            auto at = [&](int c) { return smem + S::kQ + (row & 127) * (4 * D) + ((c ^ (row & 7)) << 4); };
            if (split) {
                meet();  // no product reads the query tiles any more
                if (wg == 1) {
                    ml[row] = make_float2(m, l);
                    if (warp_live && begun) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t v[32];
                            tmem_ld_x32(t_o + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(at(c / 4 + e)) =
                                    make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                        }
                    }
                }
                meet();
                if (wg == 0) {
                    mb = ml[row].x;
                    lb = ml[row].y;
                    const float mn = fmaxf(m, mb), f = mn == -INFINITY ? 0.f : mn;
                    ga = exp2_ftz(m - f);
                    gb = exp2_ftz(mb - f);
                    m = mn;
                    l = ga * l + gb * lb;
                }
            }
            if (warp_live && !(split && wg == 1)) {
                const float inv = !final ? 1.f : l > 0.f ? 1.f / l : 0.f;
                const size_t out_row = live ? static_cast<size_t>(result_row(row)) * D : 0;
                if (live) {
                    if (final) write_lse(row, m, l);
                    else rec_ml[row] = make_float2(m, l);
                }
                const bool both = split && nb > 1;  // the other half has seen keys
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t v[32];
                    tmem_ld_x32(t_o + c, v);
                    tmem_wait_ld();
                    if (!live) continue;
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]) * ga;
                    if (both) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 b = *reinterpret_cast<const float4 *>(at(c / 4 + e));
                            f[4 * e] += gb * b.x; f[4 * e + 1] += gb * b.y;
                            f[4 * e + 2] += gb * b.z; f[4 * e + 3] += gb * b.w;
                        }
                    }
                    if (final) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4 *>(p.out + out_row + c + 8 * e) =
                                make_uint4(pack2_bf16(f[8 * e] * inv, f[8 * e + 1] * inv),
                                           pack2_bf16(f[8 * e + 2] * inv, f[8 * e + 3] * inv),
                                           pack2_bf16(f[8 * e + 4] * inv, f[8 * e + 5] * inv),
                                           pack2_bf16(f[8 * e + 6] * inv, f[8 * e + 7] * inv));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(rec_o + (static_cast<size_t>(c / 4 + e) * rec_stride + row) * 4) =
                                make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
            }
            tcgen05_fence_before();
            meet();  // the scratch and the query tiles are free again
            piece_done();
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    if (warp == kComputeWarps) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the records, a warp for 32 rows of one key head (a lane a row) and CH of
// the row's 16-byte chunks: the shared rows (the prefix's pieces, then the
// request's own) a chunk at a time, then the tiles of requests that are alone and
// that a run's end cut, four at a time. The prefix's pieces are taken in the order of
// the runs, several at a time, then the request's own, so that their loads, maxima and
// sums among them, are on their way together with the row's: the kernel is a chain of
// two loads (the plan, then rows and records), and what counts is that nothing else waits
// in between. 3 to 5 us behind the attention at up to 2048 shared rows; 11 us (40 MB of
// records) behind the 151 cut tiles of 8 prompt chunks. Four blocks an SM, of 64
// registers a thread, were no faster than three.
template <int CH>
struct PagedMerge {
    float m = -INFINITY, l = 0.f;
    float4 a[CH];
    __device__ __forceinline__ PagedMerge() {
#pragma unroll
        for (int k = 0; k < CH; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // One piece's chunks with weight 2^(s.x - f).
    __device__ __forceinline__ void fold(float2 s, const float4 *v, float f) {
        const float g = exp2_ftz(s.x - f);
        l += g * s.y;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            a[k].x += g * v[k].x; a[k].y += g * v[k].y; a[k].z += g * v[k].z; a[k].w += g * v[k].w;
        }
    }
    // Takes the maximum on to `top`; returns what weights refer to.
    __device__ __forceinline__ float raise(float top) {
        const float f = top == -INFINITY ? 0.f : top, g = exp2_ftz(m - f);
        m = top;
        l *= g;
#pragma unroll
        for (int k = 0; k < CH; ++k) a[k].x *= g, a[k].y *= g, a[k].z *= g, a[k].w *= g;
        return f;
    }
    // n pieces, the first of a run each: their maxima and sums at s, their chunks at o, `rows`
    // rows a chunk; N at a time.
    template <int D, int N>
    __device__ __forceinline__ void add(const float2 *s, const float4 *o, int rows, int n) {
        constexpr int kRun = 2 * kPagedTile;  // record rows of a run
        CFA_ROLLED for (; n > 0; n -= N, s += N * kRun, o += static_cast<size_t>(N) * kRun * (D / 4)) {
            float2 t[N];
            float4 v[N][CH];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                t[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < CH; ++k) v[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    t[i] = __ldcg(s + i * kRun);
#pragma unroll
                    for (int k = 0; k < CH; ++k) v[i][k] = __ldcg(o + i * kRun * (D / 4) + k * rows);
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < N; ++i) top = fmaxf(top, t[i].x);
            const float f = raise(top);
#pragma unroll
            for (int i = 0; i < N; ++i) fold(t[i], v[i], f);
        }
    }
    template <int D>
    __device__ __forceinline__ void write(const PagedAttnParams &p, int out_row, int chunk) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k)
            *reinterpret_cast<uint2 *>(p.out + static_cast<size_t>(out_row) * D + 4 * (chunk + k)) =
                make_uint2(pack2_bf16_cvt(a[k].x * inv, a[k].y * inv), pack2_bf16_cvt(a[k].z * inv, a[k].w * inv));
        if (p.lse && chunk == 0) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
    }
    // Four chunks of each lane's row (out_row < 0: none), by the whole warp: two lanes write one
    // row's 32 bytes together, then the other's. A lane's own pieces of 8 bytes, each a
    // transaction of its own, took 1.2 us longer for 151 tiles of 256 rows.
    template <int D>
    __device__ __forceinline__ void write_pairs(const PagedAttnParams &p, int out_row, int chunk) {
        static_assert(CH == 4, "32 bytes");
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const bool odd = threadIdx.x & 1;
        uint32_t w[8], other[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[2 * k] = pack2_bf16_cvt(a[k].x * inv, a[k].y * inv);
            w[2 * k + 1] = pack2_bf16_cvt(a[k].z * inv, a[k].w * inv);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) other[k] = __shfl_xor_sync(~0u, odd ? w[k] : w[4 + k], 1);
        const int other_row = __shfl_xor_sync(~0u, out_row, 1);
        const int even_row = odd ? other_row : out_row, odd_row = odd ? out_row : other_row;
        uint16_t *out = p.out + 4 * chunk + (odd ? 8 : 0);
        if (even_row >= 0)
            *reinterpret_cast<uint4 *>(out + static_cast<size_t>(even_row) * D) =
                odd ? make_uint4(other[0], other[1], other[2], other[3]) : make_uint4(w[0], w[1], w[2], w[3]);
        if (odd_row >= 0)
            *reinterpret_cast<uint4 *>(out + static_cast<size_t>(odd_row) * D) =
                odd ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(other[0], other[1], other[2], other[3]);
        if (p.lse && chunk == 0 && out_row >= 0) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
    }
};

// Adds the values that are not finite to the rows that see them, where paged_clear has met one (rows
// that have them already do not change). The last block does it, when all rows are written: a
// thread goes through a request's new tokens with 8 dims of a key head and holds what they
// have seen so far. Rare, so it need only end in time: a load a token.
template <int D>
__device__ __noinline__ void paged_add_odd(const PagedAttnParams &p) {
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomic_add_acq_rel_gpu(p.odd + 1, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    if (threadIdx.x < 2) p.odd[threadIdx.x] = 0;
    const int G = p.shape.G;
    for (int task = threadIdx.x; task < p.B * p.n_kv * (D / 8); task += kPagedMergeThreads) {
        const int c = task % (D / 8), b = task / (D / 8) / p.n_kv, h = task / (D / 8) - b * p.n_kv;
        const int tok0 = p.cu[b], n = p.cu[b + 1] - tok0, len = p.lens[b];
        if (len < 0 || len > static_cast<long long>(p.width) * p.page_size) continue;
        bool some = false;
        float seen[8] = {};
        // token i is the first that sees key len - n + i (the first token's keys all see)
        for (int i = max(1, n - len); i < n; ++i) {
            const int key = len - n + i, pg = key / p.by_page;
            const int id = p.tables[static_cast<size_t>(b) * p.width + pg];
            if (id >= 0 && id < p.n_pages) {
                const size_t row = static_cast<size_t>(id * p.n_kv + h) * p.page_size + key - pg * p.page_size;
                float v[8];
                unpack8_bf16(*reinterpret_cast<const uint4 *>(p.v_pages + row * D + 8 * c), v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(fabsf(v[e]) < INFINITY)) seen[e] += v[e], some = true;
            }
            if (!some) continue;
            for (int g = 0; g < G; ++g) {
                uint4 *at = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(tok0 + i) * p.n_heads + h * G + g) * D + 8 * c);
                float y[8];
                unpack8_bf16(*at, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = seen[e] == 0.f ? y[e] : y[e] + seen[e];
                *at = make_uint4(pack2_bf16_cvt(y[0], y[1]), pack2_bf16_cvt(y[2], y[3]), pack2_bf16_cvt(y[4], y[5]),
                                 pack2_bf16_cvt(y[6], y[7]));
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kPagedMergeThreads, 3)
paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
    __shared__ int cuts[kPagedMaxGrid], cut_warps[kPagedMergeThreads / 32];
    constexpr int C = D / 4;  // chunks of a row
    const int tid = threadIdx.x, lane = tid & 31;
    const PagedShape &shape = p.shape;
    const float4 *rec_o = reinterpret_cast<const float4 *>(p.rec_o);
    grid_dependency_wait();
    const PagedPlan plan = *reinterpret_cast<const PagedPlan *>(p.plan_ws);
    const PagedCut *cut_of = reinterpret_cast<const PagedCut *>(p.plan_ws + kPagedPlanInts);
    const PagedRow *row_of = reinterpret_cast<const PagedRow *>(p.plan_ws + kPagedPlanInts + 8 * shape.grid);
    const unsigned odd = __ldcg(p.odd);
    if (!plan.valid) return;
    const int shared_tasks = (plan.shared_rows + 31) / 32 * p.n_kv * C;
    const int warps = static_cast<int>(gridDim.x) * (kPagedMergeThreads / 32);
    const int first = static_cast<int>(blockIdx.x) * (kPagedMergeThreads / 32) + (tid >> 5);
    CFA_ROLLED for (int task = first; task < shared_tasks; task += warps) {
        // chunks of a row group and key head lie together, so that its warps share its lines
        const int chunk = task % C, rest = task / C;
        const int group = rest / shape.by_nkv, h = rest - group * p.n_kv, r = group * 32 + lane;
        if (r >= plan.shared_rows) continue;
        const PagedRow d = row_of[r];
        // the records of its first pieces, wherever those ran
        const long long pre_rec = paged_first_record(shape, plan, false, h), own_rec = paged_first_record(shape, plan, true, h);
        const int at = chunk * plan.shared_rows + r;
        const float2 pre_ml = __ldcg(p.rec_ml + pre_rec + r), own_ml = __ldcg(p.rec_ml + own_rec + r);
        const float4 pre = __ldcg(rec_o + pre_rec * C + at), own = __ldcg(rec_o + own_rec * C + at);
        PagedMerge<1> acc;
        if (plan.prefix_blocks > 0) {
            const int tile = r / kPagedTile, row0 = tile * kPagedTile, rows = paged_min(kPagedTile, plan.shared_rows - row0);
            const int item = plan.prefix_units / shape.by_nkv * h + tile * plan.full_units;
            const int c0 = item / plan.by_share;
            const int more = (item + (plan.prefix_blocks - 1) * paged_cost(rows)) / plan.by_share - c0;
            const long long rec = paged_run_record(shape, plan, true, c0 + 1);
            acc.fold(pre_ml, &pre, acc.raise(pre_ml.x));
            acc.template add<D, 4>(p.rec_ml + rec + r - row0, rec_o + rec * C + chunk * rows + r - row0, rows, more);
        }
        if (d.blocks > 0) {
            const int item = d.unit + h * d.head_units;
            const int d0 = item / plan.by_share;
            const int more = (item + (d.blocks - 1) * paged_cost(d.rows)) / plan.by_share - d0;
            if (plan.prefix_blocks == 0 && more == 0) continue;  // the piece wrote the result
            acc.fold(own_ml, &own, acc.raise(fmaxf(acc.m, own_ml.x)));
            if (more > 0) {
                const long long rec = paged_run_record(shape, plan, true, d0 + 1);
                acc.template add<D, 1>(p.rec_ml + rec + d.row, rec_o + rec * C + chunk * d.rows + d.row, d.rows, more);
            }
        }
        acc.template write<D>(p, d.out_row + h * shape.G, chunk);
    }
    if (plan.alone_tokens == 0) {
        if (odd) paged_add_odd<D>(p);
        return;
    }
    // the cut runs in order, the same list in every block
    static_assert(kPagedMaxGrid <= kPagedMergeThreads, "a thread looks at a run");
    const bool is_cut = tid < shape.grid && cut_of[tid].rows > 0;
    const unsigned in_warp = __ballot_sync(~0u, is_cut);
    if (lane == 0) cut_warps[tid >> 5] = __popc(in_warp);
    __syncthreads();
    int before = 0, n_cuts = 0;
    CFA_ROLLED for (int w = 0; w < kPagedMergeThreads / 32; ++w) {
        if (w < tid >> 5) before += cut_warps[w];
        n_cuts += cut_warps[w];
    }
    if (is_cut) cuts[before + __popc(in_warp & ((1u << lane) - 1))] = tid;
    __syncthreads();
    const int cut_tasks = n_cuts * (kPagedTile / 32) * (C / 4);
    CFA_ROLLED for (int task = first; task < cut_tasks; task += warps) {
        const int chunk = task % (C / 4) * 4, rest = task / (C / 4);
        const int run = cuts[rest / (kPagedTile / 32)], at = rest % (kPagedTile / 32) * 32 + lane;
        const PagedCut cut = cut_of[run];
        if (at - lane >= cut.rows) continue;
        const int row = min(at, cut.rows - 1), r = cut.row0 + row, i = r / shape.by_G;
        PagedMerge<4> acc;
        // the run's own piece and the next run's, then what further runs have
        long long rec = paged_run_record(shape, plan, true, run + 1);
        const long long recs[2] = {paged_run_record(shape, plan, false, run), rec};
        float2 t[2];
        float4 v[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            t[k] = __ldcg(p.rec_ml + recs[k] + row);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] = __ldcg(rec_o + recs[k] * C + (chunk + e) * cut.rows + row);
        }
        const float f = acc.raise(fmaxf(t[0].x, t[1].x));
        acc.fold(t[0], v[0], f);
        acc.fold(t[1], v[1], f);
        CFA_ROLLED for (int c = run + 2; c <= cut.last_run; ++c) {
            rec += 2 * kPagedTile;
            acc.template add<D, 1>(p.rec_ml + rec + row, rec_o + rec * C + chunk * cut.rows + row, cut.rows, 1);
        }
        acc.template write_pairs<D>(p, at < cut.rows ? (cut.tok0 + i) * p.n_heads + cut.h * shape.G + r - i * shape.G : -1, chunk);
    }
    if (odd) paged_add_odd<D>(p);
}

}  // namespace cfa
