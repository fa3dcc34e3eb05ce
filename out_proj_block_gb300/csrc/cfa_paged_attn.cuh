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
// A load warp streams K and V through one ring of 128-key stages (TMA boxes of
// 64 dims with 128-byte swizzle, each inside one page); what the other warps do
// with a stage depends on how many query rows the piece has:
//   up to 16 rows   eight warps, 16 keys each, on mma.sync with a running max
//                   and sum per warp, joined in shared memory at the piece's
//                   end: the bytes of the keys bound it, and the 16-row
//                   instruction wastes least on a few rows
//   up to 128 rows  tcgen05, one tile of queries; even blocks of keys go to one
//                   warpgroup and odd ones to the other, each with its own
//                   scores and outputs in TMEM, so that one's softmax runs
//                   under the other's products
//   up to 256 rows  tcgen05, two tiles of queries, one to a warpgroup, on the
//                   same keys
// On tcgen05: S = Q K^T (M = 128 rows, N = 128 keys), a thread per row takes its
// scores from TMEM, writes the weights back over them as bf16, and O += P V reads
// them from there. A row's maximum is followed lazily: O is rescaled only when
// it grew by more than 8 (a factor 2^8, far inside fp32), which is rare.
//
// Weights are rounded to bf16 for the product with V (tensor cores take both
// operands in one type; 2^-8 each, the size of the result's own rounding); their
// sum, the maxima, the outputs and the records are fp32.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "cfa_device.cuh"
#include "cfa_paged.h"
#include "cfa_paged_split.h"
#include "cfa_tile.cuh"

namespace cfa {

// D[tmem] (+)= A[tmem] . B[smem]: A's row r in lane r, two bf16 a column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 lanes; valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                   "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
                   "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                    "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                    "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(n) : "memory");
}

// Shared memory of the attention kernel for head_dim D.
template <int D>
struct PagedSmem {
    static constexpr int kStage = kPagedKeys * D * 2;           // one block of K or V
    static constexpr int kHalf = kPagedKeys * 128;              // its 64-dim column halves
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kQTile = 128 * D * 2;
    static constexpr int kQ = 0;                                // two query tiles; scratch otherwise
    static constexpr int kRing = 2 * kQTile;
    static constexpr int kRow = kRing + kStages * kStage;       // int2 [256]: token, output row
    static constexpr int kMl = kRow + 256 * 8;                  // float2 [128]: max and sum
    static constexpr int kBars = kMl + 128 * 8;
    static constexpr int kMisc = kBars + 32 * 8;                // flags, TMEM address, scan sums
    static constexpr int kArrays = kMisc + 512;                 // start, stok: int [2][B + 1]
    static int bytes(int B) { return kArrays + 8 * (B + 1) + 1024; }
};

__device__ __forceinline__ PagedRequest paged_request(const PagedAttnParams &p, int b) {
    const int c0 = __ldcg(p.cu + b), c1 = __ldcg(p.cu + b + 1), len = __ldcg(p.lens + b);
    const bool ok = len >= 0 && len <= static_cast<long long>(p.width) * p.page_size;
    return PagedRequest{c0, c1 - c0, ok ? len : 0};
}

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
    const uint32_t bar_full = base + S::kBars, bar_empty = bar_full + 8 * NS;
    const uint32_t bar_q = bar_empty + 8 * NS, bar_s = bar_q + 8, bar_p = bar_s + 16, bar_o = bar_p + 16,
                   bar_drain = bar_o + 16;
    int *misc = reinterpret_cast<int *>(smem + S::kMisc);
    volatile int *timed_out = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);
    int *start = reinterpret_cast<int *>(smem + S::kArrays), *stok = start + p.B + 1;
    int2 *row_at = reinterpret_cast<int2 *>(smem + S::kRow);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kMl);

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, kComputeWarps);
        }
        mbar_init(bar_q, kComputeThreads);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar_s + 8 * w, 1);
            mbar_init(bar_p + 8 * w, 128);
            mbar_init(bar_o + 8 * w, 1);
        }
        mbar_init(bar_drain, 1);
        *timed_out = 0;
        fence_mbar_init();
    }
    if (warp == kComputeWarps) tmem_alloc(smem_addr(tmem_slot), 512);
    tcgen05_fence_before();
    grid_dependency_wait();

    // ---- every block scans the requests
    const PagedShape shape{p.n_heads / p.n_kv, p.n_kv, p.prefix_len, static_cast<int>(gridDim.x)};
    const int B = p.B, G = shape.G;
    PagedPlan plan;
    {
        long long *sums_u = reinterpret_cast<long long *>(misc + 8);  // [10]
        int *sums_t = misc + 32;                                      // [10]
        const int per = (B + kPagedThreads - 1) / kPagedThreads;
        const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
        long long u = 0;
        int tk = 0, bad = 0, flags = 0;
        for (int b = b0; b < b1; ++b) {
            PagedRequest r = paged_request(p, b);
            if (r.tok0 < 0 || r.n < 0 || r.n > p.T || r.tok0 > p.T - r.n) {
                bad = 1;
                r.n = 0;
            }
            if (r.len != __ldcg(p.lens + b)) flags = 1;
            const long long ub = paged_request_units(shape, r);
            const int tb = paged_alone(shape, r.n) ? 0 : r.n;
            u += ub;
            tk += tb;
        }
        long long su = u;
        int st = tk;
        for (int o = 1; o < 32; o <<= 1) {
            const long long a = __shfl_up_sync(~0u, su, o);
            const int c = __shfl_up_sync(~0u, st, o);
            if (lane >= o) su += a, st += c;
        }
        if (lane == 31) sums_u[warp] = su, sums_t[warp] = st;
        bad = __syncthreads_or(bad);
        flags = __syncthreads_or(flags);
        long long all_u = 0;
        int all_t = 0;
        su -= u;
        st -= tk;
        for (int w = 0; w < kPagedThreads / 32; ++w) {
            if (w < warp) su += sums_u[w], st += sums_t[w];
            all_u += sums_u[w];
            all_t += sums_t[w];
        }
        for (int b = b0; b < b1; ++b) {
            PagedRequest r = paged_request(p, b);
            if (bad) r.n = 0;
            start[b] = static_cast<int>(su);
            stok[b] = st;
            su += paged_request_units(shape, r);
            st += paged_alone(shape, r.n) ? 0 : r.n;
        }
        if (tid == 0) start[B] = static_cast<int>(all_u), stok[B] = all_t;
        plan = paged_plan(shape, all_u, all_t, !bad);
        tcgen05_fence_after();
        __syncthreads();
        if (blockIdx.x == 0) {
            int *ws = p.plan_ws;
            if (tid == 0) {
                *reinterpret_cast<PagedPlan *>(ws) = plan;
                if (!plan.valid || flags) atomicOr(p.status, kStatusBadLengthBit);
            }
            for (int i = tid; i < 2 * (B + 1); i += kPagedThreads) ws[kPagedPlanInts + i] = start[i];
        }
    }
    grid_dependents_launch();
    const uint32_t tmem = *tmem_slot;
    const int run = blockIdx.x;
    const long long first = static_cast<long long>(run) * plan.share;
    const int u0 = static_cast<int>(min(first, static_cast<long long>(plan.units)));
    const int u1 = static_cast<int>(min(first + plan.share, static_cast<long long>(plan.units)));
    auto get = [&](int b) { return paged_request(p, b); };
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned site) {
        mbar_wait_bounded<false>(bar, parity, p.timeout_ns, timed_out, p.status, site);
    };
    // Stage `n` of the ring's life: slot n % NS, in the n / NS-th pass.
    auto slot_of = [&](uint32_t n) { return n % NS; };
    auto wait_full = [&](uint32_t n) { wait(bar_full + 8 * slot_of(n), (n / NS) & 1, kSiteStageFull); };
    // Keys of block j of a piece's item: where they lie and how many there are.
    auto block_keys = [&](const PagedPiece &x, int j, int *key0) {
        const bool pre = j < x.prefix_blocks;
        *key0 = (pre ? j : j - x.prefix_blocks) * kPagedKeys;
        return min(kPagedKeys, (pre ? p.prefix_len : x.own_limit) - *key0);
    };
    // V_i's place among a piece's 2 n stages (K0 V0 K1 V1 ..., or with the keys of two
    // blocks ahead K0 K1 V0 K2 V1 ... V_n-1).
    auto v_place = [&](bool split, int n, int i) { return !split ? 2 * i + 1 : i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

    if (warp == kComputeWarps) {
        // -------------------------------------------------------------- load warp
        uint32_t n = 0;
        const int box = p.box_rows;
        const int all_rows = p.n_pages * p.n_kv * p.page_size;
        for (int u = u0; u < u1;) {
            const PagedPiece x = paged_piece(shape, plan, start, B, u, u1, get);
            const int nb = x.b1 - x.b0;
            const bool split = x.rows > kPagedSmallRows && x.rows <= 128;
            for (int s = 0; s < 2 * nb; ++s, ++n) {
                bool is_v = s & 1;
                int i = s >> 1;
                if (split && s > 0) {
                    is_v = s == 2 * nb - 1 || (s > 1 && !(s & 1));
                    i = s == 2 * nb - 1 ? nb - 1 : is_v ? (s - 2) >> 1 : (s + 1) >> 1;
                }
                int key0;
                const int j = x.b0 + i, keys = block_keys(x, j, &key0);
                const int *table = j < x.prefix_blocks ? p.prefix_table
                                                       : p.tables + static_cast<size_t>(x.req) * p.width;
                const int boxes = keys > 0 ? (keys + box - 1) / box : 0;
                int y = all_rows;  // outside: reads as zeros
                if (lane < boxes) {
                    const int key = key0 + lane * box, pg = key / p.page_size;
                    const int id = __ldcg(table + pg);
                    if (id >= 0 && id < p.n_pages)
                        y = (id * p.n_kv + x.h) * p.page_size + key - pg * p.page_size;
                    else
                        atomicOr(p.status, kStatusBadPageBit);
                }
                const uint32_t full = bar_full + 8 * slot_of(n);
                if (lane == 0) {
                    if (n >= NS) wait(bar_empty + 8 * slot_of(n), (n / NS - 1) & 1, kSiteStageEmpty);
                    mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * box * D * 2));
                }
                __syncwarp();
                if (lane < boxes) {
                    const uint32_t dst = ring + slot_of(n) * S::kStage + lane * box * 128;
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_2d(dst + h * S::kHalf, is_v ? &tm_v : &tm_k, 64 * h, y, full);
                }
            }
            u += nb;
        }
        if (lane == 0 && *timed_out) {
            // a wait gave up: the copies in flight land before the block ends
            const uint64_t t0 = global_timer_ns();
            for (uint32_t k = n > NS ? n - NS : 0; k < n; ++k)
                while (!mbar_try_wait(bar_full + 8 * slot_of(k), (k / NS) & 1) &&
                       global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
        }
        __syncwarp();
    } else if (warp == kComputeWarps + 1) {
        // --------------------------------------------------------------- MMA warp
        if (lane == 0) {
            const uint32_t idesc_s = umma_idesc_bf16(128, kPagedKeys, false, false);
            const uint32_t idesc_o = umma_idesc_bf16(128, D, false, true);
            uint32_t n = 0, pieces = 0, probs[2] = {0, 0};
            auto scores = [&](int w, uint32_t q, uint32_t stage) {
                const uint32_t k = ring + slot_of(stage) * S::kStage;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_bf16(tmem + 128 * w,
                              umma_smem_desc(q + (ks >> 2) * S::kHalf + (ks & 3) * 32, 16, 1024),
                              umma_smem_desc(k + (ks >> 2) * S::kHalf + (ks & 3) * 32, 16, 1024),
                              idesc_s, ks > 0);
                umma_commit(bar_s + 8 * w);
            };
            auto values = [&](int w, uint32_t stage, bool accumulate) {
                const uint32_t v = ring + slot_of(stage) * S::kStage;
#pragma unroll
                for (int ks = 0; ks < kPagedKeys / 16; ++ks)
                    umma_bf16_ts(tmem + 256 + D * w, tmem + 128 * w + 8 * ks,
                                 umma_smem_desc(v + ks * 2048, S::kHalf, 1024), idesc_o,
                                 accumulate || ks > 0);
            };
            auto probs_ready = [&](int w) {
                wait(bar_p + 8 * w, probs[w]++ & 1, kSiteSoftmaxExchange);
                tcgen05_fence_after();
            };
            auto keys_ready = [&](uint32_t stage) {
                wait_full(stage);
                tcgen05_fence_after();
            };
            auto release = [&](uint32_t stage) {  // once the MMAs issued so far have read it
                mbar_arrive_n(bar_empty + 8 * slot_of(stage), kComputeWarps - 1);
                umma_commit(bar_empty + 8 * slot_of(stage));
            };
            for (int u = u0; u < u1;) {
                const PagedPiece x = paged_piece(shape, plan, start, B, u, u1, get);
                const int nb = x.b1 - x.b0;
                u += nb;
                if (x.rows <= kPagedSmallRows) {
                    n += 2 * nb;
                    continue;
                }
                wait(bar_q, pieces++ & 1, kSiteQExchange);
                tcgen05_fence_after();
                const uint32_t q = base + S::kQ;
                if (x.rows > 128) {
                    keys_ready(n);
                    scores(0, q, n);
                    scores(1, q + S::kQTile, n);
                    release(n);
                    for (int j = 0; j < nb; ++j) {
                        const uint32_t v = n + 2 * j + 1, k = v + 1;
                        keys_ready(v);
                        probs_ready(0);
                        values(0, v, j > 0);
                        if (j + 1 < nb) {
                            keys_ready(k);
                            scores(0, q, k);
                        }
                        probs_ready(1);
                        values(1, v, j > 0);
                        release(v);
                        if (j + 1 < nb) {
                            scores(1, q + S::kQTile, k);
                            release(k);
                        }
                    }
                } else {
                    for (int j = 0; j < min(nb, 2); ++j) {
                        keys_ready(n + j);
                        scores(j, q, n + j);
                        release(n + j);
                    }
                    for (int j = 0; j < nb; ++j) {
                        const uint32_t v = n + v_place(true, nb, j);
                        keys_ready(v);
                        probs_ready(j & 1);
                        values(j & 1, v, j > 1);
                        release(v);
                        if (j + 2 < nb) {
                            keys_ready(v + 1);
                            scores(j & 1, q, v + 1);
                            release(v + 1);
                        }
                    }
                }
                umma_commit(bar_o);
                umma_commit(bar_o + 8);
                n += 2 * nb;
            }
            if (*timed_out) {  // a wait gave up: the products in flight end before the block does
                umma_commit(bar_drain);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar_drain, 0) &&
                       global_timer_ns() - t0 < kDrainTimeoutFactor * p.timeout_ns) {
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- compute warps
        const int wg = warp >> 2;
        uint32_t n = 0, scored = 0, done = 0;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lanes of this warp
        for (int u = u0; u < u1;) {
            const PagedPiece x = paged_piece(shape, plan, start, B, u, u1, get);
            const int nb = x.b1 - x.b0;
            u += nb;
            const bool final = paged_final(shape, x);
            const long long rec =
                x.req >= 0 && paged_alone(shape, x.r.n)
                    ? paged_alone_record(shape, plan, x.b0, run)
                    : paged_shared_record(shape, plan, x.req, x.h, x.row0, x.rows,
                                          x.req < 0 ? 0 : stok[x.req], run);
            float *rec_o = p.rec_o + rec * D;
            float2 *rec_ml = p.rec_ml + rec;
            // where each row's query and result lie
            if (tid < x.rows) {
                const int r = x.row0 + tid, i = r / G, g = r - i * G;
                int t = x.r.tok0 + i;
                if (x.req < 0) {
                    const int b = paged_find(stok, B, i);
                    t = __ldcg(p.cu + b) + i - stok[b];
                }
                row_at[tid] = make_int2(t, t * p.n_heads + x.h * G + g);
            }
            compute_bar<kComputeThreads>();
            auto query = [&](int row) {
                const int2 at = row_at[row];
                return p.q + at.x * p.q_stride + (at.y - at.x * p.n_heads) * D;
            };
            auto write_lse = [&](int row, float m, float l) {
                if (p.lse) p.lse[row_at[row].y] = (m + log2f(l)) * 0.69314718055994531f;
            };

            if (x.rows <= kPagedSmallRows) {
                // ---- mma.sync: this warp's 16 keys of every block
                const int r0 = lane >> 2, c2 = (lane & 3) * 2;
                uint32_t q[D / 16][4];
                {
                    const uint16_t *qa = r0 < x.rows ? query(r0) : nullptr;
                    const uint16_t *qb = r0 + 8 < x.rows ? query(r0 + 8) : nullptr;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        q[k][0] = qa ? *reinterpret_cast<const uint32_t *>(qa + 16 * k + c2) : 0u;
                        q[k][1] = qb ? *reinterpret_cast<const uint32_t *>(qb + 16 * k + c2) : 0u;
                        q[k][2] = qa ? *reinterpret_cast<const uint32_t *>(qa + 16 * k + 8 + c2) : 0u;
                        q[k][3] = qb ? *reinterpret_cast<const uint32_t *>(qb + 16 * k + 8 + c2) : 0u;
                    }
                }
                float o[D / 8][4];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
                float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
                // own keys that rows r0 and r0 + 8 see
                const int see0 = paged_visible(x.r, (x.row0 + r0) / G);
                const int see1 = paged_visible(x.r, (x.row0 + r0 + 8) / G);
                const uint32_t kkey = 16 * warp + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
                const uint32_t vkey = 16 * warp + (lane & 15), vc = lane >> 4;
                for (int j = 0; j < nb; ++j, n += 2) {
                    int key0;
                    const int keys = block_keys(x, x.b0 + j, &key0) - 16 * warp;
                    key0 += 16 * warp;
                    wait_full(n);
                    float s[2][4] = {};
                    if (keys > 0) {
                        const uint32_t st = ring + slot_of(n) * S::kStage + kkey * 128;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            uint32_t b[4];
                            const uint32_t c = 2 * k + kc;
                            ldmatrix_x4(b, st + (c >> 3) * S::kHalf + (((c & 7) ^ (kkey & 7)) << 4));
                            mma_16x8x16(s[0], q[k], b[0], b[1]);
                            mma_16x8x16(s[1], q[k], b[2], b[3]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_empty + 8 * slot_of(n));
                    uint32_t pr[4];
                    if (keys > 0) {
                        const bool own = x.b0 + j >= x.prefix_blocks;
                        const int lim0 = own ? min(keys, see0 - key0) : keys;
                        const int lim1 = own ? min(keys, see1 - key0) : keys;
                        float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
                        for (int t = 0; t < 2; ++t)
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
                            const float g0 = fast_exp2(m0 - f0), g1 = fast_exp2(m1 - f1);
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
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                s[t][e] = fast_exp2(s[t][e] - f0);
                                s[t][2 + e] = fast_exp2(s[t][2 + e] - f1);
                                l0 += s[t][e];
                                l1 += s[t][2 + e];
                            }
                        pr[0] = pack2_bf16(s[0][0], s[0][1]);
                        pr[1] = pack2_bf16(s[0][2], s[0][3]);
                        pr[2] = pack2_bf16(s[1][0], s[1][1]);
                        pr[3] = pack2_bf16(s[1][2], s[1][3]);
                    }
                    wait_full(n + 1);
                    if (keys > 0) {
                        // rows past the keys may hold anything, and 0 times NaN is NaN
                        auto keep = [&](int k) {
                            return (k < keys ? 0xffffu : 0u) | (k + 1 < keys ? 0xffff0000u : 0u);
                        };
                        const uint32_t keep0 = keep(c2), keep1 = keep(c2 + 8);
                        const uint32_t st = ring + slot_of(n + 1) * S::kStage + vkey * 128;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t b[4];
                            const uint32_t c = 2 * i + vc;
                            ldmatrix_x4_trans(b, st + (c >> 3) * S::kHalf + (((c & 7) ^ (vkey & 7)) << 4));
                            mma_16x8x16(o[2 * i], pr, b[0] & keep0, b[1] & keep1);
                            mma_16x8x16(o[2 * i + 1], pr, b[2] & keep0, b[3] & keep1);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_empty + 8 * slot_of(n + 1));
                }
                // ---- join the eight warps
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    l0 += __shfl_xor_sync(~0u, l0, d);
                    l1 += __shfl_xor_sync(~0u, l1, d);
                }
                float *scr = reinterpret_cast<float *>(smem + S::kQ);  // [8][16][D]
                if (r0 < x.rows) {
                    if (c2 == 0) ml[warp * 16 + r0] = make_float2(m0, l0);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2 *>(scr + (warp * 16 + r0) * D + 8 * i + c2) = make_float2(o[i][0], o[i][1]);
                }
                if (r0 + 8 < x.rows) {
                    if (c2 == 0) ml[warp * 16 + r0 + 8] = make_float2(m1, l1);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2 *>(scr + (warp * 16 + r0 + 8) * D + 8 * i + c2) = make_float2(o[i][2], o[i][3]);
                }
                compute_bar<kComputeThreads>();
                for (int i = tid; i < x.rows * (D / 4); i += kComputeThreads) {
                    // records are chunk major, results row major
                    const int row = final ? i / (D / 4) : i % x.rows, c = final ? i % (D / 4) : i / x.rows;
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < 8; ++w) m = fmaxf(m, ml[w * 16 + row].x);
                    const float f = m == -INFINITY ? 0.f : m;
                    float l = 0.f;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < 8; ++w) {
                        const float2 s = ml[w * 16 + row];
                        const float g = fast_exp2(s.x - f);
                        const float4 v = *reinterpret_cast<const float4 *>(scr + (w * 16 + row) * D + 4 * c);
                        l += g * s.y;
                        a.x += g * v.x; a.y += g * v.y; a.z += g * v.z; a.w += g * v.w;
                    }
                    if (final) {
                        const float inv = l > 0.f ? 1.f / l : 0.f;
                        *reinterpret_cast<uint2 *>(p.out + static_cast<size_t>(row_at[row].y) * D + 4 * c) =
                            make_uint2(pack2_bf16(a.x * inv, a.y * inv), pack2_bf16(a.z * inv, a.w * inv));
                        if (c == 0) write_lse(row, m, l);
                    } else {
                        *reinterpret_cast<float4 *>(rec_o + (static_cast<size_t>(c) * x.rows + row) * 4) = a;
                        if (c == 0) rec_ml[row] = make_float2(m, l);
                    }
                }
                compute_bar<kComputeThreads>();
                continue;
            }

            // ---- tcgen05
            const bool split = x.rows <= 128;
            for (int i = tid; i < (split ? 128 : 256) * (D / 8); i += kComputeThreads) {
                const int row = i / (D / 8), c = i % (D / 8);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (row < x.rows) v = *reinterpret_cast<const uint4 *>(query(row) + 8 * c);
                *reinterpret_cast<uint4 *>(smem + S::kQ + (row >> 7) * S::kQTile + (c >> 3) * S::kHalf +
                                           (row & 127) * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
            }
            fence_proxy_async_smem();
            tcgen05_fence_before();
            mbar_arrive(bar_q);

            const int row = (split ? 0 : 128 * wg) + 32 * (warp & 3) + lane;
            const bool live = row < x.rows;
            const bool warp_live = (row & ~31) < x.rows;
            const int see = x.req < 0 ? 0 : paged_visible(x.r, (x.row0 + min(row, x.rows - 1)) / G);
            const uint32_t t_s = tmem + lanes + 128 * wg, t_o = tmem + lanes + 256 + D * wg;
            float m = -INFINITY, l = 0.f;
            bool begun = false;
            for (int j = split ? wg : 0; j < nb; j += split ? 2 : 1) {
                int key0;
                const int keys = block_keys(x, x.b0 + j, &key0);
                const int lim = x.b0 + j < x.prefix_blocks ? keys : min(keys, see - key0);
                wait(bar_s + 8 * wg, scored++ & 1, kSiteKvExchange);
                tcgen05_fence_after();
                if (warp_live) {
                    uint32_t s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_x32(t_s + 32 * c, s + 32 * c);
                    tmem_wait_ld();
                    if (!__all_sync(~0u, lim >= kPagedKeys)) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) s[c] = c < lim ? s[c] : 0xff800000u;
                    }
                    float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[e] = fmaxf(a[e], fmaxf(__uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1])));
                    const float top = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * p.scale_log2;
                    if (__any_sync(~0u, top > m + 8.f || (m == -INFINITY && top > m))) {
                        // rescale to the new maximum (m = -inf: nothing is there yet)
                        const float mn = fmaxf(m, top);
                        const float g = m == mn ? 1.f : fast_exp2(m - mn);
                        m = mn;
                        l *= g;
                        if (begun) {
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
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x0 = fast_exp2(fmaf(__uint_as_float(s[32 * c + 2 * e]), p.scale_log2, f));
                            const float x1 = fast_exp2(fmaf(__uint_as_float(s[32 * c + 2 * e + 1]), p.scale_log2, f));
                            sum[e & 3] += x0 + x1;
                            w[e] = pack2_bf16(x0, x1);
                        }
                        tmem_st_x16(t_s + 16 * c, w);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                begun = true;
                if (keys < kPagedKeys) {
                    // rows past the keys may hold anything, and 0 times NaN is NaN
                    const uint32_t vn = n + v_place(split, nb, j);
                    wait_full(vn);
                    const int z = max(keys, 0);
                    for (int i = tid & 127; i < (kPagedKeys - z) * (D / 8); i += 128) {
                        const int r = z + i / (D / 8), c = i % (D / 8);
                        *reinterpret_cast<uint4 *>(smem + S::kRing + slot_of(vn) * S::kStage + (c >> 3) * S::kHalf +
                                                   r * 128 + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tcgen05_fence_before();
                mbar_arrive(bar_p + 8 * wg);
            }
            n += 2 * nb;
            wait(bar_o + 8 * wg, done++ & 1, kSiteKvExchange);
            tcgen05_fence_after();
            // ---- the tile's results, or its record
            float mb = -INFINITY, lb = 0.f, ga = 1.f, gb = 0.f;
            // the other half's outputs
            auto at = [&](int c) { return smem + S::kQ + (row & 127) * (4 * D) + ((c ^ (row & 7)) << 4); };
            if (split) {
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
                compute_bar<kComputeThreads>();
                if (wg == 0) {
                    mb = ml[row].x;
                    lb = ml[row].y;
                    const float mn = fmaxf(m, mb), f = mn == -INFINITY ? 0.f : mn;
                    ga = fast_exp2(m - f);
                    gb = fast_exp2(mb - f);
                    m = mn;
                    l = ga * l + gb * lb;
                }
            }
            if (warp_live && !(split && wg == 1)) {
                const float inv = !final ? 1.f : l > 0.f ? 1.f / l : 0.f;
                const size_t out_row = live ? static_cast<size_t>(row_at[row].y) * D : 0;
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
                            *reinterpret_cast<float4 *>(rec_o + (static_cast<size_t>(c / 4 + e) * x.rows + row) * 4) =
                                make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                }
            }
            tcgen05_fence_before();
            compute_bar<kComputeThreads>();  // row_at, ml and the query tiles are free again
        }
    }
    tcgen05_fence_before();
    __syncthreads();
    if (warp == kComputeWarps) {
        tcgen05_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the records: a block for 32 rows of one key head (a lane per row), its
// warps taking the row's 16-byte chunks in turn, pieces in the order of the
// runs. The first blocks take the shared rows (the prefix's pieces, then the
// request's own), the others the tiles of requests that are alone and were cut
// at the end of run (block / 8).
template <int D>
__global__ void __launch_bounds__(256)
paged_merge_kernel(const PagedAttnParams p, int grid, int shared_blocks) {
    extern __shared__ int sh[];
    constexpr int kPer = D / 32;  // chunks of a warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.B;
    grid_dependency_wait();
    const PagedPlan plan = *reinterpret_cast<const PagedPlan *>(p.plan_ws);
    const PagedShape shape{p.n_heads / p.n_kv, p.n_kv, p.prefix_len, grid};
    const int G = shape.G;
    const bool alone = static_cast<int>(blockIdx.x) >= shared_blocks;
    if (!plan.valid) return;
    if (!alone && static_cast<int>(blockIdx.x) / p.n_kv * 32 >= plan.shared_rows) return;
    const int run = (static_cast<int>(blockIdx.x) - shared_blocks) / 8;
    const long long end = static_cast<long long>(run + 1) * plan.share;
    if (alone && end >= plan.units) return;
    int *start = sh, *stok = sh + B + 1;
    float2 *mls = reinterpret_cast<float2 *>(sh + 2 * (B + 1));  // [pieces][32]
    for (int i = tid; i < 2 * (B + 1); i += 256) sh[i] = __ldcg(p.plan_ws + kPagedPlanInts + i);
    __syncthreads();

    // pieces c0..c1 that all the lanes have, at record rows rec(c) + row, then the lane's own
    int c0 = 0, c1 = -1, row = 0, rows = 1, h, out_row = 0;
    int d0 = 0, d1 = -1, own_row = 0, own_rows = 1;
    long long own_rec = 0;
    bool live, skip = false;
    PagedPiece x;
    if (alone) {
        x = paged_piece(shape, plan, start, B, static_cast<int>(end) - 1, static_cast<int>(end),
                        [&](int b) { return paged_request(p, b); });
        // cut here for the first time?
        if (x.req < 0 || !paged_alone(shape, x.r.n) || x.b1 == x.blocks ||
            x.first_unit < static_cast<long long>(run) * plan.share)
            return;
        c0 = run;
        c1 = (x.first_unit + x.blocks - 1) / plan.share;
        h = x.h;
        row = (static_cast<int>(blockIdx.x) - shared_blocks) % 8 * 32 + lane;
        rows = x.rows;
        live = row < rows;
        const int r = x.row0 + (live ? row : 0), i = r / G;
        out_row = (x.r.tok0 + i) * p.n_heads + h * G + r - i * G;
    } else {
        h = static_cast<int>(blockIdx.x) % p.n_kv;
        const int r = static_cast<int>(blockIdx.x) / p.n_kv * 32 + lane;
        live = r < plan.shared_rows;
        const int tile = r / kPagedTile;
        row = r % kPagedTile;
        rows = paged_min(kPagedTile, plan.shared_rows - tile * kPagedTile);
        if (plan.prefix_blocks > 0) {
            const int item = (h * plan.tiles + tile) * plan.prefix_blocks;
            c0 = item / plan.share;
            c1 = (item + plan.prefix_blocks - 1) / plan.share;
        }
        if (live) {
            const int b = paged_find(stok, B, r / G);
            const PagedRequest q = paged_request(p, b);
            own_rows = q.n * G;
            own_row = r - stok[b] * G;
            out_row = (q.tok0 + own_row / G) * p.n_heads + h * G + own_row % G;
            own_rec = paged_shared_record(shape, plan, b, h, 0, own_rows, stok[b], 0);
            const int nb = (start[b + 1] - start[b]) / p.n_kv;
            if (nb > 0) {
                const int item = plan.prefix_units + start[b] + h * nb;
                d0 = item / plan.share;
                d1 = (item + nb - 1) / plan.share;
            }
            skip = plan.prefix_blocks == 0 && d0 == d1;  // the piece wrote the result
        }
        x.row0 = tile * kPagedTile;
    }
    auto rec = [&](int c) {
        return alone ? paged_alone_record(shape, plan, c == c0 ? 0 : 1, c)
                     : paged_shared_record(shape, plan, -1, h, x.row0, rows, 0, c);
    };
    if (!__syncthreads_or(live && !skip)) return;
    for (int c = c0 + warp; c <= c1; c += 8)
        mls[(c - c0) * 32 + lane] = live ? __ldcg(p.rec_ml + rec(c) + row) : make_float2(-INFINITY, 0.f);
    __syncthreads();
    if (!live || skip) return;
    float m = -INFINITY, l = 0.f;
    for (int c = c0; c <= c1; ++c) m = fmaxf(m, mls[(c - c0) * 32 + lane].x);
    for (int c = d0; c <= d1; ++c)
        m = fmaxf(m, __ldcg(p.rec_ml + own_rec + static_cast<long long>(c) * kPagedTile + own_row).x);
    const float f = m == -INFINITY ? 0.f : m;
    float4 a[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 s, const float *o, int nrows, int r) {
        const float g = fast_exp2(s.x - f);
        l += g * s.y;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                o + (static_cast<size_t>(warp + 8 * k) * nrows + r) * 4));
            a[k].x += g * v.x; a[k].y += g * v.y; a[k].z += g * v.z; a[k].w += g * v.w;
        }
    };
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) add(mls[(c - c0) * 32 + lane], p.rec_o + rec(c) * D, rows, row);
    for (int c = d0; c <= d1; ++c) {
        const long long at = own_rec + static_cast<long long>(c) * kPagedTile;
        add(__ldcg(p.rec_ml + at + own_row), p.rec_o + at * D, own_rows, own_row);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        *reinterpret_cast<uint2 *>(p.out + static_cast<size_t>(out_row) * D + 4 * (warp + 8 * k)) =
            make_uint2(pack2_bf16(a[k].x * inv, a[k].y * inv), pack2_bf16(a[k].z * inv, a[k].w * inv));
    if (p.lse && warp == 0) p.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace cfa
