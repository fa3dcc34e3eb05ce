// cfa_latent.h -- launch parameters of the paged latent-cache kernels. Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cfa_paged.h"
#include "cfa_paged_split.h"

namespace cfa {

constexpr int kLatC = 512;               // latent dims
constexpr int kLatR = 64;                // rotated dims
constexpr int kLatRow = kLatC + kLatR;   // a cache row
constexpr int kLatN = 128;               // unrotated query dims of a head
constexpr int kLatV = 128;               // value dims of a head
constexpr int kLatQ = kLatN + kLatR;     // a head's query
constexpr int kLatKv = kLatN + kLatV;    // a head's columns of W_kvb, an expanded key and value

// ------------------------------------------------------- norm, rotation, append

struct LatentAppendParams {
    const uint16_t *a;     // [T] rows of 576
    const uint16_t *g_kv;  // [512]
    const uint16_t *q;     // [T] rows of n_heads * 192
    long long a_stride, q_stride;
    const int *positions, *slots;
    uint16_t *pages;       // [n_pages * page_size][576]
    uint16_t *q_out;       // [T][n_heads][192]
    unsigned *status;
    int n_heads;
    int n_rows;            // slots there are
    int copy;              // q_out is not q: its unrotated dims are copied
    int rope;
    float eps, magnitude;
    unsigned long long turns[kLatR / 2];  // turns per position of pair i as a fraction of 2^64
};

constexpr int kLatAppendHeads = 32;     // heads of a block's queries
constexpr int kLatAppendThreads = 128;

// ------------------------------------------------------------ fold and unfold

struct LatentHeadsParams {
    const uint16_t *x;    // fold: queries, rows x_stride apart; unfold: [T][H][512]
    long long x_stride;
    const uint16_t *w;    // W_kvb
    uint16_t *y;          // fold: [T][H][576]; unfold: [T][H][128]
    int T, H;
    unsigned *status;
    uint32_t timeout_ns;
};

constexpr int kHeadsTokens = 16;       // of a block, where there are few
constexpr int kHeadsMmaThreads = 320;  // two warpgroups for the results, a load warp, one that issues the products

// ------------------------------------------------------- attention over rows

struct LatentAttnParams {
    const int *cu;        // [B + 1]
    const int *lens;      // [B]
    const int *tables;    // [B][width]
    const uint16_t *q, *pages;  // [T][H][576], rows of 576 (but for prefetches, read by tensor maps)
    uint16_t *out;        // [T][H][512]
    float *lse;           // [T][H] or null
    unsigned *status;
    float *rec_o;         // records, two a run: unnormalised outputs in 16-byte chunks [128][128 rows][4]
    float2 *rec_ml;       // and each row's maximum (base 2) and sum
    int4 *cuts;           // for the merge: the tile that each run's end cuts
    int T, B, H, page_size, n_pages, width;
    int runs;             // clusters of the attention kernel
    int box_rows;         // cache rows of one TMA box
    FastDiv by_H, by_page;
    float scale_log2;     // scale * log2(e)
    uint32_t timeout_ns;
};

// four compute warps; a load warp for queries and keys and one for values, a relay, one that
// issues the products (with a ninth warp an SM's quarter would hold three, of 168 registers a thread)
constexpr int kLatLoadWarp = 4, kLatMmaWarp = 7;
constexpr int kLatAttnThreads = 256;
constexpr int kLatMergeThreads = 256;
constexpr int kLatMaxRuns = 256;     // a thread of the merge looks at a run
static_assert(kLatMaxRuns <= kLatMergeThreads, "it does");

// ------------------------------------------- attention over expanded keys and values

struct LatentExpandedParams {
    const uint16_t *kv;      // rows of H * 256 (but for one rare pass, read by a tensor map)
    long long kv_stride;
    const int *cu, *cu_k;
    uint16_t *out;           // [T][H][128]
    float *lse;              // [T][H] or null
    unsigned *status;
    unsigned *odd;           // {a value that is not finite was cleared, arrivals of the merge's blocks}; 0 between calls
    unsigned char *odd_tiles;  // [kExpMarks] for every 256 tokens: it was in a tile that begins among them; 0 between calls
    float *rec_o;            // records of parts: unnormalised outputs in 16-byte chunks [32][512 rows][4]
    float2 *rec_ml;          // and each row's maximum (base 2) and sum
    int *rest;               // for the merge: how many tasks are split,
    int4 *splits;            // and of each of their two tiles its first row's place, rows, parts and first record
    int T, S, B, H;
    FastDiv by_H;
    float scale_log2;
    uint32_t timeout_ns;
};

// eight softmax warps; a load warp for keys and queries and one for values, one that issues the products, a relay
constexpr int kExpLoadWarp = 8, kExpMmaWarp = 10, kExpRelayWarp = 11;
constexpr int kExpThreads = 384;
constexpr int kExpMaxParts = 8;  // of a task of the last round
constexpr int kExpLeast = 3;     // least blocks of a part
constexpr int kExpTile = 256;    // tokens of a tile, half of them to either block of a cluster
constexpr int kExpMarks = kPagedMaxTokens / kExpTile;
constexpr int kLatWords = 4 + kExpMarks / 4;  // of a plan: status; odd, its arrivals, rest; odd_tiles

}  // namespace cfa
