// cfa_latent.h -- launch parameters of the paged latent-cache kernels. Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

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
};

// ------------------------------------------------------- attention over rows

struct LatentAttnParams {
    const uint16_t *q;    // [T][H][576]
    const uint16_t *pages;
    const int *cu, *lens, *tables;
    uint16_t *out;        // [T][H][512]
    float *lse;           // [T][H] or null
    unsigned *status;
    int T, B, H, page_size, n_pages, width;
    float scale_log2;     // scale * log2(e)
    uint32_t timeout_ns;
};

// ------------------------------------------- attention over expanded keys and values

struct LatentExpandedParams {
    const uint16_t *q;       // rows of H * 192
    long long q_stride;
    const uint16_t *kv;      // rows of H * 256
    long long kv_stride;
    const uint16_t *k_rope;  // rows of 64
    long long k_rope_stride;
    const int *cu, *cu_k;
    uint16_t *out;           // [T][H][128]
    float *lse;              // [T][H] or null
    unsigned *status;
    int T, S, B, H;
    float scale_log2;
    uint32_t timeout_ns;
};

}  // namespace cfa
