// cfa_paged.h -- launch parameters of the paged-cache kernels (block tables,
// rotary append, attention over a shared prefix). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "cfa_paged_split.h"

namespace cfa {

constexpr int kPagedMaxSeqs = 1024;         // requests per call
constexpr int kPagedMaxTokens = 1 << 17;    // new tokens per call
constexpr int kPagedMaxTableWidth = 1 << 18;

// ------------------------------------------------- block tables and slot maps

struct TablesParams {
    const int *lens;        // [B] cached tokens of each request
    const int *fresh;       // [B] new tokens of each request
    const int *free_pages;  // ids of free pages
    const int *pool;        // {entries of free_pages taken so far, entries there are}
    int *tables;            // [B][width] page ids; entries past the held pages are written
    int *lens_out;          // [B] lens + fresh (may be lens)
    int *pool_out;          // [2] (may be pool)
    int *cu;                // [B + 1] first token row of each request
    int *positions;         // [n_slots]
    int *slots;             // [n_slots]
    unsigned *ticket;       // arrivals of the grid's blocks; 0 between calls
    unsigned *status;
    int B, width, page_size, n_free, n_slots, base;
    int max_page;           // the last page whose slots an int holds
};

constexpr int kTablesThreads = 512;

// Free pages that a pool has left, by its two counters; -1 where one of them is below zero.
CFA_HD int paged_pool_left(int taken, int there, int n_free) {
    if (taken < 0 || there < 0) return -1;
    return paged_max(0, paged_min(there, n_free) - taken);
}

// ------------------------------------------------------------ rotary append

struct AppendParams {
    const uint16_t *q, *k, *v;  // [T] rows of heads; strides in elements
    long long q_stride, k_stride, v_stride;
    const int *positions, *slots;
    uint16_t *k_pages, *v_pages;  // [n_pages][n_kv][page_size][d]
    uint16_t *q_out;              // [T][n_heads][d]
    unsigned *status;
    int n_heads, n_kv, d, page_size;
    int n_rows;        // slots there are: n_pages * page_size
    int rd;            // rotated dims of a head; 0: none
    int interleaved;   // pairs (2i, 2i+1) instead of (i, i + rd/2)
    FastDiv by_units;  // 16-byte chunks (or pairs) of a head's q or k
    int heads_a_pass;  // heads that a block's threads take at a time
    FastDiv by_page;
    float magnitude;   // factor on cos and sin
    // turns per position of pair i as a fraction of 2^64
    unsigned long long turns[64];
};

constexpr int kAppendThreads = 128;  // at most (append_threads)

// ----------------------------------------- attention over a shared prefix

struct PagedAttnParams {
    const uint16_t *q;          // [T][n_heads][d], row stride q_stride elements
    long long q_stride;
    const uint16_t *v_pages;    // (the attention reads keys and values by tensor maps)
    const int *cu;              // [B + 1]
    const int *lens;            // [B]
    const int *tables;          // [B][width]
    const int *prefix_table;    // [ceil(prefix_len / page_size)]
    uint16_t *out;              // [T][n_heads][d]
    float *lse;                 // [T][n_heads] or null
    unsigned *status;
    unsigned *odd;              // {a value that is not finite was cleared, arrivals of the merge's
                                // blocks}; 0 between calls
    int *plan_ws;               // for the merge: the scan's totals, every run's PagedCut, every
                                // shared row's PagedRow
    float *rec_o;               // records: unnormalised outputs, a piece's rows in 16-byte chunks,
                                // [D / 4][rows][4]
    float2 *rec_ml;             // and each row's maximum (base 2) and sum
    int T, B, n_heads, n_kv, page_size, n_pages, width, prefix_len;
    PagedShape shape;
    FastDiv by_page;            // page_size
    int box_rows;               // cache rows of one TMA box
    int block_clocks;           // of paged_plan
    float scale_log2;           // scale * log2(e)
    uint32_t timeout_ns;
};

// 8 compute warps; two load warps, an address, a prep, two MMA warps, a merge-rows warp, one idle
constexpr int kPagedThreads = 512;
constexpr int kPagedPlanInts = 16;
static_assert(sizeof(PagedPlan) <= 4 * kPagedPlanInts, "the totals fit");
constexpr int kPagedMaxGrid = 256;    // blocks of the attention kernel, one per SM
constexpr int kPagedMergeThreads = 256;

// The tile of a request that is alone which a run's end cuts for the first time.
struct PagedCut {
    int rows;  // 0: none
    int row0, tok0, h, last_run, unused[3];
};

// A shared row.
struct alignas(16) PagedRow {
    int out_row;           // output row with key head 0
    int unit, head_units;  // first unit of its own keys' item, and units of a key head
    int blocks;            // the item's blocks
    int rows, row;         // rows of the item's tile, and this one among them
};

// (the merge finds them by 8 ints each)
static_assert(sizeof(PagedCut) == 32 && sizeof(PagedRow) == 32, "their places in plan_ws");

}  // namespace cfa
