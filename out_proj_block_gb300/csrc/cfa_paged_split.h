// cfa_paged_split.h -- how the attention over a shared prefix is cut into work
// for a fixed grid, from the requests' offsets and lengths. The same code runs
// in the kernels (which find the lengths in device memory) and on the host.
//
// A request's query rows are its tokens times the G heads of a key head, token
// major. A request with at most kPagedAloneRows rows shares: its rows join the
// shared rows, whose tiles of 256 go over the prefix together, and one more
// item goes over the request's own keys. A request with more rows fills tiles
// by itself: it is alone, and each of its tiles goes over the prefix's keys and
// its own in one item, with nothing to merge.
//
// An item is cut into blocks of 128 keys, its units; prefix and own keys never
// share a block. The units of all items, in a fixed order (shared prefix by
// key head and tile; then requests in order, by key head and tile), are dealt
// out to the grid's blocks in equal runs. A run's part of one item is a piece.
// A piece that is a whole item, and the only item of its rows, writes its
// result; every other piece leaves a record (max, sum and unnormalised output
// of its rows), which are merged in the order of the runs.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CFA_HD __host__ __device__ __forceinline__
#define CFA_ROLLED _Pragma("unroll 1")  // a loop that is not worth the instruction cache
#else
#define CFA_HD inline
#define CFA_ROLLED
#endif

namespace cfa {

constexpr int kPagedKeys = 128;       // keys of a block
constexpr int kPagedTile = 256;       // rows of a tile
constexpr int kPagedSmallRows = 16;   // rows that go through mma.sync
constexpr int kPagedAloneRows = 128;  // rows up to which a request shares the prefix's tiles

struct PagedShape {
    int G, nkv, prefix_len, grid;
};

// What one scan over the requests finds.
struct PagedPlan {
    int shared_rows;    // of one key head
    int prefix_blocks;  // blocks of the prefix
    int tiles;          // tiles of the shared rows
    int prefix_units;   // units of the shared prefix
    int units;          // of everything
    int share;          // units of one run
    int valid;
};

struct PagedRequest {
    int tok0, n, len;  // first token row, tokens, own keys
};

struct PagedPiece {
    int req;            // request, or -1: the shared rows over the prefix
    int h;              // key head
    int row0, rows;     // rows of the request (or the shared rows)
    int prefix_blocks;  // the item's blocks before its own keys
    int blocks;         // the item's blocks
    int own_limit;      // own keys that the last row sees
    int b0, b1;         // the piece: blocks [b0, b1) of the item
    int first_unit;     // the item's first unit
    PagedRequest r;
};

CFA_HD int paged_min(int a, int b) { return a < b ? a : b; }
CFA_HD int paged_max(int a, int b) { return a > b ? a : b; }
CFA_HD int paged_cdiv(int a, int b) { return (a + b - 1) / b; }

// Own keys that token i of a request sees.
CFA_HD int paged_visible(const PagedRequest &r, int i) {
    return paged_min(r.len, paged_max(0, r.len - r.n + i + 1));
}
CFA_HD bool paged_alone(const PagedShape &s, int n) {
    return static_cast<long long>(n) * s.G > kPagedAloneRows;
}
// Blocks of tile `tile` of a request that is alone; a tile whose rows see no key
// still has one block, which finds none.
CFA_HD int paged_alone_blocks(const PagedShape &s, const PagedRequest &r, int tile) {
    const int last = paged_min(r.n * s.G, (tile + 1) * kPagedTile) - 1;
    return paged_max(1, paged_cdiv(s.prefix_len, kPagedKeys) +
                            paged_cdiv(paged_visible(r, last / s.G), kPagedKeys));
}
// Units of a request's own items.
CFA_HD long long paged_request_units(const PagedShape &s, const PagedRequest &r) {
    if (r.n == 0) return 0;
    if (!paged_alone(s, r.n)) return static_cast<long long>(s.nkv) * paged_cdiv(r.len, kPagedKeys);
    long long u = 0;
    CFA_ROLLED for (int t = 0; t * kPagedTile < r.n * s.G; ++t) u += paged_alone_blocks(s, r, t);
    return u * s.nkv;
}

// The totals: `own_units` of all requests and `shared_tokens` of those that share.
CFA_HD PagedPlan paged_plan(const PagedShape &s, long long own_units, int shared_tokens, bool valid) {
    PagedPlan p;
    p.shared_rows = shared_tokens * s.G;
    p.prefix_blocks = paged_cdiv(s.prefix_len, kPagedKeys);
    p.tiles = paged_cdiv(p.shared_rows, kPagedTile);
    const long long pu = static_cast<long long>(s.nkv) * p.tiles * p.prefix_blocks;
    const long long all = pu + own_units;
    p.valid = valid && all < (1ll << 31) - s.grid;
    p.prefix_units = p.valid ? static_cast<int>(pu) : 0;
    p.units = p.valid ? static_cast<int>(all) : 0;
    p.share = paged_max(1, paged_cdiv(p.units, s.grid));
    return p;
}

// Index of the last entry of a[0..B] (ascending, a[0] = 0) that is at most x, below B:
// requests without units share their start with the next one and are passed over.
CFA_HD int paged_find(const int *a, int B, int x) {
    int lo = 0, hi = B;
    CFA_ROLLED while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// The piece of the run ending before unit `end` that starts at unit u. start[b]:
// units of the requests before b; get(b): request b.
template <typename Get>
CFA_HD PagedPiece paged_piece(const PagedShape &s, const PagedPlan &p, const int *start, int B, int u,
                              int end, Get get) {
    PagedPiece x;
    int rem;
    if (u < p.prefix_units) {
        const int item = u / p.prefix_blocks;
        x.req = -1;
        x.h = item / p.tiles;
        x.row0 = (item - x.h * p.tiles) * kPagedTile;
        x.rows = paged_min(kPagedTile, p.shared_rows - x.row0);
        x.prefix_blocks = x.blocks = p.prefix_blocks;
        x.own_limit = 0;
        x.r = PagedRequest{0, 0, 0};
        rem = u - item * p.prefix_blocks;
    } else {
        x.req = paged_find(start, B, u - p.prefix_units);
        x.r = get(x.req);
        const int mine = u - p.prefix_units - start[x.req];
        const int per_head = (start[x.req + 1] - start[x.req]) / s.nkv;
        x.h = mine / per_head;
        rem = mine - x.h * per_head;
        if (!paged_alone(s, x.r.n)) {
            x.row0 = 0;
            x.rows = x.r.n * s.G;
            x.prefix_blocks = 0;
            x.blocks = per_head;
            x.own_limit = x.r.len;
        } else {
            int t = 0, n = paged_alone_blocks(s, x.r, 0);
            CFA_ROLLED while (rem >= n) {
                rem -= n;
                n = paged_alone_blocks(s, x.r, ++t);
            }
            x.row0 = t * kPagedTile;
            x.rows = paged_min(kPagedTile, x.r.n * s.G - x.row0);
            x.prefix_blocks = p.prefix_blocks;
            x.blocks = n;
            x.own_limit = paged_visible(x.r, (x.row0 + x.rows - 1) / s.G);
        }
    }
    x.first_unit = u - rem;
    x.b0 = rem;
    x.b1 = paged_min(x.blocks, rem + end - u);
    return x;
}

// Whether a request's item holds all the keys its rows see.
CFA_HD bool paged_sole(const PagedShape &s, const PagedPiece &x) {
    return x.req >= 0 && (s.prefix_len == 0 || paged_alone(s, x.r.n));
}
// Whether a piece writes its rows' results itself.
CFA_HD bool paged_final(const PagedShape &s, const PagedPiece &x) {
    return x.b0 == 0 && x.b1 == x.blocks && paged_sole(s, x);
}

// First record row of a piece of run c. Items that share have room for their rows at every
// run they meet: the rows of all the items before them plus a tile a run (so that neither the
// next item nor the next run reaches back). Tiles of requests that are alone are cut at most at
// a run's ends: two tiles a run, behind the others.
CFA_HD long long paged_shared_record(const PagedShape &s, const PagedPlan &p, int req, int h, int row0,
                                     int rows, int shared_tok0, int c) {
    const long long before = req < 0 ? static_cast<long long>(h) * p.shared_rows + row0
                                     : static_cast<long long>(s.nkv) * (p.shared_rows + static_cast<long long>(shared_tok0) * s.G) +
                                           static_cast<long long>(h) * rows;
    return before + static_cast<long long>(c) * kPagedTile;
}
CFA_HD long long paged_alone_record(const PagedShape &s, const PagedPlan &p, int b0, int c) {
    return 2ll * s.nkv * p.shared_rows + static_cast<long long>(s.grid) * kPagedTile +
           (2ll * c + (b0 > 0 ? 0 : 1)) * kPagedTile;
}
CFA_HD long long paged_record_rows(const PagedShape &s, long long shared_rows) {
    return 2 * s.nkv * shared_rows + 3ll * s.grid * kPagedTile;
}

}  // namespace cfa
