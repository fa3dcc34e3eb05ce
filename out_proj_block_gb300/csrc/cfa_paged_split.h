// cfa_paged_split.h -- how the attention over a shared prefix is cut into work
// for a fixed grid, from the requests' offsets and lengths. The same code runs
// in the kernels (which find the lengths in device memory) and on the host.
//
// A request's query rows are its tokens times the G heads of a key head, token
// major. A request with at most kPagedAloneRows rows shares: its rows join the
// shared rows, whose tiles of 256 go over the prefix together, and further items
// go over the request's own keys (one for all its rows, or, up to kPagedNarrowRows,
// one for every 16: mma.sync takes 16 rows, and reads the keys again from L2
// cheaper than a tensor-core tile is set up for a few blocks). A request with more
// rows fills tiles by itself: it is alone, and each of its tiles goes over the
// prefix's keys and its own in one item, with nothing to merge.
//
// An item is cut into blocks of 128 keys; prefix and own keys never share a
// block. A block costs so many units by how many rows its item has, and an item some more
// behind its blocks (paged_plan says how many). The units of all items, in a fixed order
// (shared prefix by key head and tile; then requests in order, by key head and tile),
// are dealt out to the grid's blocks in equal runs; a block of keys goes to the run in
// which its first unit lies. A
// run's part of one item is a piece. A piece that is a whole item, and the only
// item of its rows, writes its result; every other piece leaves a record (max, sum
// and unnormalised output of its rows), which are merged in the order of the runs.
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
constexpr int kPagedNarrowRows = 64;  // rows up to which own keys go to tiles of 16
constexpr int kPagedMaxCost = 8;
constexpr int kPagedMaxUnits = (1 << 30) - 1;  // two of them added stay below 2^31

// Division of 0 <= n < 2^31 by a divisor that the host knows: n / d = (n mul) >> (32 + shift)
// with mul = 2^(31 + l) / d rounded up, l = ceil(log2 d), shift = l - 1; the rounding adds less
// than n / 2^(31 + l) < 1 / d to the quotient. An integer division takes some 30 instructions.
struct FastDiv {
    uint32_t d, mul;
    int shift;
    FastDiv() = default;
    CFA_HD explicit FastDiv(uint32_t divisor) : d(divisor), mul(0), shift(0) {
        int l = 0;
        CFA_ROLLED while ((1ull << l) < divisor) ++l;
        if (l > 0) {
            mul = static_cast<uint32_t>(((1ull << (31 + l)) + divisor - 1) / divisor);
            shift = l - 1;
        }
    }
};
CFA_HD int operator/(int n, const FastDiv &f) {
    if (f.d == 1) return n;
#ifdef __CUDA_ARCH__
    return static_cast<int>(__umulhi(static_cast<uint32_t>(n), f.mul) >> f.shift);
#else
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * f.mul >> 32) >> f.shift);
#endif
}

struct PagedShape {
    int G, nkv, prefix_len, grid;
    FastDiv by_G, by_nkv, by_grid;
    PagedShape() = default;
    PagedShape(int G_, int nkv_, int prefix, int grid_)
        : G(G_), nkv(nkv_), prefix_len(prefix), grid(grid_), by_G(static_cast<uint32_t>(G_)),
          by_nkv(static_cast<uint32_t>(nkv_)), by_grid(static_cast<uint32_t>(grid_)) {}
};

// What one scan over the requests finds.
struct PagedPlan {
    int by_bytes;       // the bytes of the keys bound the whole
    int item_units;     // units of an item whose paged_item_cost() is 1
    int shared_rows;    // of one key head
    int prefix_blocks;  // blocks of the prefix
    int tiles;          // tiles of the shared rows
    int full_units;     // units of a full tile's item
    int prefix_units;   // units of the shared prefix
    int units;          // of everything
    int share;          // units of one run
    int alone_tokens;   // tokens of the requests that are alone
    FastDiv by_share;   // (set by whoever divides by it)
    int valid;
};

struct PagedRequest {
    int tok0, n, len;  // first token row, tokens, own keys
};

// A request as the scan leaves it; entry B holds the totals.
struct alignas(16) PagedEntry {
    int unit;  // units of the requests before it, behind the shared prefix's
    int tok;   // tokens that share of the requests before it
    int tok0, len;
};
CFA_HD PagedRequest paged_request_at(const PagedEntry *e, int b) {
    return PagedRequest{e[b].tok0, e[b + 1].tok0 - e[b].tok0, e[b].len};
}
struct PagedPiece {
    int req;            // request, or -1: the shared rows over the prefix
    int h;              // key head
    int row0, rows;     // rows of the request (or the shared rows)
    int prefix_blocks;  // the item's blocks before its own keys
    int blocks;         // the item's blocks
    int own_limit;      // own keys that the last row sees
    int b0, b1;         // the piece: blocks [b0, b1) of the item
    int first_unit = 0; // the item's first unit
    int cost, units = 0;  // units of a block, and of the item
    int final;          // the piece writes its rows' results
    long long rec;      // else its record (paged_record)
    int rec_row, rec_stride;
    PagedRequest r;
};

CFA_HD int paged_min(int a, int b) { return a < b ? a : b; }
CFA_HD int paged_max(int a, int b) { return a > b ? a : b; }
CFA_HD int paged_cdiv(int a, int b) { return (a + b - 1) / b; }

// Clocks by 400 of a block of keys, and by 400 kPagedItemClocks of beginning and ending an
// item, as fitted to the runs' times of batches whose work bounds them (head_dim 128: 16 rows
// 1900 a block, with the other warpgroup's block beside it, and 2000 an item; tiles of
// 128 and 256 rows 1700 and 3200 a block, 12000 an item).
CFA_HD int paged_cost(int rows) { return rows <= kPagedAloneRows ? 5 : kPagedMaxCost; }
CFA_HD int paged_item_cost(int rows) { return rows <= kPagedSmallRows ? 1 : 6; }
constexpr int kPagedItemClocks = 5;
// Where the bytes of the keys bound the whole, an item costs next to nothing: what the warps
// do at its ends goes on under the loads.

// Own keys that token i of a request sees.
CFA_HD int paged_visible(const PagedRequest &r, int i) {
    return paged_min(r.len, paged_max(0, r.len - r.n + i + 1));
}
CFA_HD bool paged_alone(const PagedShape &s, int n) {
    return static_cast<long long>(n) * s.G > kPagedAloneRows;
}
// Rows of the tiles in which a request that shares goes over its own keys.
CFA_HD int paged_own_tile(int rows) { return rows <= kPagedNarrowRows ? kPagedSmallRows : kPagedAloneRows; }
// Blocks of tile `tile` of a request that is alone; a tile whose rows see no key
// still has one block, which finds none.
CFA_HD int paged_alone_blocks(const PagedShape &s, const PagedRequest &r, int tile) {
    const int last = paged_min(r.n * s.G, (tile + 1) * kPagedTile) - 1;
    return paged_max(1, paged_cdiv(s.prefix_len, kPagedKeys) +
                            paged_cdiv(paged_visible(r, last / s.by_G), kPagedKeys));
}
// How many tiles from `tile` on, which has so many blocks, are full and have as many (itself
// in any case): those of the tokens that see no more keys than these blocks hold. A request
// has up to 2^19 tiles, but only some n / 128 numbers of blocks.
CFA_HD int paged_alike(const PagedShape &s, const PagedRequest &r, int tile, int blocks) {
    const int keys = (blocks - paged_cdiv(s.prefix_len, kPagedKeys)) * kPagedKeys;
    return paged_max(1, paged_min(r.n, keys - r.len + r.n) * s.G / kPagedTile - tile);
}
// What a request's own items cost: units of their blocks, and items.
struct PagedCost {
    long long blocks, items;
};
CFA_HD PagedCost paged_request_cost(const PagedShape &s, const PagedRequest &r) {
    if (r.n == 0) return PagedCost{0, 0};
    const int all = r.n * s.G;
    if (!paged_alone(s, r.n)) {
        if (r.len == 0) return PagedCost{0, 0};
        const int tile = paged_own_tile(all);  // (a last tile of fewer rows costs the same)
        const long long items = static_cast<long long>(s.nkv) * paged_cdiv(all, tile);
        return PagedCost{items * paged_cdiv(r.len, kPagedKeys) * paged_cost(paged_min(all, tile)),
                         items * paged_item_cost(paged_min(all, tile))};
    }
    PagedCost c{0, 0};
    int n = 1;
    CFA_ROLLED for (int row = 0, t = 0; row < all; row += n * kPagedTile, t += n) {
        const int blocks = paged_alone_blocks(s, r, t);
        n = paged_alike(s, r, t, blocks);
        c.blocks += static_cast<long long>(n) * blocks * paged_cost(all - row);
        c.items += static_cast<long long>(n) * paged_item_cost(all - row);
    }
    return PagedCost{c.blocks * s.nkv, c.items * s.nkv};
}

CFA_HD int paged_item_units(const PagedPlan &p, int rows, int cost, int blocks) {
    return blocks * cost + paged_item_cost(rows) * p.item_units;
}

// The totals: what all requests' own items cost, and the tokens of those that share and of
// those that are alone. block_bytes_clocks: clocks by 400 that the device's memory takes to
// deliver a block's keys and values to one of its SMs while it serves them all. valid: the
// offsets are in order.
CFA_HD PagedPlan paged_plan(const PagedShape &s, const PagedCost &own, int shared_tokens, int alone_tokens,
                            int block_bytes_clocks, bool valid) {
    PagedPlan p;
    p.shared_rows = shared_tokens * s.G;
    p.prefix_blocks = paged_cdiv(s.prefix_len, kPagedKeys);
    p.tiles = p.prefix_blocks == 0 ? 0 : paged_cdiv(p.shared_rows, kPagedTile);
    const int last_rows = p.shared_rows - (p.tiles - 1) * kPagedTile;  // every tile but the last is full
    const bool some = p.tiles > 0;
    // units of a block of all the prefix's items, and their paged_item_cost()s
    const int block = some ? s.nkv * ((p.tiles - 1) * kPagedMaxCost + paged_cost(last_rows)) : 0;
    const int items = some ? s.nkv * ((p.tiles - 1) * paged_item_cost(kPagedTile) + paged_item_cost(last_rows)) : 0;
    const long long prefix = static_cast<long long>(block) * p.prefix_blocks;
    // (requests that are alone have more work than bytes)
    const int own_blocks = static_cast<int>(own.blocks < kPagedMaxUnits ? own.blocks : kPagedMaxUnits) / paged_cost(1);
    const long long bytes =
        alone_tokens > 0 ? 0 : (own_blocks + (some ? static_cast<long long>(s.nkv) * p.prefix_blocks : 0)) * block_bytes_clocks;
    p.by_bytes = bytes > prefix + own.blocks + (items + own.items) * kPagedItemClocks;
    p.item_units = p.by_bytes ? 1 : kPagedItemClocks;
    p.full_units = paged_item_units(p, kPagedTile, kPagedMaxCost, p.prefix_blocks);
    const long long pu = prefix + static_cast<long long>(items) * p.item_units;
    const long long all = pu + own.blocks + own.items * p.item_units;
    p.valid = valid && all < kPagedMaxUnits;
    p.prefix_units = p.valid ? static_cast<int>(pu) : 0;
    p.units = p.valid ? static_cast<int>(all) : 0;
    // at least a block, so that a run inside an item never comes away empty
    p.share = paged_max(kPagedMaxCost, (p.units + s.grid - 1) / s.by_grid);
    p.alone_tokens = alone_tokens;
    // A refused batch has no rows either: offsets that go up and down count tokens more than
    // once, beyond what the workspace has room for.
    if (!p.valid) p.shared_rows = p.tiles = p.alone_tokens = 0;
    return p;
}

// The last request b whose `at(b)` (ascending, at(0) = 0) is at most x: requests that add
// nothing share theirs with the next one and are passed over.
template <typename At>
CFA_HD int paged_find(int B, int x, At at) {
    int lo = 0, hi = B;
    CFA_ROLLED while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// The item that holds unit u, of the requests e[0..B]; x: the item found before, if any.
CFA_HD void paged_item(const PagedShape &s, const PagedPlan &p, const PagedEntry *e, int B, int u, PagedPiece &x) {
    int rem;  // units of the item before u
    if (u < p.prefix_units) {
        const int head_units = p.prefix_units / s.by_nkv, full = p.full_units;
        x.req = -1;
        x.h = u / head_units;
        rem = u - x.h * head_units;
        const int tile = p.tiles == 1 ? 0 : paged_min(rem / full, p.tiles - 1);
        rem -= tile * full;
        x.row0 = tile * kPagedTile;
        x.rows = paged_min(kPagedTile, p.shared_rows - x.row0);
        x.prefix_blocks = x.blocks = p.prefix_blocks;
        x.own_limit = 0;
        x.cost = paged_cost(x.rows);
        x.r = PagedRequest{0, 0, 0};
    } else {
        x.req = paged_find(B, u - p.prefix_units, [&](int b) { return e[b].unit; });
        x.r = paged_request_at(e, x.req);
        const int mine = u - p.prefix_units - e[x.req].unit;
        const int per_head = (e[x.req + 1].unit - e[x.req].unit) / s.by_nkv;
        x.h = mine / per_head;
        rem = mine - x.h * per_head;
        if (!paged_alone(s, x.r.n)) {
            x.row0 = 0;
            const int all = x.r.n * s.G, tile = paged_own_tile(all);
            x.prefix_blocks = 0;
            x.blocks = paged_cdiv(x.r.len, kPagedKeys);
            if (all > tile) {
                const int each = paged_item_units(p, tile, paged_cost(tile), x.blocks);
                x.row0 = rem / each * tile;
                rem %= each;
            }
            x.rows = paged_min(tile, all - x.row0);
            x.own_limit = x.r.len;
        } else {
            const int all = x.r.n * s.G;
            int t = 0;
            if (rem > 0 && u == x.first_unit + x.units) {  // the tile behind the last one
                t = x.row0 / kPagedTile + 1;
                rem = 0;
            }
            CFA_ROLLED for (;;) {
                x.blocks = paged_alone_blocks(s, x.r, t);
                const int each = paged_item_units(p, all - t * kPagedTile, paged_cost(all - t * kPagedTile), x.blocks);
                const int n = paged_alike(s, x.r, t, x.blocks);
                if (rem < n * each) {
                    const int at = n > 1 ? rem / each : 0;
                    t += at;
                    rem -= at * each;
                    break;
                }
                rem -= n * each;
                t += n;
            }
            x.row0 = t * kPagedTile;
            x.rows = paged_min(kPagedTile, all - x.row0);
            x.prefix_blocks = p.prefix_blocks;
            x.own_limit = paged_visible(x.r, (x.row0 + x.rows - 1) / s.by_G);
        }
    }
    if (x.req >= 0) x.cost = paged_cost(x.rows);
    x.units = paged_item_units(p, x.rows, x.cost, x.blocks);
    x.first_unit = u - rem;
}

// The next piece of the run that ends before unit `end`, from unit u on; u moves behind it.
// False: the run has no more.
CFA_HD bool paged_next(const PagedShape &s, const PagedPlan &p, const PagedEntry *e, int B, int &u, int end,
                       PagedPiece &x) {
    CFA_ROLLED while (u < end) {
        paged_item(s, p, e, B, u, x);
        x.b0 = paged_cdiv(u - x.first_unit, x.cost);
        x.b1 = paged_min(x.blocks, paged_cdiv(end - x.first_unit, x.cost));
        u = paged_min(end, x.first_unit + x.units);
        if (x.b0 < x.b1) return true;
    }
    return false;
}

// Whether a request's item holds all the keys its rows see.
CFA_HD bool paged_sole(const PagedShape &s, const PagedPiece &x) {
    return x.req >= 0 && (s.prefix_len == 0 || paged_alone(s, x.r.n));
}
// Whether a piece writes its rows' results itself.
CFA_HD bool paged_final(const PagedShape &s, const PagedPiece &x) {
    return x.b0 == 0 && x.b1 == x.blocks && paged_sole(s, x);
}

// The runs of an item's first and last blocks.
CFA_HD int paged_first_run(const PagedPlan &p, int first_unit) { return first_unit / p.share; }
CFA_HD int paged_last_run(const PagedPlan &p, int first_unit, int blocks, int cost) {
    return (first_unit + (blocks - 1) * cost) / p.share;
}

// Where a piece leaves its record: rows of the record arrays. An item's first piece over the
// prefix and its first over a shared request's own keys have their places by key head and
// shared row, where the merge finds them without looking anything up. A run's first piece, where
// it goes on with an item, has the run's own place; so has a tile of a request that is alone
// and that the run's end cuts (a request that is alone has no place by shared row).
CFA_HD long long paged_first_record(const PagedShape &s, const PagedPlan &p, bool own, int h) {
    return (static_cast<long long>(own ? s.nkv : 0) + h) * p.shared_rows;
}
CFA_HD long long paged_run_record(const PagedShape &s, const PagedPlan &p, bool first_of_run, int run) {
    return 2ll * s.nkv * p.shared_rows + (2ll * run + (first_of_run ? 0 : 1)) * kPagedTile;
}
CFA_HD long long paged_record_rows(const PagedShape &s, long long shared_rows) {
    return 2 * s.nkv * shared_rows + 2ll * s.grid * kPagedTile;
}
// A piece's record: outputs at rec D + (chunk stride + row) 4, maximum and sum at rec + row,
// for rows from rec_row on. shared_tok0: shared tokens before the request.
CFA_HD void paged_record(const PagedShape &s, const PagedPlan &p, int shared_tok0, int run, PagedPiece &x) {
    if (x.b0 > 0 || (x.req >= 0 && paged_alone(s, x.r.n))) {
        x.rec = paged_run_record(s, p, x.b0 > 0, run);
        x.rec_row = 0;
        x.rec_stride = x.rows;
    } else {
        x.rec = paged_first_record(s, p, x.req >= 0, x.h);
        x.rec_row = shared_tok0 * s.G + x.row0;
        x.rec_stride = p.shared_rows;
    }
}

}  // namespace cfa
