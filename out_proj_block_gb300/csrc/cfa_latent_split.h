// cfa_latent_split.h -- how the attention over paged latent rows is cut into work for a fixed
// number of runs, from the requests' offsets and lengths. The same code runs in the kernels
// and on the host.
//
// A request's query rows are its tokens times the heads, token major, which is how they lie in
// memory; they are cut into tiles of kLatTile. A tile goes over the cache rows that its last token sees,
// in blocks of kLatKeys. The units of all tiles (kLatItem for the tile's beginning and end, then one for each
// block) in the order of requests and tiles are dealt out in equal runs; a block goes to the run in
// which its unit lies. A run's part of one tile is a piece; a piece that is a whole tile writes its
// result, every other one leaves a record, and the records of a tile are merged in the order of the runs.
#pragma once

#include "cfa_paged_split.h"

namespace cfa {

constexpr int kLatTile = 128;  // query rows of a tile
constexpr int kLatKeys = 128;  // cache rows of a block
constexpr int kLatItem = 2;    // units of a tile beside its blocks
constexpr int kLatMaxUnits = (1 << 30) - 1;  // two of them added stay below 2^31

struct LatentRequest {
    int tok0, n, len;  // first token, tokens, cache rows
};

// Cache rows that token i of a request sees.
CFA_HD int latent_visible(const LatentRequest &r, int i) {
    return paged_max(0, paged_min(r.len, r.len - r.n + i + 1));
}

// Rows of a tile, and how many of them the first block of a cluster takes: half, so that few rows are
// spread over both.
CFA_HD int latent_rows(const LatentRequest &r, int H, int tile) { return paged_min(kLatTile, r.n * H - tile * kLatTile); }
CFA_HD int latent_split(int rows) { return (rows + 1) / 2; }

CFA_HD int latent_tiles(int n, int H) { return (n * H + kLatTile - 1) / kLatTile; }

// Blocks of a tile: those its last token sees.
CFA_HD int latent_blocks(const LatentRequest &r, const FastDiv &by_H, int tile) {
    const int last = paged_min(r.n - 1, (tile * kLatTile + kLatTile - 1) / by_H);
    return (latent_visible(r, last) + kLatKeys - 1) / kLatKeys;
}

// The last tile from `tile` on that has as many blocks: they grow along the tokens, and equal
// ones are counted together, as a prompt of 131,072 tokens has a million tiles.
CFA_HD int latent_like(const LatentRequest &r, int H, int tile, int blocks) {
    const int tiles = latent_tiles(r.n, H);
    // tokens up to `most` see no more than that many blocks
    const long long most = static_cast<long long>(blocks) * kLatKeys - (r.len - r.n) - 1;
    if (most >= r.n - 1) return tiles - 1;
    // the last tile whose last row, 128 i + 127, belongs to one of them
    const int i = static_cast<int>((most + 1) * H / kLatTile) - 1;
    return paged_max(tile, paged_min(i, tiles - 1));
}

// Units of all tiles of a request, at most kLatMaxUnits.
CFA_HD int latent_units(const LatentRequest &r, int H, const FastDiv &by_H) {
    const int tiles = latent_tiles(r.n, H);
    long long units = 0;
    CFA_ROLLED for (int i = 0; i < tiles;) {
        const int blocks = latent_blocks(r, by_H, i), last = latent_like(r, H, i, blocks);
        units += static_cast<long long>(last - i + 1) * (blocks + kLatItem);
        i = last + 1;
    }
    return units > kLatMaxUnits ? kLatMaxUnits : static_cast<int>(units);
}

// Units of several requests together, and whether a call may have that many.
CFA_HD int latent_more(int a, int b) { return paged_min(a + b, kLatMaxUnits); }
CFA_HD bool latent_fits(int units) { return units < kLatMaxUnits; }

// A part of one tile.
struct LatentPiece {
    LatentRequest r;
    int req, tile;
    int unit;    // the tile's first unit
    int blocks;  // the tile's blocks
    int b0, b1;  // of which this piece takes [b0, b1)
};

// Goes from tile to tile of a run, the units [u0, u1) of all. `request(b)` reads request b.
struct LatentWalk {
    int u0, u1;
    LatentPiece x;
    bool fresh;  // the piece that x holds has not been given out

    // At the run's begin, which lies in request b, r, whose first unit is `unit`.
    CFA_HD void begin(int from, int to, int b, const LatentRequest &r, int unit, int H, const FastDiv &by_H) {
        u0 = from;
        u1 = to;
        fresh = false;
        if (u0 >= u1) return;
        x.req = b;
        x.r = r;
        x.tile = 0;
        x.unit = unit;
        fresh = true;
        // on to the tile in which u0 lies
        const int tiles = latent_tiles(x.r.n, H);
        CFA_ROLLED while (x.tile < tiles) {
            x.blocks = latent_blocks(x.r, by_H, x.tile);
            const int cost = x.blocks + kLatItem, like = latent_like(x.r, H, x.tile, x.blocks) - x.tile + 1;
            const int skip = paged_min(like, paged_max(0, u0 - x.unit) / cost);
            x.tile += skip;
            x.unit += skip * cost;
            if (skip < like) break;
        }
        if (x.tile >= tiles) fresh = false;  // (does not happen: u0 lies in the request)
    }

    // The next piece of the run with anything to do (blocks, or a tile without any, whose rows
    // become zeros); false at the end.
    template <typename Request>
    CFA_HD bool next(int B, int H, const FastDiv &by_H, const Request &request) {
        if (u0 >= u1) return false;
        for (;;) {
            if (!fresh) {
                x.unit += x.blocks + kLatItem;
                ++x.tile;
                if (x.unit >= u1) return false;
                CFA_ROLLED while (x.tile >= latent_tiles(x.r.n, H)) {
                    if (++x.req >= B) return false;
                    x.r = request(x.req);
                    x.tile = 0;
                }
                x.blocks = latent_blocks(x.r, by_H, x.tile);
            }
            fresh = false;
            const int first = x.unit + kLatItem;
            x.b0 = paged_max(0, paged_min(x.blocks, u0 - first));
            x.b1 = paged_max(0, paged_min(x.blocks, u1 - first));
            if (x.b0 < x.b1 || (x.blocks == 0 && x.unit >= u0)) return true;
        }
    }
};

}  // namespace cfa
