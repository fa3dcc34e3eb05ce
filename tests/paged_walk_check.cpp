// Checks how csrc/cfa_paged_split.h goes through the tiles of long requests: what it counts and
// finds against a plain list of the tiles, and that the longest calls are cut up in time (some
// 500,000 tiles of one request, which no block can go through for every piece). Prints "ok" or
// what is wrong.
#include "cfa_paged_split.h"

#include <chrono>
#include <cstdio>
#include <random>
#include <vector>

using namespace cfa;

namespace {

struct Tile {
    int req, h, row0, rows, blocks, own_limit;
};

// The items of requests that are alone, in order, from the definition: a tile's last row sees
// the prefix and its own keys up to its position.
std::vector<Tile> tiles(const PagedShape &s, const std::vector<PagedRequest> &req) {
    std::vector<Tile> out;
    for (size_t b = 0; b < req.size(); ++b)
        for (int h = 0; h < s.nkv; ++h)
            for (int row0 = 0; row0 < req[b].n * s.G; row0 += 256) {
                const int rows = req[b].n * s.G - row0 < 256 ? req[b].n * s.G - row0 : 256;
                const int token = (row0 + rows - 1) / s.G;
                int sees = req[b].len - req[b].n + token + 1;
                sees = sees < 0 ? 0 : sees;
                const int blocks = (s.prefix_len + 127) / 128 + (sees + 127) / 128;
                out.push_back({static_cast<int>(b), h, row0, rows, blocks < 1 ? 1 : blocks, sees});
            }
    return out;
}

const char *check(const PagedShape &s, const std::vector<PagedRequest> &req, int clocks, bool each) {
    PagedCost total{0, 0};
    std::vector<PagedCost> costs;
    int tokens = 0;
    for (const PagedRequest &r : req) {
        costs.push_back(paged_request_cost(s, r));
        total.blocks += costs.back().blocks;
        total.items += costs.back().items;
        tokens += r.n;
    }
    const PagedPlan p = paged_plan(s, total, 0, tokens, clocks, true);
    if (!p.valid) return "not valid";
    std::vector<PagedEntry> e;
    int unit = 0;
    for (size_t b = 0; b < req.size(); ++b) {
        e.push_back(PagedEntry{unit, 0, req[b].tok0, req[b].len});
        unit += static_cast<int>(costs[b].blocks + costs[b].items * p.item_units);
    }
    e.push_back(PagedEntry{unit, 0, tokens, 0});
    if (unit != p.units) return "units lost";
    const std::vector<Tile> all = tiles(s, req);
    long long blocks = 0, items = 0;
    for (const Tile &t : all) {
        blocks += t.blocks * (t.rows <= 128 ? 5 : 8);
        items += t.rows <= 16 ? 1 : 6;
    }
    if (blocks != total.blocks || items != total.items) return "the totals are not the tiles'";
    // every run's pieces follow one another through the list
    size_t at = 0;
    int done = 0;  // blocks of tile `at` that are dealt out
    for (int run = 0; run < s.grid; ++run) {
        const long long begin = static_cast<long long>(run) * p.share;
        int u = static_cast<int>(begin < p.units ? begin : p.units);
        const int end = static_cast<int>(begin + p.share < p.units ? begin + p.share : p.units);
        PagedPiece x;
        while (paged_next(s, p, e.data(), static_cast<int>(req.size()), u, end, x)) {
            const Tile &t = all[at];
            if (x.req != t.req || x.h != t.h || x.row0 != t.row0 || x.rows != t.rows || x.blocks != t.blocks ||
                x.own_limit != t.own_limit || x.b0 != done)
                return "a piece out of its place";
            done = x.b1;
            if (done == x.blocks) ++at, done = 0;
            if (!each) continue;
            PagedPiece y;  // the same piece found without the one before it
            int v = x.first_unit + x.b0 * x.cost;
            if (!paged_next(s, p, e.data(), static_cast<int>(req.size()), v, end, y)) return "a piece is not found again";
            if (y.row0 != x.row0 || y.b0 != x.b0 || y.b1 != x.b1 || y.first_unit != x.first_unit || y.units != x.units)
                return "a piece is found elsewhere";
        }
    }
    return at == all.size() ? nullptr : "tiles without a piece";
}

}  // namespace

int main() {
    std::mt19937 rng(5);
    auto rnd = [&](int a, int b) { return a + static_cast<int>(rng() % static_cast<unsigned>(b - a + 1)); };
    const int groups[] = {1, 2, 3, 4, 7, 8, 12, 16, 40, 100, 129, 255, 256, 257, 1024};
    for (int it = 0; it < 4000; ++it) {
        const int G = groups[rnd(0, 14)];
        const PagedShape s(G, rnd(1, 3), rnd(0, 2) ? rnd(1, 700) : 0, rnd(0, 1) ? 152 : rnd(1, 20));
        std::vector<PagedRequest> req;
        int tok0 = 0;
        for (int b = rnd(1, 4); b > 0; --b) {
            const int least = 128 / G + 1, n = rnd(0, 3) ? rnd(least, least + 400) : rnd(least, least + 3000);
            req.push_back({tok0, n, rnd(0, 3) ? rnd(0, n + 900) : rnd(0, 1) ? n : rnd(0, 3)});
            tok0 += n;
        }
        if (const char *wrong = check(s, req, rnd(1, 9), true)) return std::printf("batch %d: %s\n", it, wrong), 1;
    }
    const struct { int G, nkv, n, len, prefix; } longest[] = {
        {1024, 1, 1 << 17, 40, 9}, {1024, 1, 1 << 17, 0, 0}, {1024, 1, 40000, 45000, 300}, {1, 32, 1 << 17, 1 << 17, 0},
        {4, 8, 1 << 17, 1 << 17, 0}, {7, 4, 131071, 200000, 12345}};
    for (const auto &c : longest) {
        const PagedShape s(c.G, c.nkv, c.prefix, 152);
        const auto t0 = std::chrono::steady_clock::now();
        if (const char *wrong = check(s, {{0, c.n, c.len}}, 7, false)) return std::printf("G %d: %s\n", c.G, wrong), 1;
        const double took = std::chrono::duration<double>(std::chrono::steady_clock::now() - t0).count();
        if (took > 3.0) return std::printf("G %d, %d tokens: %.1f s\n", c.G, c.n, took), 1;
    }
    std::puts("ok");
    return 0;
}
