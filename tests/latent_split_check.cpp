// Check of how the attention over latent rows is cut: every block of every tile lies in exactly one
// run's piece, runs know which records belong to a tile, and equal tiles counted together add up.
// Prints "ok" or what is wrong.
#include "cfa_latent_split.h"

#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

using namespace cfa;

namespace {

int failed(const char *what, int a, int b, int c) {
    std::printf("%s: %d %d %d\n", what, a, b, c);
    return 1;
}

int check(const std::vector<LatentRequest> &reqs, int H, int runs, int least) {
    const FastDiv by_H(static_cast<uint32_t>(H));
    const int B = static_cast<int>(reqs.size());
    std::vector<int> first(B + 1, 0);
    std::vector<int> tiles(B);
    for (int b = 0; b < B; ++b) {
        tiles[b] = latent_tiles(reqs[b].n, H);
        long long units = 0;
        for (int i = 0; i < tiles[b]; ++i) {
            const int last = std::min(reqs[b].n - 1, (i * kLatTile + kLatTile - 1) / H);
            const int want = (std::max(0, std::min(reqs[b].len, reqs[b].len - reqs[b].n + last + 1)) + kLatKeys - 1) / kLatKeys;
            if (latent_blocks(reqs[b], by_H, i) != want) return failed("blocks", b, i, want);
            units += want + kLatItem;
        }
        if (latent_units(reqs[b], H, by_H) != units) return failed("units", b, latent_units(reqs[b], H, by_H), static_cast<int>(units));
        first[b + 1] = first[b] + static_cast<int>(units);
    }
    const int all = first[B], share = std::max(least, (all + runs - 1) / runs);
    auto request = [&](int b) { return reqs[b]; };
    struct Tile {
        int done = 0, pieces = 0, zeros = 0, begun = -1, last = -1;
    };
    std::map<std::pair<int, int>, Tile> seen;
    for (int run = 0; run < runs; ++run) {
        const int u0 = static_cast<int>(std::min<long long>(static_cast<long long>(run) * share, all));
        const int u1 = static_cast<int>(std::min<long long>(static_cast<long long>(run) * share + share, all));
        LatentWalk w;
        int b = 0;
        while (b < B && first[b + 1] <= u0) ++b;
        if (u0 < u1 && b >= B) return failed("start", run, u0, u1);
        w.begin(u0, u1, b < B ? b : 0, reqs[b < B ? b : 0], b < B ? first[b] : 0, H, by_H);
        int cut = 0, went_on = 0;
        while (w.next(B, H, by_H, request)) {
            const LatentPiece &x = w.x;
            Tile &t = seen[{x.req, x.tile}];
            const int blocks = latent_blocks(reqs[x.req], by_H, x.tile), rows = latent_rows(x.r, H, x.tile);
            if (rows < 1 || rows > kLatTile || latent_split(rows) > 64 || rows - latent_split(rows) > 64)
                return failed("rows", run, x.req, rows);
            if (x.blocks != blocks || x.tile >= tiles[x.req]) return failed("piece", run, x.req, x.tile);
            if (x.b0 == x.b1) {
                ++t.zeros;
                continue;
            }
            if (x.b0 != t.done) return failed("order", x.req, x.tile, x.b0);
            t.done = x.b1;
            ++t.pieces;
            if (x.b0 == 0) t.begun = run;
            if (x.b0 == 0 && x.b1 < blocks) {
                ++cut;
                t.last = (x.unit + x.blocks + kLatItem - 1) / share;
            }
            if (x.b0 > 0) {
                ++went_on;
                if (t.begun + t.pieces - 1 != run) return failed("a run without a piece", run, x.req, x.tile);
            }
            if (x.b0 > 0 && x.b1 == blocks && t.last != run) return failed("last run", run, t.last, x.tile);
        }
        if (cut > 1 || went_on > 1) return failed("records", run, cut, went_on);
    }
    for (int b = 0; b < B; ++b)
        for (int i = 0; i < tiles[b]; ++i) {
            const Tile t = seen[{b, i}];
            const int blocks = latent_blocks(reqs[b], by_H, i);
            if (t.done != blocks || t.zeros != (blocks == 0)) return failed("cover", b, i, t.done);
        }
    return 0;
}

}  // namespace

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<unsigned>(hi - lo + 1)); };
    const int heads[] = {1, 2, 3, 5, 8, 20, 32, 33, 64, 100, 127, 128, 129, 130, 200, 256, 1000, 1024};
    for (int round = 0; round < 4000; ++round) {
        const int H = heads[pick(0, 17)], B = pick(1, round % 7 == 0 ? 60 : 5), runs = pick(1, 90);
        std::vector<LatentRequest> reqs;
        int tok = 0;
        for (int b = 0; b < B; ++b) {
            const int kind = pick(0, 5);
            const int n = kind == 0 ? 0 : kind < 4 ? pick(1, 4) : pick(1, 400);
            const int len = kind == 1 ? pick(0, 6) : kind == 4 ? n + pick(0, 300) : pick(0, 6000);
            reqs.push_back({tok, n, len});
            tok += n;
        }
        if (check(reqs, H, runs, pick(1, 4))) return std::printf("round %d, %d heads\n", round, H), 1;
    }
    // the most tiles there are: counted by groups, in a blink
    const FastDiv by(1024);
    const LatentRequest most{0, 131072, 131072};
    long long want = 0;
    for (int i = 0; i < latent_tiles(most.n, 1024); ++i) want += latent_blocks(most, by, i) + kLatItem;
    if (want > kLatMaxUnits) want = kLatMaxUnits;
    if (latent_units(most, 1024, by) != want) return failed("most", latent_units(most, 1024, by), static_cast<int>(want), 0);
    std::printf("ok\n");
    return 0;
}
