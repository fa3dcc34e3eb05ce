// Checks of csrc/cfa_paged_split.h on random batches: every block of keys of every row lies in
// exactly one piece, pieces follow the runs that the merge computes, records lie in their array
// and apart from one another, and FastDiv divides. Prints "ok" or what is wrong.
#include "cfa_paged_split.h"

#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <vector>

using namespace cfa;

namespace {

std::mt19937 rng(1);
int rnd(int a, int b) { return a + static_cast<int>(rng() % static_cast<unsigned>(b - a + 1)); }

struct Batch {
    std::vector<PagedRequest> req;
    std::vector<PagedEntry> entry;
    int tokens = 0, shared = 0;
};

const char *check(const PagedShape &s, const PagedPlan &p, const Batch &b) {
    const int B = static_cast<int>(b.req.size());
    std::map<std::vector<int>, std::vector<char>> seen;  // blocks of an item
    std::map<std::vector<int>, std::pair<int, int>> runs;  // pieces of an item, and what the merge expects
    std::vector<std::pair<long long, long long>> records;
    long long units = 0;
    for (int run = 0; run < s.grid; ++run) {
        const long long begin = static_cast<long long>(run) * p.share;
        const int end = static_cast<int>(std::min<long long>(p.units, begin + p.share));
        int u = static_cast<int>(std::min<long long>(p.units, begin));
        PagedPiece x;
        while (paged_next(s, p, b.entry.data(), B, u, end, x)) {
            if (x.rows < 1 || x.rows > kPagedTile || x.b1 <= x.b0 || x.b1 > x.blocks || x.h < 0 || x.h >= s.nkv)
                return "a piece out of range";
            if (x.req >= 0 && x.r.n == 0) return "a piece of a request without tokens";
            const std::vector<int> item{x.req, x.h, x.row0};
            std::vector<char> &blocks = seen[item];
            if (blocks.empty()) blocks.resize(x.blocks);
            if (static_cast<int>(blocks.size()) != x.blocks) return "an item's length changes";
            for (int j = x.b0; j < x.b1; ++j) {
                if (blocks[j]) return "a block twice";
                blocks[j] = 1;
            }
            const int first = paged_first_run(p, x.first_unit);
            const int last = paged_last_run(p, x.first_unit, x.blocks, x.cost);
            if (run < first || run > last || (x.b0 == 0) != (run == first) || (x.b1 == x.blocks) != (run == last))
                return "a piece in another run than the merge looks for";
            ++runs[item].first;
            runs[item].second = last - first + 1;
            units += (x.b1 - x.b0) * x.cost + (x.b1 == x.blocks ? x.units - x.blocks * x.cost : 0);
            if (paged_final(s, x)) continue;
            paged_record(s, p, x.req < 0 ? 0 : b.entry[x.req].tok, run, x);
            if (x.rec_stride != x.rows && (x.rec_stride != p.shared_rows || x.rec_row + x.rows > p.shared_rows))
                return "a record beyond its key head";
            records.push_back({x.rec + x.rec_row, x.rec + x.rec_row + x.rows});
        }
    }
    if (units != p.units) return "units lost";
    for (const auto &r : runs)
        if (r.second.first != r.second.second) return "a run without its piece";
    for (const auto &v : seen)
        for (char c : v.second)
            if (!c) return "a block without a piece";
    for (int i = 0; i < B; ++i)
        for (int h = 0; h < s.nkv && b.req[i].n > 0; ++h) {
            const bool alone = paged_alone(s, b.req[i].n);
            if (!alone && b.req[i].len == 0) continue;
            const int rows = b.req[i].n * s.G, tile = alone ? kPagedTile : paged_own_tile(rows);
            for (int r = 0; r < rows; r += tile)
                if (!seen.count({i, h, r})) return "rows without an item";
        }
    for (int h = 0; h < s.nkv && s.prefix_len > 0; ++h)
        for (int r = 0; r < p.shared_rows; r += kPagedTile)
            if (!seen.count({-1, h, r})) return "shared rows without an item";
    std::sort(records.begin(), records.end());
    for (size_t i = 0; i < records.size(); ++i) {
        if (records[i].first < 0 || records[i].second > paged_record_rows(s, p.shared_rows)) return "a record out of range";
        if (i > 0 && records[i - 1].second > records[i].first) return "records overlap";
    }
    return nullptr;
}

}  // namespace

int main() {
    int by_bytes[2] = {0, 0};
    for (int it = 0; it < 3000; ++it) {
        const PagedShape s(rnd(1, 3) == 1 ? 1 : rnd(1, 40), rnd(1, 5), rnd(0, 2) ? rnd(1, 3000) : 0, rnd(0, 1) ? 152 : rnd(1, 20));
        const int kind = rnd(0, 3), B = rnd(1, 40);
        Batch b;
        PagedCost total{0, 0};
        std::vector<PagedCost> costs;
        for (int i = 0; i < B; ++i) {
            PagedRequest r;
            r.tok0 = b.tokens;
            r.n = kind == 0 ? 1 : kind == 1 ? rnd(0, 9) : kind == 2 ? rnd(0, 300) : rnd(0, 5) ? rnd(0, 2) : rnd(0, 700);
            r.len = rnd(0, 4) ? rnd(0, 900) : rnd(0, 3);
            b.tokens += r.n;
            if (!paged_alone(s, r.n)) b.shared += r.n;
            b.req.push_back(r);
            costs.push_back(paged_request_cost(s, r));
            total.blocks += costs[i].blocks;
            total.items += costs[i].items;
        }
        PagedPlan p = paged_plan(s, total, b.shared, b.tokens - b.shared, rnd(1, 9), true);
        if (!p.valid) return std::puts("not valid"), 1;
        ++by_bytes[p.by_bytes];
        int unit = 0, shared = 0;
        for (int i = 0; i < B; ++i) {
            b.entry.push_back(PagedEntry{unit, shared, b.req[i].tok0, b.req[i].len});
            unit += static_cast<int>(costs[i].blocks + costs[i].items * p.item_units);
            shared += paged_alone(s, b.req[i].n) ? 0 : b.req[i].n;
        }
        b.entry.push_back(PagedEntry{unit, shared, b.tokens, 0});
        if (const char *wrong = check(s, p, b)) return std::printf("batch %d: %s\n", it, wrong), 1;
    }
    if (by_bytes[0] < 100 || by_bytes[1] < 100) return std::puts("a kind of plan was not met"), 1;
    for (long i = 0; i < 2000000; ++i) {
        const uint32_t d = 1 + rng() % (i % 3 == 0 ? 4u : i % 3 == 1 ? 300u : 1u << 20);
        const int n = static_cast<int>(rng() & 0x7fffffffu) >> (rng() % 31);
        if (n / FastDiv(d) != n / static_cast<int>(d)) return std::printf("%d / %u\n", n, d), 1;
    }
    // batches whose units pass what an int holds are refused, not wrapped
    const PagedShape big(1024, 1, 1 << 28, 152);
    if (paged_plan(big, PagedCost{0, 0}, 128, 0, 5, true).valid) return std::puts("a plan too large"), 1;
    std::puts("ok");
    return 0;
}
