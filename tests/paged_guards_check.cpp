// Checks of what the paged kernels make of device data that is out of range, by the rules they
// share with the host (csrc/cfa_paged.h, csrc/cfa_paged_split.h). Prints "ok" or what is wrong.
#include "cfa_paged.h"
#include "cfa_paged_split.h"

#include <algorithm>
#include <climits>
#include <cstdio>
#include <vector>

using namespace cfa;

namespace {

// The scan of the attention kernel over offsets that go up and down: every request that looks
// right by itself is counted, whatever lies between.
const char *offsets(int max_seqs, int max_tokens, int G, int prefix, int each) {
    const PagedShape s(G, 1, prefix, 152);
    std::vector<int> cu;
    for (int b = 0; b <= max_seqs; ++b) cu.push_back(b % 2 ? each : 0);
    PagedCost total{0, 0};
    int shared = 0;
    bool valid = true;
    for (int b = 0; b < max_seqs; ++b) {
        const PagedRequest r{cu[b], cu[b + 1] - cu[b], 40};
        if (r.tok0 < 0 || r.n < 0 || r.n > max_tokens || r.tok0 > max_tokens - r.n) {
            valid = false;
            continue;
        }
        const PagedCost c = paged_request_cost(s, r);
        total.blocks += c.blocks;
        total.items += c.items;
        shared += paged_alone(s, r.n) ? 0 : r.n;
    }
    if (valid) return "offsets that go down were taken";
    const int room = std::min(max_tokens * G, max_seqs * kPagedAloneRows);
    if (shared * G <= room) return "the batch does not reach past the workspace";
    const PagedPlan p = paged_plan(s, total, shared, cu[max_seqs] - cu[0] - shared, 7, valid);
    // the rows that are described for the merge, and the work of the blocks
    if (p.valid || p.units || p.prefix_units) return "a refused plan has work";
    if (p.shared_rows || p.tiles || p.alone_tokens) return "a refused plan has rows";
    return nullptr;
}

// Pages that a pool can give: never more than lie between its first counter and the list's end.
const char *pools() {
    const int counts[] = {INT_MIN, INT_MIN + 1, -5, -2, -1, 0, 1, 3, 4, 5, 100, 1 << 30, INT_MAX - 1, INT_MAX};
    for (int taken : counts)
        for (int there : counts)
            for (int n_free : {0, 1, 4, 5, INT_MAX}) {
                const int left = paged_pool_left(taken, there, n_free);
                if (taken < 0 || there < 0) {
                    if (left != -1) return "a counter below zero was taken";
                    continue;
                }
                const long long end = std::min(there, n_free);
                if (left != std::max(0ll, end - taken)) return "pages that are not there";
            }
    return nullptr;
}

}  // namespace

int main() {
    const struct { int seqs, tokens, G, prefix, each; } batches[] = {
        {64, 32, 4, 0, 32}, {256, 256, 4, 4096, 32}, {256, 256, 4, 100, 7}, {1024, 128, 1, 0, 128}, {9, 2, 3, 64, 2}};
    for (const auto &b : batches)
        if (const char *wrong = offsets(b.seqs, b.tokens, b.G, b.prefix, b.each))
            return std::printf("%d requests: %s\n", b.seqs, wrong), 1;
    if (const char *wrong = pools()) return std::puts(wrong), 1;
    // more work than its units can count is refused in the same way
    const PagedShape big(1024, 1, 1 << 28, 152);
    const PagedPlan p = paged_plan(big, PagedCost{0, 0}, 128, 0, 5, true);
    if (p.valid || p.units || p.shared_rows || p.tiles) return std::puts("a plan too large has rows"), 1;
    std::puts("ok");
    return 0;
}
