// Check of how much attention over latent rows one call may ask for: the units of its requests together,
// on either side of the limit. Prints "ok" or what is wrong.
#include "cfa_latent_split.h"

#include <cstdio>
#include <vector>

using namespace cfa;

namespace {

// As the kernel adds them up: each thread its requests, then the threads' sums.
bool fits(const std::vector<LatentRequest> &reqs, int H) {
    const FastDiv by_H(static_cast<uint32_t>(H));
    int all = 0;
    for (const LatentRequest &r : reqs) all = latent_more(all, latent_units(r, H, by_H));
    return latent_fits(all);
}

}  // namespace

int main() {
    constexpr int H = 128, kRows = 1 << 30;  // a tile a token
    const auto many = [&](int requests, int rows, int last) {
        std::vector<LatentRequest> r;
        for (int b = 0; b < requests; ++b) r.push_back({b, 1, rows});
        if (last > 0) r.push_back({requests, 1, last});
        return r;
    };
    if (!fits(many(100, kRows, 0), H)) return std::puts("838,861,000 units were refused"), 1;
    // 127 requests of 2^23 blocks and two units leave room for one of `left` units
    const long long left = (1ll << 30) - 1 - 127ll * ((1 << 23) + 2);
    const int most = static_cast<int>((left - 1 - 2) * kLatKeys);  // rows of a request that still fits
    if (!fits(many(127, kRows, most), H)) return std::puts("2^30 - 2 units were refused"), 1;
    if (fits(many(127, kRows, most + 1), H)) return std::puts("2^30 - 1 units were taken"), 1;
    if (fits(many(128, kRows, 0), H)) return std::puts("2^30 + 256 units were taken"), 1;
    if (fits(many(1024, kRows, 0), H)) return std::puts("2^33 units were taken"), 1;
    // eight tiles to a token
    if (fits({{0, 16, kRows}}, 1024) || !fits({{0, 15, kRows}}, 1024)) return std::puts("tiles of one request"), 1;
    std::puts("ok");
    return 0;
}
