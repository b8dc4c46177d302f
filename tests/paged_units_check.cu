// The closed forms by which the attention's unit walk counts blocks, against sums block by block (host code only).
#include <algorithm>
#include <cstdio>
#include <random>

#include "paged_work.cuh"

using namespace dgen::paged;

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    long bad = 0, checks = 0;
    for (int it = 0; it < 100000; ++it) {  // sum of floor((a i + b) / m)
        const uint32_t n = pick(0, 60), m = pick(1, 300), a = pick(0, 4000), b = pick(0, 100000);
        long long want = 0;
        for (uint32_t i = 0; i < n; ++i) want += (static_cast<long long>(a) * i + b) / m;
        if (floor_sum(n, m, a, b) != want && bad++ < 5) printf("floor_sum(%u, %u, %u, %u)\n", n, m, a, b);
        ++checks;
    }
    const int groups[] = {1, 2, 3, 4, 5, 7, 8, 16, 48, 128};
    for (int it = 0; it < 200000; ++it) {  // blocks before each super tile of a sequence
        Partition p{};
        p.G = groups[pick(0, 9)];
        p.R = pick(0, 1) && p.G <= 16 ? 16 / p.G * p.G : 128 / p.G * p.G;
        p.TS = 1 << pick(0, 2);
        p.KB = p.align = pick(0, 1) ? 128 : 64;
        p.log2_kb = p.KB == 64 ? 6 : 7;
        p.tokens = p.R / p.G * p.TS;
        p.causal = pick(0, 1);
        const int kind = pick(0, 9);
        p.window = kind < 5 ? 0 : kind < 9 ? pick(1, 700) : 2147483647 - pick(0, 3);
        SeqInfo s{};
        s.n = pick(1, pick(0, 1) ? 900 : 40);
        s.tiles = (s.n * p.G + p.R * p.TS - 1) / (p.R * p.TS);
        s.pos0 = pick(0, 2) == 0 ? 0 : pick(0, 3000);
        if (pick(0, 9) == 0)  // as far as the calls allow: all units' blocks below 2^31, positions below 2^30
            s.pos0 = static_cast<int>(std::min((1LL << 30), (2147480000LL / s.tiles - 8) * p.KB)) - s.n - pick(0, 300);
        s.len = s.pos0 + s.n;
        long long want = 0;
        for (int k = 0; k <= s.tiles; ++k) {
            if (prefix_blocks(s, p, k) != want && bad++ < 5)
                printf("tile %d: G %d R %d TS %d KB %d causal %d window %d n %d pos0 %d\n", k, p.G, p.R, p.TS, p.KB,
                       p.causal, p.window, s.n, s.pos0);
            ++checks;
            if (k == s.tiles) break;
            // keys that the tile's tokens see, from the definition: j <= p if causal, |p - j| < window
            const long long first = s.pos0 + static_cast<long long>(k) * p.tokens;
            const long long last = std::min<long long>(s.len, first + p.tokens) - 1;
            const long long w = p.window ? p.window : 1LL << 40;
            const long long lo = std::max(0LL, first - w + 1), hi = std::min<long long>(s.len - 1, p.causal ? last : last + w - 1);
            want += p.causal || p.window ? hi / p.KB - lo / p.KB + 1 : (s.len + p.KB - 1) / p.KB;
        }
        if (want > 2147483647LL) printf("beyond 32 bits\n"), ++bad;
    }
    printf("%ld checks, %ld bad\n", checks, bad);
    return bad != 0;
}
