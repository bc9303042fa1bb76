// Which kernel takes the products of rows grouped by expert, and in which clusters: host
// arithmetic alone. M rows for E experts with weights of N x K each.
#pragma once

#include <algorithm>

namespace qg {
namespace fp8 {

// What joining the parts of a tile takes, in k blocks (0.4 us each): parts into shared
// memory, a barrier of the epilogue's threads, arrivals at every CTA and the wait for theirs,
// the reads from the others, the outputs, and a second round of barrier and arrivals before
// the next tile. Charged alike for 1 and for 64 rows (up to 32 KB per CTA to exchange).
constexpr int kJoin = 10;

// The kernel of few rows: CTAs per cluster (0: the GPU holds none of them), and the k
// blocks that one of them takes one after the other if no expert has more than 64 rows.
struct FewPlan {
    int split;
    long long chain;
};

// The size of the clusters: the one with the fewest k blocks one after the other if the
// rows are spread over as many experts as there can be; a larger one has to save 4 %.
// room[i]: how many clusters of i CTAs the GPU holds at once, i = 1 .. 8.
inline FewPlan few_plan(const int* room, long long M, long long E, long long N, long long K) {
    const long long kb = (K + 127) / 128, tiles = (N + 127) / 128 * std::min(M, E);
    FewPlan p{0, 0};
    for (int i = 1; i < 9 && (i == 1 || kb >= 2 * i); ++i) {
        if (room[i] < 1) continue;
        const long long ctas = (long long)i * room[i], rest = tiles % ctas;
        const long long shares = (rest + room[i] - 1) / room[i];
        const long long chain = tiles / ctas * kb + shares * (i == 1 ? kb : (kb + i - 1) / i + kJoin);
        if (p.split == 0 || chain * 100 < p.chain * 96) p = {i, chain};
    }
    return p;
}

// Whether the kernel of few rows takes them, by the rows that an expert has on average:
// at 32 it takes 93 us of 32 experts, N = K = 4096, and the other one 100; at 48 107 and
// 104, at 64 133 and 112. Up to 64 it is also taken where it leaves fewer SMs idle, since
// it splits K for its last tiles (9 experts of 34 rows, N = 2200, K = 5200). The host knows
// no more than the average, and counts rows that no expert has: both kernels are right for
// every spread.
inline bool may_be_few(long long M, long long E) { return M <= 64 * E; }
inline bool takes_few(const FewPlan& p, int sms, long long M, long long E, long long N, long long K) {
    if (p.split == 0 || !may_be_few(M, E)) return false;
    if (M <= 32 * E) return true;
    const long long pairs = std::max(1, sms / 2), tiles = (N + 255) / 256 * E;
    return 5 * p.chain < 4 * ((tiles + pairs - 1) / pairs) * ((K + 127) / 128);
}

}  // namespace fp8
}  // namespace qg
