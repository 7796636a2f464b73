// head_split.h -- how a token's heads are split over groups of lanes (host arithmetic).
#pragma once

#include <cstdint>

namespace moe {

// Parts of a token's query and key heads: at least one of a kind that is there, none larger
// in number than its heads.
struct HeadParts {
    int q, k;
};

// The heads of a token are split over several groups of lanes until four items fall to
// each resident group, down to eight heads an item (8192 tokens of 20 heads: 18.0 us, four
// heads an item 19.9, sixteen 17.4; the gradient 31.8, 32.4, 31.6, but of 4096 tokens 13.9,
// 15.1, 18.2); to one head where all heads are under way at once.  room: resident threads.
inline HeadParts head_parts(int64_t T, int hq, int hk, int lanes, int64_t room) {
    const int64_t have = T * lanes;
    const int64_t want = (4 * room + have - 1) / have, heads = static_cast<int64_t>(hq) + hk;
    const int least = have * heads <= room ? 1 : 8;
    auto part = [&](int n) {   // the kind's share of the groups
        int64_t s = (want * n + heads - 1) / heads;
        const int64_t most = (n + least - 1) / least;
        s = s > most ? most : s;
        return static_cast<int>(s < 1 ? (n > 0) : s);
    };
    return {part(hq), part(hk)};
}

// n heads in runs of `each` neighbours, the last run what is left and never empty: with
// `each` rounded up, fewer runs than parts may hold all heads (81 heads in 10 parts: 9 each,
// 9 runs; a tenth would begin behind the last head).
struct HeadRuns {
    int runs, each;
};

inline HeadRuns head_runs(int n, int parts) {
    if (n <= 0) return {0, 0};
    const int each = (n + parts - 1) / parts;
    return {(n + each - 1) / each, each};
}

}  // namespace moe
