// Brute force over the addressing of parts of packed sequences: every place a
// launch provides for, with starts that rise, stand still, fall and lie outside
// the tokens.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "linear_places.h"

using namespace skinny;

#define CHECK(c)                                                                                                       \
    do {                                                                                                               \
        if (!(c)) {                                                                                                    \
            printf("line %d: %s\n", __LINE__, #c);                                                                     \
            exit(1);                                                                                                   \
        }                                                                                                              \
    } while (0)

// the kernels' search: how many sequences start at or before the place
static int seq_at(const std::vector<int> &starts, int tokens, int size, int place)
{
    int count = 0;
    for (size_t i = 0; i + 1 < starts.size(); ++i)
        count += first_place(starts[i], tokens, size, (int)i) <= place;
    return count - 1;
}

int main()
{
    std::mt19937 rng(7);
    const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    for (int round = 0; round < 20000; ++round) {
        const int size = 64 * pick(1, 6), b = pick(1, 70);
        const int tokens = pick(0, 3) ? pick(0, 3000) : 64 * pick(0, 40);
        const bool good = round % 2 == 0;
        std::vector<int> starts(b + 1);
        for (int &s : starts)
            s = good ? pick(0, tokens) : pick(0, 9) ? pick(-tokens - 100, 2 * tokens + 100) : (int)rng();
        if (good) {
            std::sort(starts.begin(), starts.end());
            starts[0] = 0;
            starts[b] = tokens;
        }
        const int places = tokens / size + b;
        std::set<std::pair<int, int>> seen;
        for (int place = 0; place < places; ++place) {
            const int seq = seq_at(starts, tokens, size, place);
            if (seq < 0)
                continue;
            CHECK(seq < b);
            Place p;
            if (!place_of(starts[seq], starts[seq + 1], tokens, size, place, seq, p))
                continue;
            // every token the part touches exists
            CHECK(p.seq == seq && p.part >= 0 && p.len >= 0 && p.first >= 0 && p.first + p.len <= tokens);
            CHECK((long long)p.part * size < p.len || (p.part == 0 && p.len == 0));
            CHECK(seen.insert({seq, p.part}).second);
        }
        // the joining kernel goes over a sequence's places itself
        for (int seq = 0; seq < b; ++seq) {
            const int place0 = first_place(starts[seq], tokens, size, seq);
            Place p;
            place_of(starts[seq], starts[seq + 1], tokens, size, place0, seq, p);
            const int parts = parts_of(p.len, size);
            CHECK(place0 >= 0 && place0 + parts <= places);
            if (good)
                for (int j = 0; j < parts; ++j)
                    CHECK(seen.count({seq, j}));
        }
    }
    printf("places ok\n");
    return 0;
}
