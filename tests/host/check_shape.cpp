// A prompt's workspace: large enough for the parts that its sizes are cut into
// and for those of every smaller prompt, and each part's state in a place of its
// own, whatever the starts.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "linear_shape.h"

using namespace skinny;

#define CHECK(c, ...)                                                                                              \
    do {                                                                                                           \
        if (!(c)) {                                                                                                \
            printf("line %d: ", __LINE__);                                                                         \
            printf(__VA_ARGS__);                                                                                   \
            printf("\n");                                                                                          \
            exit(1);                                                                                               \
        }                                                                                                          \
    } while (0)

static int extra(int tokens, int sequences, int heads, int dk, int dv)
{
    const Shape s = shape_of(tokens, sequences, heads, dk, dv);
    CHECK(s.part > 0 && s.part % kChunk == 0 && s.places == tokens / s.part + sequences, "part %d", s.part);
    return s.multi ? extra_states(tokens, s.part) : 0;
}

static void sizes()
{
    std::mt19937 rng(3);
    const auto log_pick = [&](double lo, double hi) {
        return (int)(lo * std::exp2(std::uniform_real_distribution<double>(0.0, std::log2(hi / lo))(rng)));
    };
    for (int round = 0; round < 400000; ++round) {
        const int heads = log_pick(1, 900), dk = 8 * log_pick(1, 32.9), dv = 8 * log_pick(1, 128.9);
        const int tokens = round % 100 ? log_pick(1, 300000) : log_pick(1, 0x7FFFF000), sequences = log_pick(1, 65535);
        const int most = most_extra_parts(tokens, sequences, heads, dv);
        const int have = extra(tokens, sequences, heads, dk, dv);
        CHECK(have <= most, "%d tokens of %d, %d heads of %d, %d: %d parts, %d", tokens, sequences, heads, dk, dv, have, most);
        const int less = log_pick(1, tokens + 0.5), fewer = log_pick(1, sequences + 0.5);
        CHECK(less <= tokens && fewer <= sequences, "%d %d", less, fewer);
        CHECK(most_extra_parts(less, fewer, heads, dv) <= most, "%d tokens of %d against %d of %d, %d heads of %d", less,
              fewer, tokens, sequences, heads, dv);
    }
}

static void states()
{
    std::mt19937 rng(11);
    const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    for (int round = 0; round < 20000; ++round) {
        const int size = 64 * pick(1, 4), sequences = pick(1, round % 3 ? 9 : 60), tokens = pick(0, 2500);
        const bool rising = round % 2 == 0;
        std::vector<int> starts(sequences + 1);
        for (int &s : starts)
            s = rising ? (pick(0, 3) ? pick(0, tokens) : pick(0, tokens / size) * size) : (int)rng();
        if (rising) {
            starts[0] = 0;
            starts[sequences] = tokens;
            std::sort(starts.begin(), starts.end());
        }
        std::set<int> parts_seen, starts_seen;
        for (int seq = 0; seq < sequences; ++seq) {
            const int first = cut_to(starts[seq], 0, tokens), end = cut_to(starts[seq + 1], first, tokens);
            const int parts = parts_of(end - first, size);
            if (parts < 2)
                continue;
            const int at = start_state(first, tokens, size, sequences, seq);
            CHECK(at >= 0 && at < start_states(tokens, size, sequences), "round %d: start %d", round, at);
            CHECK(starts_seen.insert(at).second || !rising, "round %d: start %d twice", round, at);
            for (int j = 1; j < parts; ++j) {
                const int p = part_state(first, tokens, size, j);
                CHECK(p >= 0 && p < extra_states(tokens, size), "round %d: part %d", round, p);
                CHECK(parts_seen.insert(p).second || !rising, "round %d: part %d twice", round, p);
            }
        }
    }
}

int main()
{
    sizes();
    states();
    puts("ok");
    return 0;
}
