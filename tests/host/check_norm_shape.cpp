// How norms' rows go to threads: every element has a place, and none of the sizes
// on the way overflows (undefined-behaviour sanitizer), up to the longest row.
// Without arguments it checks that; with "name" it reads calls and prints the
// kernel of each:
//   norm M K x_type vec q_kind
//   join M K y_type residual_type vec q_kind token_gate
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>

#include "norm_shape.h"

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

static void check_row(int M, int K, Mode mode)
{
    const RowShape s = row_shape_of(M, K, mode);
    const long long octets = ((long long)K + 7) / 8, turns = (octets + s.lanes - 1) / s.lanes;
    CHECK(octets_of(K) == octets, "K=%d: %d octets, not %lld", K, octets_of(K), octets);
    CHECK(s.lanes >= 16 && s.lanes <= 1024 && (s.lanes & (s.lanes - 1)) == 0 && s.threads % s.lanes == 0 &&
              s.threads >= 256 && s.threads <= 1024, "M=%d K=%d: %d lanes", M, K, s.lanes);
    // all of a row's octets: in registers, or turn by turn
    CHECK(s.octets ? s.octets >= turns : turns > (mode == kVectors ? 4 : mode == kStrided ? 2 : 1),
          "M=%d K=%d mode %d: %d octets for %lld turns", M, K, mode, s.octets, turns);
    // an element's index in a row has 32 bits
    CHECK(8 * turns * s.lanes <= 0xFFFFFFFFLL, "K=%d", K);
    const long long most = rows_of_launch(s);
    CHECK(most > 0 && (most + s.threads / s.lanes - 1) / (s.threads / s.lanes) * s.threads <= 0xFFFFFFFFLL, "K=%d", K);
}

static void check_stream(const RowStream &s, int M, int K, int most_waves)
{
    if (!s.c)
        return;
    CHECK(K % 8 == 0 && s.threads % 64 == 0 && s.threads <= 1024 && (long long)s.c * s.threads >= K / 8 &&
              (long long)(s.c - 1) * s.threads < K / 8, "M=%d K=%d: %d octets, %d threads", M, K, s.c, s.threads);
    CHECK(s.groups >= 1 && s.groups <= (s.rows - 1LL + M) / s.rows && s.groups * (s.threads / 64) <= 256 * most_waves,
          "M=%d K=%d: %d workgroups", M, K, s.groups);
}

static void sizes()
{
    std::mt19937 rng(1);
    const auto log_pick = [&](double hi) {
        return (int)std::exp2(std::uniform_real_distribution<double>(0.0, std::log2(hi))(rng));
    };
    const int ends[] = {1, 7, 8, 9, 127, 128, 129, 8191, 8192, 8193, 16384, 16385, 0x7FFFFFF7, 0x7FFFFFF8, 0x7FFFFFF9,
                        0x7FFFFFFA, 0x7FFFFFFC, 0x7FFFFFFE, 0x7FFFFFFF};
    for (int round = 0; round < 300000; ++round) {
        const int K = round < 3000 ? ends[round % 19] : log_pick(2147483647.0);
        const int M = round % 7 == 0 ? 0x7FFFFFFF : log_pick(2147483647.0);
        for (const Mode mode : {kVectors, kElements, kStrided})
            if (mode == kStrided || K % (mode == kVectors ? 8 : 32) == 0)
                check_row(M, K, mode);
        for (int type = 0; type < 3; ++type) {
            check_stream(norm_stream_of(M, K, type, K % 8 == 0), M, K, 32);
            for (int other = 0; other < 3; ++other)
                check_stream(join_stream_of(M, K, type, other, K % 8 == 0, false), M, K, 16);
        }
    }
}

static void print(const RowStream &s, const char *op, int M, int K, int vec, int q_kind)
{
    if (s.c) {
        printf("%s_stream %d %d\n", op, s.c, s.rows);
        return;
    }
    const Mode mode = mode_of(vec, q_kind);
    printf("%s_kernel %d %s\n", op, row_shape_of(M, K, mode).octets,
           mode == kVectors ? "vectors" : mode == kElements ? "elements" : "strided");
}

int main(int argc, char **)
{
    if (argc == 1) {
        sizes();
        printf("ok\n");
        return 0;
    }
    char op[8];
    int M, K, y, r, vec, q, token;
    while (scanf("%7s", op) == 1)
        if (!strcmp(op, "norm")) {
            CHECK(scanf("%d %d %d %d %d", &M, &K, &y, &vec, &q) == 5, "norm?");
            print(norm_stream_of(M, K, y, vec), op, M, K, vec, q);
        } else {
            CHECK(scanf("%d %d %d %d %d %d %d", &M, &K, &y, &r, &vec, &q, &token) == 7, "join?");
            print(join_stream_of(M, K, y, r, vec, token), op, M, K, vec, q);
        }
    return 0;
}
