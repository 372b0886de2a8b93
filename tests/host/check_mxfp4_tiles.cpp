// Which kernel a 4-bit product takes.  Without arguments: its tiles cover the
// product, and nothing on the way overflows (undefined-behaviour sanitizer), up to the
// largest sizes.  With "reach": every kernel that some size takes.  With
// "name": reads lines of M N bits words and prints the kernel of each.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <set>
#include <string>

#include "mxfp4_tiles.h"

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

static std::string name(int M, int N, int bits, bool words)
{
    const Product p = product_of(M, N, bits, words);
    char b[80];
    if (p.many)
        snprintf(b, sizeof b, "tiles %d bits %d %s", p.t, bits, words ? "words" : "any");
    else
        snprintf(b, sizeof b, "rows %dx%d bits %d x %d %s", p.r, p.t, bits, p.x_rows, p.once ? "once" : "again");
    return b;
}

int main(int argc, char **argv)
{
    std::mt19937 rng(1);
    const auto log_pick = [&](double hi) {
        return (int)std::exp2(std::uniform_real_distribution<double>(0.0, std::log2(hi))(rng));
    };
    if (argc == 1) {
        const int most = 0x7FFFF000;            // of both: kMaxRows in mxfp4.hip
        for (int round = 0; round < 400000; ++round) {
            const int M = round % 9 == 0 ? most : log_pick(most), N = round % 11 == 0 ? most : log_pick(most);
            const int bits = round % 2 ? 4 : 8;
            const bool words = round % 4 < 2;
            const Product p = product_of(M, N, bits, words);
            const long long rows = p.many ? 256 : 16 * p.r, tokens = p.many ? 32 * p.t : 16 * p.t;
            CHECK(p.n_tiles * rows >= N && (p.n_tiles - 1) * rows < N, "%d rows", N);
            CHECK(p.m_tiles * tokens >= M && (p.m_tiles - 1) * tokens < M, "%d tokens", M);
            CHECK(!p.many || (M > 64 && p.t >= kFewest && p.t <= most_tiles(bits, words)), "%d x %d", M, N);
            // rows of a load of x hold all of the tokens; one token tile has all of them
            CHECK(p.many || M <= p.x_rows || p.x_rows == 16, "%d x %d", M, N);
            CHECK(p.many || p.x_rows == 16 || p.once, "%d x %d", M, N);
            CHECK(p.once == (!p.many && M <= tokens), "%d x %d", M, N);
        }
        printf("ok\n");
    } else if (!strcmp(argv[1], "reach")) {
        std::set<std::string> seen;
        for (const int bits : {4, 8})
            for (const bool words : {false, true}) {
                for (int M = 1; M <= 800; ++M)
                    for (int N = 1; N <= 20000; N += 16)
                        seen.insert(name(M, N, bits, words));
                for (int round = 0; round < 100000; ++round) {
                    const int M = log_pick(1 << 17), N = log_pick(1 << 19);
                    seen.insert(name(M, N, bits, words));
                }
            }
        for (const std::string &s : seen)
            printf("%s\n", s.c_str());
    } else {
        int M, N, bits, words;
        while (scanf("%d %d %d %d", &M, &N, &bits, &words) == 4)
            printf("%s\n", name(M, N, bits, words).c_str());
    }
    return 0;
}
