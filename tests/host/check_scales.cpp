// The powers of two of linear attention's FP16 operands: values come into
// range, the powers are each other's inverse, and the factors that bring an
// output's sum from the state's range into the score tiles' stay finite.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "linear_scales.h"

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

static unsigned bits(float f)
{
    unsigned u;
    memcpy(&u, &f, 4);
    return u;
}

static float value(unsigned u)
{
    float f;
    memcpy(&f, &u, 4);
    return f;
}

static void range(float top, unsigned least, float &mul, float &back)
{
    unsigned m, b;
    half_range_bits(bits(top), least, m, b);
    mul = value(m);
    back = value(b);
}

int main()
{
    std::vector<float> tops = {0.0f, 1e-45f, 3e38f, INFINITY};
    for (int e = -126; e <= 127; ++e)
        for (float m : {1.0f, 1.5f, 1.9999999f})
            tops.push_back(std::ldexp(m, e));
    for (unsigned least : {kLeastExponent, kLeastScoreExponent})
        for (float top : tops) {
            float mul, back;
            range(top, least, mul, back);
            CHECK(std::isnormal(mul) && std::isnormal(back) && mul * back == 1.0f, "powers of %g: %g %g", top, mul, back);
            CHECK(value(inverse_power_bits(bits(back))) == mul, "inverse of %g", back);
            if (std::isfinite(top)) {
                CHECK(top * mul < 32768.0f, "%g times %g", top, mul);
                CHECK(bits(top) >> 23 < least || top * mul >= 16384.0f, "%g times %g", top, mul);
            }
        }
    // dk = 256 products of a state's term, below 2^15, with an FP16 value, at decay and scale 1; a lane's 32 are summed
    const float sum = std::ldexp(1.0f, 15 + 16 + 8), lane = 32.0f;
    for (float state : tops) {
        float mul, s_back;
        range(state, kLeastExponent, mul, s_back);
        if (!(state < std::ldexp(1.0f, 58)))
            continue;
        for (float score : tops) {
            float back0;
            range(score, kLeastScoreExponent, mul, back0);
            const float f = s_back * value(inverse_power_bits(bits(back0)));
            CHECK(std::isfinite(sum * f * lane), "state %g, scores %g: factor %g", state, score, f);
            // 32 scores below 2^15 times FP16 values come to it in this tile's range
            const float first = sum * f + std::ldexp(1.0f, 15 + 16 + 5);
            if (!(score < std::ldexp(1.0f, 42)))            // q . k of 256 FP16 values is below 2^40
                continue;
            for (float next : tops) {
                float back1;
                range(next, kLeastScoreExponent, mul, back1);
                const float g = back0 * value(inverse_power_bits(bits(back1)));
                CHECK(std::isfinite(first * g * lane), "state %g, scores %g, %g: factor %g", state, score, next, g);
            }
        }
    }
    puts("ok");
    return 0;
}
