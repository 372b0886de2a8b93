// Powers of two that bring fp32 values into FP16's range for linear_attention.hip,
// free of HIP so that they are tested on the CPU too.
#pragma once

#ifdef __HIPCC__
#define SKINNY_SCALE __host__ __device__ __forceinline__
#else
#define SKINNY_SCALE inline
#endif

namespace skinny {

// Lowest fp32 exponent field that values are taken to have: as far down as the
// power for them is finite, and for the scores.  The output's sum is brought
// from the state's range into a score tile's, so the smaller the tile's power
// the larger that sum: a tile of zeros (keys of zero, padded tokens) with 2^-126
// overflowed it.  2^-40 is small enough: a score's rounding is then 2^-64 or
// less, 2^-42 of an output, whose own FP16 step is 2^-24 at least.
constexpr unsigned kLeastExponent = 15, kLeastScoreExponent = 101;

// `mul` brings values of at most `top` below 2^15, `back` is its inverse; all as
// the bits of fp32 values, top not negative.
SKINNY_SCALE void half_range_bits(unsigned top, unsigned least, unsigned &mul, unsigned &back)
{
    unsigned e = top >> 23;
    e = e < least ? least : (e > 254u ? 254u : e);
    mul = (268u - e) << 23;
    back = (e - 14u) << 23;
}

// 1 / p of a power of two between 2^-126 and 2^126
SKINNY_SCALE unsigned inverse_power_bits(unsigned p) { return (254u << 23) - p; }

}  // namespace skinny
