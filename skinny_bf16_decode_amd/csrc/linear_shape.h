// How a prompt of linear_attention.hip is cut into parts and workgroups, from
// its sizes alone: host code without HIP, so that it is tested without it too.
#pragma once

#include "linear_places.h"

namespace skinny {

constexpr int kChunk = 64;

// Launch shape of a prompt, from its sizes alone.
struct Shape {
    int cols, col_tiles, part, places, multi;
    int eight;                  // eight waves of 16 columns, one workgroup a CU, in place of four of 32
};

// Workgroups the chip runs at once, two on each of 256 CUs: what the widest form
// holds.  It stands for all (four waves at dk <= 64 fit three, eight waves one or two).
constexpr int kSlots = 512;
constexpr int kOnePass = 384;   // tokens up to which nothing is done in parts

// Tokens of a part, for workgroups of `cols` columns.  The average is all that
// the host knows of the lengths.
inline int part_of(int tokens, int sequences, int heads, int dv, int cols)
{
    const long long columns = (long long)heads * ((dv + cols - 1) / cols), count = sequences > 0 ? sequences : 1;
    const long long average = ((long long)tokens + count - 1) / count;
    // as many parts as run at once, the same number for every sequence of the average length
    const long long units = columns * count, per_sequence = units < kSlots ? kSlots / units : 1;
    const long long even = ((average + per_sequence - 1) / per_sequence + kChunk - 1) / kChunk * kChunk;
    // none shorter than 192 tokens, or 256 where those do not all run at once: parts are done twice.  While there
    // are CUs left, of 64 tokens, since a lone workgroup waits most of a chunk's 5 us (8 sequences, 1720 tokens, two
    // heads of 128: parts of 64, 128, 256 24, 27, 37 us).  Where sequences are short, only the far longer ones are
    // cut, for every part that a launch has room for costs time (1000 sequences of 70 tokens, 12 heads, dk 64: parts
    // of 64, 192, 384 780, 721, 663 us; with one of 1200 tokens among 41, two heads, 23, 26, 38 us)
    const auto fits = [&](int part, int most) { return columns * (tokens / part + count) <= most; };
    const int least = average < 80 ? kOnePass : fits(64, 160) ? 64 : fits(192, kSlots) ? 192 : 256;
    return (int)(even > least ? even : least);
}

inline Shape shape_of(int tokens, int sequences, int heads, int dk, int dv)
{
    Shape s;
    // 128 columns a workgroup, or 64: where there are no more, or a last tile would be half empty; where the
    // wide ones leave many CUs with one workgroup or none (1000 tokens, 12 heads of 128: 35 against 42 us); and where
    // that makes enough workgroups of whole sequences, of which no part is done twice (20 of 3000 tokens, 12 heads,
    // dk 64: 211 against 308 us), unless they are so long that uneven ones leave CUs idle (20 of 7000 in the mean,
    // uneven: 765 against 664 us)
    const int part = part_of(tokens, sequences, heads, dv, 128);
    const long long wide = (dv + 127) / 128, narrow = (dv + 63) / 64, parts = tokens / part;
    const bool few = heads * wide * (parts > sequences ? parts : sequences) <= 300;
    const bool whole = heads * wide * sequences <= 300 && heads * narrow * sequences >= 3 * kSlots / 4 &&
                       (long long)tokens <= 4096LL * sequences;
    // 64 < dk <= 128: one workgroup of eight waves a CU, sequences uncut, where there are that many and few more
    // (12 heads of 128, 16 prompts of 2048 tokens: 168 against 195 us); two of four waves a CU past that, which wait
    // less in all (24 prompts: 274 against 317 us).  Fewer leave CUs idle (8 of 2048 tokens: 151 against 120 us),
    // which short ones make up for (8 of 380: 39 against 47 us); long ones may be too uneven (16 of 6000: 707
    // against 576 us with lengths within 30 %, but 461 against 517 with equal ones, and the host knows neither)
    const long long units = heads * wide * sequences, average = sequences > 0 ? tokens / sequences : 0;
    const bool middle = dk > 64 && dk <= 128 && dv > 64 && (dv <= 128 || dv > 192);
    s.eight = middle && units <= kSlots / 2 && average <= 4096 && (units >= 128 || (units >= 96 && average <= 384));
    const bool many = middle && units > kSlots / 2;
    s.cols = dv <= 64 || (dv > 128 && dv <= 192) || ((few || whole) && !s.eight && !many) ? 64 : 128;
    s.col_tiles = (dv + s.cols - 1) / s.cols;
    s.part = s.cols == 128 ? part : part_of(tokens, sequences, heads, dv, 64);
    if (s.eight)                                // room for lengths about the average
        s.part = (int)((average + average / 8) / kChunk + 1) * kChunk;
    s.multi = tokens > kOnePass && s.part < tokens;
    if (!s.multi)                               // past every start: sequence i is place i
        s.part = (tokens / kChunk + 1) * kChunk;
    s.places = tokens / s.part + sequences;
    return s;
}

// Parts past their sequences' first that any prompt of at most so many tokens
// and sequences has room for: what a workspace is sized by, so that one for a
// caller's largest prompt serves all smaller ones.  A part is kChunk tokens at
// least; with fewer than kSlots workgroups of whole sequences there are at most
// kSlots parts' in all; else a part is 256 tokens at least, and the average
// sequence one part.
inline int most_extra_parts(int tokens, int sequences, int heads, int dv)
{
    const long long columns = (long long)heads * ((dv + 127) / 128);
    const int few = cut_to(tokens / kChunk, 0, (int)(kSlots / columns)), many = cut_to(tokens / 256, 0, sequences);
    return few > many ? few : many;
}

}  // namespace skinny
