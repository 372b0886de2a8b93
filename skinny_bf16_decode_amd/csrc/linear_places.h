// Where the parts of packed sequences lie: the arithmetic that the prompt
// kernels of linear_attention.hip address memory with, free of HIP so that it
// is tested on the CPU too.
#pragma once

#ifdef __HIPCC__
#define SKINNY_HD __host__ __device__ __forceinline__
#else
#define SKINNY_HD inline
#endif

namespace skinny {

// Part `part` of a sequence: the sequence's first token and length.
struct Place {
    int seq, part, first, len;
};

SKINNY_HD int cut_to(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Sequence i holds the places from starts[i] / size + i on.  It has at most
// floor(end / size) - floor(start / size) + 1 parts of `size` tokens, so
// sequences do not overlap, and tokens / size + sequences places are enough
// whatever the lengths: a grid follows from the token count alone.
SKINNY_HD int first_place(int start, int tokens, int size, int seq) { return cut_to(start, 0, tokens) / size + seq; }

// Parts of a sequence of `len` tokens (one for an empty sequence, which still
// has a state to pass on).
SKINNY_HD int parts_of(int len, int size) { return len == 0 ? 1 : (len - 1) / size + 1; }

// Place `place` of sequence `seq` with the token range start .. end; false if
// the sequence has no such part.  Any integers are safe as starts: they are cut
// to 0 <= start <= end <= tokens.
SKINNY_HD bool place_of(int start, int end, int tokens, int size, int place, int seq, Place &p)
{
    const int s = cut_to(start, 0, tokens), e = cut_to(end, s, tokens);
    p.seq = seq;
    p.first = s;
    p.len = e - s;
    p.part = place - first_place(start, tokens, size, seq);
    return p.part >= 0 && p.part < parts_of(p.len, size);
}

}  // namespace skinny
