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

// Workgroups take the places in another order: block b < sequences the first
// part of sequence b, and block sequences + e the extra part e: sequence i has
// those from starts[i] / size on, as many as it has parts less one.  The parts
// that are surely there come first, so that they fill the chip evenly; most of
// the extra ones may be empty (16 prompts of 700 tokens, 12 heads, the places
// in their own order: 36 of 192 workgroups on one XCD of 32 CUs, 121 against
// 66 us).  A sequence of more than j whole parts ends past starts / size + j,
// where the next one's extra parts begin, so the sequence of extra part e is
// the last one with starts / size <= e.
SKINNY_HD bool extra_starts_by(int start, int tokens, int size, int extra)
{
    return cut_to(start, 0, tokens) / size <= extra;
}

// Place of block b, `seq` being b or the extra part's sequence.
SKINNY_HD int block_place(int start, int tokens, int size, int sequences, int block, int seq)
{
    return block < sequences ? first_place(start, tokens, size, block) : block - sequences + 1 + seq;
}

// States in the workspace.  A sequence in several parts has one for its start
// and one for every later part: what the part before it adds, then the state it
// starts from.  The later parts' lie in the order of the extra parts, tokens /
// size of them whatever the sequences; the starts', behind them, by sequence, or
// by their sequence's first extra part, whichever are fewer.  No other sequence
// has a state here.
SKINNY_HD int extra_states(int tokens, int size) { return tokens / size; }

SKINNY_HD int start_states(int tokens, int size, int sequences)
{
    return sequences < extra_states(tokens, size) ? sequences : extra_states(tokens, size);
}

// Of part `part` >= 1 of a sequence in several.
SKINNY_HD int part_state(int start, int tokens, int size, int part) { return cut_to(start, 0, tokens) / size + part - 1; }

// Of the start of sequence `seq`, among the starts'.
SKINNY_HD int start_state(int start, int tokens, int size, int sequences, int seq)
{
    return sequences < extra_states(tokens, size) ? seq : cut_to(start, 0, tokens) / size;
}

}  // namespace skinny
