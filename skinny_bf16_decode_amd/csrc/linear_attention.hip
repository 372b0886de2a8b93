// HIP kernels and entry points of linear attention with a decay for each head
// and token, for gfx950 (CDNA4):
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T        S [dk][dv], fp32
//   o_t = scale q_t^T S_t
//
// for every value head, over packed sequences (prompt) or one new token of
// each sequence (step).
//
// The prompt works in chunks of 64 tokens.  With G_t the sum of the log decays
// of a chunk through token t and S the state before it,
//
//   o_t   = scale (exp(G_t) q_t^T S + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s)
//   S_new = exp(G_63) S + sum_s k_s (exp(G_63 - G_s) v_s)^T
//
// which are four matrix products a chunk.  A workgroup of four or eight waves
// walks the chunks of one (sequence part, head, 64 or 128 value columns); each
// wave keeps the state of its own 16 or 32 columns in registers, in the result layout
// of the 16x16x32 MFMA, from one chunk to the next.
#include <hip/hip_runtime.h>

#include <atomic>
#include <stdarg.h>
#include <stdio.h>

#include "linear_places.h"
#include "linear_scales.h"
#include "linear_shape.h"
#include "skinny_internal.h"

namespace skinny {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

constexpr int kThreads = 256;

// Kernel arguments.  Strides are in elements.
struct LArgs {
    const void *q, *k, *v;
    void *out;
    const float *g;
    const float *state_in;
    float *state_out;
    const int *starts;          // prompt: [sequences + 1]
    const int *slots;           // [sequences], or NULL: sequence i holds slot i
    // prompt in parts, see the states of linear_places.h
    float *ws_part;             // [later part][head][dk][dv]
    float *ws_start;            // [start][head][dk][dv]
    double *ws_decay;           // [later part][head], sums of log2 decays of the part before
    int *ws_serial;             // [start][head], the part from which on the sequence is taken in one go
    long long q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head, g_token, g_head;
    long long in_slot, in_head, so_slot, so_head;
    int tokens, sequences, heads, share, dk, dv, pool;
    int part;                   // tokens of a part of a sequence, a multiple of 64
    int places;                 // parts a launch provides for
    int col_tiles;              // workgroups along dv
    int groups;                 // key heads of all places
    int runs;                   // consecutive groups on one XCD
    int multi;                  // a sequence may have more than one part
    float scale;
};

template <bool H>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (H)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
}

// One 16-bit value of an LDS tile or of a register half, as fp32.
template <bool H>
__device__ __forceinline__ float to_float(unsigned short bits)
{
    if constexpr (H)
        return (float)__builtin_bit_cast(_Float16, bits);
    else
        return __uint_as_float((unsigned)bits << 16);
}

template <bool H>
__device__ __forceinline__ unsigned short to_bits(float v)
{
    if constexpr (H)
        return __builtin_bit_cast(unsigned short, (_Float16)v);
    else
        return __builtin_bit_cast(unsigned short, (__bf16)v);
}

template <bool H>
__device__ __forceinline__ unsigned int pack2(float a, float b)
{
    if constexpr (H) {
        typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
        return __builtin_bit_cast(unsigned int, f16x2{(_Float16)a, (_Float16)b});
    } else {
        typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
        return __builtin_bit_cast(unsigned int, bf16x2{(__bf16)a, (__bf16)b});
    }
}

template <bool H>
__device__ __forceinline__ void unpack2(unsigned int w, float &lo, float &hi)
{
    lo = to_float<H>((unsigned short)(w & 0xFFFFu));
    hi = to_float<H>((unsigned short)(w >> 16));
}

// 16-bit terms of an fp32 operand of a matrix product.  Three BF16 terms (8 bits
// and a sign each) hold all 24 bits.  With two, 17 bits, what cancellation left
// of a sum over the state was off by 2.5e-6 of the terms' size, 35 times as far
// as in a step, which multiplies in fp32 (prompts 5 to 11 % longer with three:
// 16 of 2048 tokens 152 -> 167 us).  Two FP16 terms hold 22 bits, and that sum is
// off by 1.1e-7, against a step's 0.7e-7; a third made FP16 prompts 9 to 14 %
// longer for little more, and is not taken.
template <bool H>
constexpr int kTerms = H ? 2 : 3;

// Two fp32 values as the sum of kTerms pairs of 16-bit values, each term the
// rounded rest, which is exact.  FP16 terms (the caller scales into their range,
// see half_range) are cut off, the form that takes two values at once.
template <bool H>
__device__ __forceinline__ void split2(float a, float b, unsigned int (&w)[kTerms<H>])
{
#pragma unroll
    for (int i = 0; i < kTerms<H>; ++i) {
        if constexpr (H) {
            const auto p = __builtin_amdgcn_cvt_pkrtz(a, b);
            w[i] = __builtin_bit_cast(unsigned int, p);
            if (i + 1 < kTerms<H>) {
                a -= (float)p[0];
                b -= (float)p[1];
            }
        } else {
            typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
            const bf16x2 p = {(__bf16)a, (__bf16)b};
            w[i] = __builtin_bit_cast(unsigned int, p);
            if (i + 1 < kTerms<H>) {
                asm("" : "+v"(w[i]));       // else the low half is rounded a second time, alone
                a -= __uint_as_float(w[i] << 16);
                b -= __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
}

// Eight fp32 values into kTerms MFMA operands.
template <bool H>
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&f)[kTerms<H>])
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        unsigned int w[kTerms<H>];
        split2<H>(x[2 * p], x[2 * p + 1], w);
#pragma unroll
        for (int i = 0; i < kTerms<H>; ++i)
            f[i][p] = w[i];
    }
}

// Largest value over the four lanes of one column, l % 16 (values >= 0; NaN is passed over).
__device__ __forceinline__ float column_max(float x)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Value of the column that lane group g's result row r belongs to, lane 4 g + r of 16.
__device__ __forceinline__ float of_row(float x, int r)
{
    int first = 4 * (4 * ((threadIdx.x & 63) >> 4));
    asm volatile("" : "+v"(first));             // one address kept over the chunks, not one for every r
    return __uint_as_float(__builtin_amdgcn_ds_bpermute(first + 4 * r, __float_as_uint(x)));
}

// See linear_scales.h.  An FP16 split of the scaled values, two terms cut off, is good to 2^-21 of a value, and to
// 2^-38 of `top` where the value is far smaller (FP16's subnormal step, 2^-24, against 2^14).  So the power is one for
// each sum that the values enter -- a value column, a token's scores of one tile -- and not one for several, of which
// the smaller would lose its bits to the larger.
__device__ __forceinline__ void half_range(float top, unsigned least, float &mul, float &back)
{
    unsigned m, b;
    half_range_bits(__float_as_uint(top), least, m, b);
    mul = __uint_as_float(m);
    back = __uint_as_float(b);
}

__device__ __forceinline__ float inverse_power(float p)
{
    return __uint_as_float(inverse_power_bits(__float_as_uint(p)));
}

// Whether any lane of the wave saw a value that is not finite: acc gathers x * 0.
__device__ __forceinline__ bool wave_any_nan(float acc) { return __ballot(acc != 0.0f) != 0ull; }

// The place of a workgroup, see linear_places.h; false if it is empty.
__device__ __forceinline__ bool locate(const LArgs &a, int block, Place &p)
{
    int seq = block;
    if (block >= a.sequences) {
        const int lane = threadIdx.x & 63;
        int count = 0;
        for (int i0 = 0; i0 < a.sequences; i0 += 64) {
            const int i = i0 + lane;
            bool by = false;
            if (i < a.sequences)
                by = extra_starts_by(a.starts[i], a.tokens, a.part, block - a.sequences);
            count += __popcll(__ballot(by));
        }
        if (count == 0)
            return false;
        seq = __builtin_amdgcn_readfirstlane(count - 1);
    }
    const int place = block_place(a.starts[seq], a.tokens, a.part, a.sequences, block, seq);
    return place_of(a.starts[seq], a.starts[seq + 1], a.tokens, a.part, place, seq, p);
}

// Slot of a sequence, or -1 where the pool has none of that number.
__device__ __forceinline__ int slot_of(const LArgs &a, int seq)
{
    const int s = a.slots ? a.slots[seq] : seq;
    return s >= 0 && s < a.pool ? s : -1;
}

// A buffer load whose offset is past its resource reads zero and touches no
// memory, a store writes none: rows and columns to be left out take kSkip as
// their offset, so that loads and stores need no branches.  Offsets inside a
// chunk stay below it: 63 rows at strides below 2^24 elements of 2 bytes.
constexpr unsigned kSkip = 0x7FF00000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)kSkip, 0x00020000);
}

// k is read by rows (scores) and, transposed, by columns (states), both without
// bank conflicts: in row r, 16-byte unit u lies at u ^ h(r), so that sixteen
// rows of one unit, and eight rows of two, fall on all 64 banks (a row of 128
// bytes, pitch 64, covers half of them).  Byte offset of column c of row r; the
// row pitch is a multiple of 128 bytes, so that columns can be XORed in.
__device__ __forceinline__ unsigned key_address(int pitch, int r, int c)
{
    const unsigned h = (pitch >= 128 ? 2 * (r & 7) : 2 * ((r >> 1) & 3)) + ((r >> 3) & 1);
    return (unsigned)(r * pitch) * 2 + ((((unsigned)c >> 3) ^ h) << 4) + ((unsigned)c & 7) * 2;
}

// A tile of 64 token rows of COLS 16-bit columns on its way from global memory
// through registers to LDS.  Rows from `rows` on and columns from `cols` on
// are zero.
template <int COLS, int THREADS>
struct Tile {
    static constexpr int kPerRow = COLS / 8;
    static constexpr int kVecs = (kChunk * kPerRow + THREADS - 1) / THREADS;
    static constexpr int kRowStep = THREADS / kPerRow;
    u32x4 r[kVecs];
    unsigned off, step;         // byte offset of the first vector, bytes between vectors

    __device__ __forceinline__ void init(long long stride, int cols)
    {
        const int row = threadIdx.x / kPerRow, col = (threadIdx.x % kPerRow) * 8;
        off = col < cols ? (unsigned)row * (unsigned)(2 * stride) + 2 * col : kSkip;
        step = kRowStep * (unsigned)(2 * stride);
    }

    __device__ __forceinline__ void load(const unsigned short *base, int rows)
    {
        const __amdgpu_buffer_rsrc_t src = make_rsrc(base);
        const int row = threadIdx.x / kPerRow;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(src, row + i * kRowStep < rows ? off : kSkip, i * step, 0);
        }
    }

    __device__ __forceinline__ void store(unsigned short *lds, int pitch) const
    {
        const int row = threadIdx.x / kPerRow, col = (threadIdx.x % kPerRow) * 8;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (kRowStep <= kChunk || row < kChunk)     // more threads than vectors
                *reinterpret_cast<u32x4 *>(lds + (row + i * kRowStep) * pitch + col) = r[i];
    }

    // Columns where key_address has them.
    __device__ __forceinline__ void store_keys(unsigned short *lds, int pitch) const
    {
        const int row = threadIdx.x / kPerRow, col = (threadIdx.x % kPerRow) * 8;
        char *base = reinterpret_cast<char *>(lds);
        const unsigned at = key_address(pitch, row, col);   // kRowStep is a multiple of 8: h differs by its last bit
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (kRowStep <= kChunk || row < kChunk)
                *reinterpret_cast<u32x4 *>(base + (at ^ (((i * kRowStep >> 3) & 1) << 4)) + i * kRowStep * pitch * 2) =
                    r[i];
    }

    // Columns in the order of operand_position.
    __device__ __forceinline__ void store_operands(unsigned short *lds, int pitch) const
    {
        const int row = threadIdx.x / kPerRow, col = (threadIdx.x % kPerRow) * 8;
        unsigned short *at = lds + row * pitch + (col & ~31) + 2 * (col & 8) + ((col >> 2) & 4);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (kRowStep <= kChunk || row < kChunk) {
                *reinterpret_cast<u32x2 *>(at + i * kRowStep * pitch) = u32x2{r[i].x, r[i].y};
                *reinterpret_cast<u32x2 *>(at + i * kRowStep * pitch + 8) = u32x2{r[i].z, r[i].w};
            }
    }
};

// Position in an LDS row of q of column c: within 32 columns, the four
// 16 h + 4 g + 0..3 lie at 8 g + 4 h, the order of the MFMA operand below, so
// that it is one 16-byte read.
__device__ __forceinline__ int operand_position(int c)
{
    return (c & ~31) + 8 * ((c >> 2) & 3) + 4 * ((c >> 4) & 1) + (c & 3);
}

// MFMA operand from 16 token rows of q as stored by store_operands.
__device__ __forceinline__ u32x4 query_operand(const unsigned short *lds, int pitch, int row0, int j)
{
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const u32x4 *>(lds + (row0 + (lane & 15)) * pitch + 32 * j + 8 * (lane >> 4));
}

template <typename T>
__device__ __forceinline__ const T *at_byte(const unsigned short *lds, unsigned off)
{
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(lds) + off);
}

// MFMA operand from 16 rows of k: lane (row l % 16) holds columns
// 32 j + 4 (l / 16) + 0..3 and the 4 columns 16 further on, the order in
// which the state's result registers hold dk.
__device__ __forceinline__ u32x4 key_row_operand(const unsigned short *lds, int pitch, int row0, int j)
{
    const int lane = threadIdx.x & 63;
    unsigned off = key_address(pitch, lane & 15, 4 * (lane >> 4));      // row0: a multiple of 16
    asm volatile("" : "+v"(off));               // one address kept over the chunks, not one for every j
    off ^= 64 * j;
    const u32x2 a = *at_byte<u32x2>(lds + row0 * pitch, off), b = *at_byte<u32x2>(lds + row0 * pitch, off ^ 32);
    return u32x4{a.x, a.y, b.x, b.y};
}

// The same of 16 columns over the 32 tokens 32 j.., see column_operand.
__device__ __forceinline__ u32x4 key_column_operand(const unsigned short *lds, int pitch, int col0, int j)
{
    const int lane = threadIdx.x & 63, in = lane & 15;
    unsigned off = key_address(pitch, 4 * (lane >> 4) + (in >> 2), 4 * (in & 3));
    asm volatile("" : "+v"(off));
    off ^= 2 * col0;
    const unsigned short *p = at_byte<unsigned short>(lds + 32 * j * pitch, off);
    typedef __attribute__((address_space(3))) s16x4 *lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 16 * pitch));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x.x, x.y, y.x, y.y};
}

// Column, among the wave's 16 NV, of MFMA column m of its group n.  Two groups
// are interleaved by fours, so that a lane's results of both, rows 4 g .. 4 g + 3
// of the transposed output, are eight columns in a row: one 16-byte store.
template <int NV>
__device__ __forceinline__ int value_column(int n, int m)
{
    return NV == 2 ? 8 * (m >> 2) + 4 * n + (m & 3) : m;
}

// MFMA operand from column group n of v over the 32 tokens 32 j..: lane (column l % 16)
// holds tokens 32 j + 4 (l / 16) + 0..3 and the 4 tokens 16 further on.  The
// transposing LDS read gives each lane of 16 four rows of its own column.
template <int NV>
__device__ __forceinline__ u32x4 column_operand(const unsigned short *lds, int pitch, int n, int j)
{
    const int lane = threadIdx.x & 63, in = lane & 15;
    const unsigned short *p = lds + (32 * j + 4 * (lane >> 4) + (in >> 2)) * pitch + value_column<NV>(n, 4 * (in & 3));
    typedef __attribute__((address_space(3))) s16x4 *lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 16 * pitch));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x.x, x.y, y.x, y.y};
}

// Per-token decay values of a chunk, in LDS.
struct alignas(16) Decays {
    float hi[kChunk], lo[kChunk];   // G_t log2 e as a sum of two fp32 values
    float grown[kChunk];            // exp(G_t)
    float rest[kChunk];             // exp(G_63 - G_t)
    float own[kChunk];              // exp(g_t)
    float total;                    // exp(G_63)
};

// One wave: lane t has g_t (0 past the end).  Sums are in 64 bits, so that the
// differences of far-decayed chunks keep their bits.  Finite sums are wanted
// of -inf too: -200 gives 0 as well.  NaN stays.
__device__ __forceinline__ double chunk_decays(float g, Decays &d)
{
    const int lane = threadIdx.x & 63;
    double x = (double)(g < -200.0f ? -200.0f : g) * 1.44269504088896340736;
    const float own = (float)x;
#pragma unroll
    for (int step = 1; step < 64; step *= 2) {
        const double y = __shfl_up(x, step, 64);
        if (lane >= step)
            x += y;
    }
    const double all = __shfl(x, 63, 64);
    const float hi = (float)x;
    d.hi[lane] = hi;
    d.lo[lane] = (float)(x - (double)hi);
    d.grown[lane] = __builtin_amdgcn_exp2f(hi);
    d.rest[lane] = __builtin_amdgcn_exp2f((float)(all - x));
    d.own[lane] = __builtin_amdgcn_exp2f(own);
    if (lane == 63)
        d.total = __builtin_amdgcn_exp2f(hi);
    return all;
}

// The (t-tile, 32-token step) operands of the masked scores that the causal
// mask leaves: tiles 0 and 1 have one, 2 and 3 two.
__device__ __host__ constexpr int score_slot(int tile, int j) { return (tile < 2 ? tile : 2 * tile - 2) + j; }
constexpr int kScoreSlots = 6;

template <int DK, int WAVES, int NV, bool OUT>
struct Layout {
    static constexpr int kCols = 16 * WAVES * NV;    // value columns of a workgroup
    static constexpr int kQPitch = DK + 8;      // row reads: 16 rows x 16 bytes on all banks
    static constexpr int kKPitch = DK < 64 ? 64 : DK;   // swizzled, see key_address
    static constexpr int kVPitch = kCols + 16;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + (OUT ? kChunk * kQPitch * 2 : 0);
    static constexpr int kV = kK + kChunk * kKPitch * 2;
    static constexpr int kScores = kV + kChunk * kVPitch * 2;
    static constexpr int kBytes = kScores + (OUT ? kScoreSlots * 3 * 64 * 16 : 0);
};

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The recurrence token by token, as it is defined, for one wave's columns of a
// chunk in LDS, its state in memory (T, laid out like the registers): used
// where a value is not finite, since 0 * inf in a product over masked tokens, or in a split into
// terms, would spread NaN to outputs that the definition leaves alone.  A wave
// that has come here stays here for the rest of its part, and carries the
// state in registers along unused: merging the two would cost every wave a
// second copy of it.
template <bool H, int DK, int WAVES, int NV, bool OUT>
__device__ __forceinline__ void recur(const LArgs &a, const unsigned short *lds, const Decays &d, int rows, f32x4 *T,
                                      unsigned short *out, int col0)
{
    using L = Layout<DK, WAVES, NV, OUT>;
    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4;
    const unsigned short *qs = lds + L::kQ / 2, *ks = lds + L::kK / 2, *vs = lds + L::kV / 2;
#pragma unroll 1
    for (int nt = 0; nt < rows * NV; ++nt) {
        const int n = nt / rows, t = nt - n * rows;     // one column group after the other
        const float e = d.own[t], v = to_float<H>(vs[t * L::kVPitch + 16 * NV * wave + value_column<NV>(n, lane & 15)]);
        float o = 0.0f;
#pragma unroll 1
        for (int i = 0; i < DK / 16; ++i) {
            f32x4 S = T[n * (DK / 16) + i];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = 16 * i + 4 * g + r;
                const float k = to_float<H>(ks[key_address(L::kKPitch, t, c) / 2]);
                // rows past dk hold no state: 0 * a v that is not finite is not theirs to add
                const float s = c < a.dk ? S[r] * e + k * v : 0.0f;
                S[r] = s;
                if constexpr (OUT)
                    o += c < a.dk ? to_float<H>(qs[t * L::kQPitch + operand_position(c)]) * s : 0.0f;
            }
            T[n * (DK / 16) + i] = S;
        }
        if constexpr (OUT) {
            o += __shfl_xor(o, 16, 64);
            o += __shfl_xor(o, 32, 64);
            const int c = col0 + 16 * NV * wave + value_column<NV>(n, lane & 15);
            if (g == 0 && c < a.dv)
                out[t * a.out_token + c] = to_bits<H>(o * a.scale);
        }
    }
}

// Natural [dk][dv] state <-> result registers of the wave's columns.  Lane
// group g holds rows 4 g .. 4 g + 3 of each 16; dk is a multiple of 8, so the
// four are all in or all out.
__device__ __forceinline__ unsigned state_offset(const LArgs &a, int c)
{
    const int lane = threadIdx.x & 63;
    return c < a.dv ? 4u * (lane >> 4) * 4u * (unsigned)a.dv + 4u * c : kSkip;
}

// c: the lane's column, of one of the wave's groups.
template <int DK>
__device__ __forceinline__ void load_state(const LArgs &a, const float *p, int c, f32x4 (&S)[DK / 16])
{
    const __amdgpu_buffer_rsrc_t src = make_rsrc(p);
    const unsigned off = p ? state_offset(a, c) : kSkip;
    const int row = 4 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int i = 0; i < DK / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[i][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                src, 16 * i + row < a.dk ? off : kSkip, (unsigned)(16 * i + r) * 4u * (unsigned)a.dv, 0));
}

template <int DK>
__device__ __forceinline__ void store_state(const LArgs &a, float *p, int c, const f32x4 (&S)[DK / 16])
{
    const __amdgpu_buffer_rsrc_t dst = make_rsrc(p);
    const unsigned off = state_offset(a, c);
    const int row = 4 * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int i = 0; i < DK / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), dst, 16 * i + row < a.dk ? off : kSkip,
                                                  (unsigned)(16 * i + r) * 4u * (unsigned)a.dv, 0);
}

// The wave's columns of v over the tokens of step j, each times exp(G_63 - G_s).
template <bool H>
__device__ __forceinline__ void decayed_values(u32x4 v, const Decays &d, int j, float (&x)[8])
{
    const int g = (threadIdx.x & 63) >> 4;
    const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&d.rest[32 * j + 4 * g]);
    const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&d.rest[32 * j + 16 + 4 * g]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float lo, hi;
        const unsigned int w = v[p];
        unpack2<H>(w, lo, hi);
        x[2 * p] = lo * (p < 2 ? w0[2 * p] : w1[2 * p - 4]);
        x[2 * p + 1] = hi * (p < 2 ? w0[2 * p + 1] : w1[2 * p - 3]);
    }
}

// S = exp(G_63) S + sum_s k_s (exp(G_63 - G_s) v_s)^T over the chunk in LDS.
// k is exact in 16 bits; the decayed v is fp32 and goes in as kTerms.
template <bool H, int DK, int WAVES, int NV, bool OUT>
__device__ __forceinline__ void update_state(const unsigned short *lds, const Decays &d, f32x4 (&S)[NV][DK / 16])
{
    using L = Layout<DK, WAVES, NV, OUT>;
    const unsigned short *ks = lds + L::kK / 2, *vs = lds + L::kV / 2 + 16 * NV * wave_id();
    const float total = d.total;
    u32x4 f[NV][2][kTerms<H>];
    float back[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float x[2][8];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            decayed_values<H>(column_operand<NV>(vs, L::kVPitch, n, j), d, j, x[j]);
        if constexpr (H) {
            float top = 0.0f, mul;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    top = fmaxf(top, fabsf(x[j][p]));
            half_range(column_max(top), kLeastExponent, mul, back[n]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    x[j][p] *= mul;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            split8<H>(x[j], f[n][j]);
    }
    u32x4 k[2][2];                              // of this row tile and the next
#pragma unroll
    for (int j = 0; j < 2; ++j)
        k[0][j] = key_column_operand(ks, L::kKPitch, 0, j);
#pragma unroll
    for (int i = 0; i < DK / 16; ++i) {
        if (i + 1 < DK / 16) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                k[(i + 1) & 1][j] = key_column_operand(ks, L::kKPitch, 16 * (i + 1), j);
        }
        __builtin_amdgcn_sched_barrier(0);
        f32x4 add[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if constexpr (H) {
                add[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[n][i][r] *= total;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int m = 0; m < kTerms<H>; ++m)
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    if constexpr (H)
                        add[n] = mma16<H>(k[i & 1][j], f[n][j][m], add[n]);
                    else
                        S[n][i] = mma16<H>(k[i & 1][j], f[n][j][m], S[n][i]);
                }
        if constexpr (H) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[n][i][r] = S[n][i][r] * total + add[n][r] * back[n];
        }
    }
}

// One part of a sequence for one head and 16 WAVES NV value columns, 16 NV a wave.
// Bound by the waits of a chunk's four products, one after the other with three
// barriers between: 5 to 6 us a chunk alone on a CU at dk = dv = 128, the matrix
// units busy for a third of it and the vector units for two fifths (BF16, 32768
// tokens of 12 heads: 65 us for the parts' own states, 132 us for the outputs,
// against 85 us for the bytes; 16 sequences of 2048 tokens, whole: 159 us).
// OUT: outputs, and the sequence's new state after its last part.  Otherwise:
// what the part alone adds to the state, for the parts after it.
// Registers for two waves a SIMD; for one where LDS holds one workgroup a CU and
// that has four waves (dk = 256: with two it spilled 5 registers).
template <bool H, int DK, int WAVES, int NV, bool OUT>
__global__ __launch_bounds__(64 * WAVES, DK == 256 && WAVES == 4 && OUT ? 1 : 2) void linear_chunks(LArgs a)
{
    using L = Layout<DK, WAVES, NV, OUT>;
    constexpr int kGateWave = WAVES == 8 ? 7 : 2;   // it has the least of the scores to do
    extern __shared__ __align__(16) unsigned short lds[];
    __shared__ Decays decays[2];
    __shared__ float score_back[4][2][16];
    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4;
    unsigned short *qs = lds + L::kQ / 2, *ks = lds + L::kK / 2, *vs = lds + L::kV / 2;
    u32x4 *scores = reinterpret_cast<u32x4 *>(lds + L::kScores / 2);

    // the workgroups that share keys -- the column tiles of a head, the heads of a key head -- on one XCD, whose
    // L2 then serves their common q and k.  The next such group is on the next XCD, since the last ones may be
    // empty, or on the same one, where few can be (see a.runs)
    const unsigned xcd = blockIdx.x & 7u, turn = blockIdx.x >> 3, of_group = (unsigned)(a.share * a.col_tiles);
    const unsigned nth = turn / of_group;
    const unsigned group = a.runs ? xcd * (((unsigned)a.groups + 7u) / 8u) + nth : nth * 8u + xcd;
    if (group >= (unsigned)a.groups)
        return;
    const unsigned id = group * of_group + (turn - nth * of_group);
    const int tile = (int)(id % (unsigned)a.col_tiles);
    const unsigned hp = id / (unsigned)a.col_tiles;
    const int head = (int)(hp % (unsigned)a.heads), block = (int)(hp / (unsigned)a.heads);

    Place p;
    if (!locate(a, block, p))
        return;
    const int parts = parts_of(p.len, a.part);
    if (!OUT && p.part == parts - 1)
        return;                                 // nothing follows it
    const int t0 = p.part * a.part;
    int n_tok = min(p.len - t0, a.part);
    bool last = p.part == parts - 1;
    // of the sequence's start, and of the part after this one; used where there are several parts
    const long long start_at = (long long)start_state(p.first, a.tokens, a.part, a.sequences, p.seq) * a.heads + head;
    const long long next_at = (long long)part_state(p.first, a.tokens, a.part, p.part + 1) * a.heads + head;
    if (OUT && a.multi && parts > 1) {
        // a join that is no sum (see linear_join): the part before it goes on to the end
        const int serial = a.ws_serial[start_at];
        if (serial < p.part)
            return;
        if (serial == p.part) {
            n_tok = p.len - t0;
            last = true;
        }
    }
    const int chunks = (n_tok + kChunk - 1) / kChunk;
    const int col0 = tile * L::kCols, cols = min(a.dv - col0, L::kCols);
    const int khead = head / a.share;
    const int slot = slot_of(a, p.seq);

    const long long tok = (long long)p.first + t0;
    const unsigned short *qp = static_cast<const unsigned short *>(a.q) + tok * a.q_token + khead * a.q_head;
    const unsigned short *kp = static_cast<const unsigned short *>(a.k) + tok * a.k_token + khead * a.k_head;
    const unsigned short *vp = static_cast<const unsigned short *>(a.v) + tok * a.v_token + head * a.v_head + col0;
    const float *gp = a.g + tok * a.g_token + head * a.g_head;
    unsigned short *op = static_cast<unsigned short *>(a.out) + tok * a.out_token + head * a.out_head;
    const unsigned out_step = (unsigned)(2 * a.out_token);
    const int wave_col = col0 + 16 * NV * wave;
    const int out_col = wave_col + 4 * NV * g;  // dv is a multiple of 8: 4 NV columns are all in or all out
    const unsigned out_off = out_col < a.dv ? (lane & 15) * out_step + 2 * out_col : kSkip;

    f32x4 S[NV][DK / 16];
    f32x4 memory[NV * (DK / 16)], *T = memory;         // the state of a wave that goes token by token
    asm volatile("" : "+v"(T) : : "memory");    // an address of its own: not turned back into registers
    bool slow = false;
    if constexpr (OUT) {
        const float *from = nullptr;
        if (a.multi && parts > 1)
            from = p.part == 0 ? a.ws_start + start_at * a.dk * a.dv : a.ws_part + (next_at - a.heads) * a.dk * a.dv;
        else if (a.state_in && slot >= 0)
            from = a.state_in + slot * a.in_slot + head * a.in_head;
#pragma unroll
        for (int n = 0; n < NV; ++n)
            load_state<DK>(a, from, wave_col + value_column<NV>(n, lane & 15), S[n]);
    }

    // the parts-only kernel takes a second, token by token, pass if its state is not finite
    for (int attempt = 0; attempt < 2; ++attempt) {
        if constexpr (!OUT) {
#pragma unroll
            for (int i = 0; i < NV * (DK / 16); ++i) {
                T[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                S[i / (DK / 16)][i % (DK / 16)] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        Tile<DK, 64 * WAVES> tq, tk;
        Tile<L::kCols, 64 * WAVES> tv;
        tq.init(a.q_token, a.dk);
        tk.init(a.k_token, a.dk);
        tv.init(a.v_token, cols);
        double sum = 0.0;
        float gate = 0.0f;
        if (chunks > 0) {
            if constexpr (OUT)
                tq.load(qp, n_tok);
            tk.load(kp, n_tok);
            tv.load(vp, n_tok);
            if (wave == kGateWave) {
                gate = lane < n_tok ? gp[lane * a.g_token] : 0.0f;
                sum = chunk_decays(gate, decays[0]);
                gate = kChunk + lane < n_tok ? gp[(kChunk + lane) * a.g_token] : 0.0f;
            }
        }
        for (int c = 0; c < chunks; ++c) {
            const int rows = min(n_tok - c * kChunk, kChunk);
            const Decays &d = decays[c & 1];
            if constexpr (OUT)
                tq.store_operands(qs, L::kQPitch);
            tk.store_keys(ks, L::kKPitch);
            tv.store(vs, L::kVPitch);
            __syncthreads();
            // the next chunk, a tile at a time between the products: all at once they fill the CU's queue, and
            // the wave waits to issue them (2200 of 16700 cycles a chunk)
            const bool more = c + 1 < chunks;
            const long long at = (long long)(c + 1) * kChunk;
            const int left = n_tok - (c + 1) * kChunk;
            if (more) {
                tk.load(kp + at * a.k_token, left);
                if (wave == kGateWave) {
                    sum += chunk_decays(gate, decays[(c + 1) & 1]);
                    gate = kChunk + lane < left ? gp[(at + kChunk + lane) * a.g_token] : 0.0f;
                }
            }
            if constexpr (OUT) {
                // masked, decayed, scaled scores of 16 tokens t with the 32 tokens of step j: the six that the
                // causal mask leaves, (tile, step) 00 10 20 21 30 31, over the waves; of four, 0 and 1 have
                // three tiles of 16 tokens, 2 and 3 two
#pragma unroll
                for (int jj = 0; jj < (WAVES == 8 ? 1 : 2); ++jj) {
                    const int job = WAVES == 8 ? wave : (wave < 2 ? 2 * wave + jj : (jj ? 6 : 2 + wave));
                    if (job >= kScoreSlots)
                        continue;
                    const int tt = job < 2 ? job : (job + 2) >> 1, j = job < 2 ? 0 : job & 1;
                    u32x4 qf[DK / 32];
#pragma unroll
                    for (int i = 0; i < DK / 32; ++i)
                        qf[i] = query_operand(qs, L::kQPitch, 16 * tt, i);
                    const int t = 16 * tt + (lane & 15);
                    const float th = d.hi[t], tl = d.lo[t];
                    float x[8], top = 0.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int st = 2 * j + h;   // tokens 16 st ..; past tile tt all later
                        f32x4 sc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        if (h == 0 || st <= tt) {
#pragma unroll
                            for (int i = 0; i < DK / 32; ++i)
                                sc = mma16<H>(key_row_operand(ks, L::kKPitch, 16 * st, i), qf[i], sc);
                        }
                        const f32x4 sh = *reinterpret_cast<const f32x4 *>(&d.hi[16 * st + 4 * g]);
                        const f32x4 sl = *reinterpret_cast<const f32x4 *>(&d.lo[16 * st + 4 * g]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // a later token: exp2(-inf) = 0 (times a score that is not finite: NaN, see recur)
                            const bool seen = st < tt || (st == tt && 4 * g + r <= (lane & 15));
                            const float e = seen ? (th - sh[r]) + (tl - sl[r]) : -INFINITY;
                            x[4 * h + r] = sc[r] * (__builtin_amdgcn_exp2f(e) * a.scale);
                            if constexpr (H)
                                top = fmaxf(top, fabsf(x[4 * h + r]));
                        }
                    }
                    if constexpr (H) {
                        float mul, back;
                        half_range(column_max(top), kLeastScoreExponent, mul, back);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            x[r] *= mul;
                        if (g == 0)
                            score_back[tt][j][lane] = back;
                    }
                    u32x4 f[kTerms<H>];
                    split8<H>(x, f);
#pragma unroll
                    for (int m = 0; m < kTerms<H>; ++m)
                        scores[(job * kTerms<H> + m) * 64 + lane] = f[m];
                }
                if (more)
                    tq.load(qp + at * a.q_token, left);
                // S^T q of all 64 tokens
                f32x4 acc[4][NV];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                float s_mul[NV], s_back[NV];
                if constexpr (H) {
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        float top = 0.0f;
#pragma unroll
                        for (int i = 0; i < DK / 16; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                top = fmaxf(top, fabsf(S[n][i][r]));
                        half_range(column_max(top), kLeastExponent, s_mul[n], s_back[n]);
                    }
                }
#pragma unroll
                for (int j = 0; j < DK / 32; ++j) {
                    u32x4 qf[4], f[NV][kTerms<H>];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qf[i] = query_operand(qs, L::kQPitch, 16 * i, j);
                    __builtin_amdgcn_sched_barrier(0);      // on their way while the state is split
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        float x[8];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            x[r] = S[n][2 * j][r];
                            x[4 + r] = S[n][2 * j + 1][r];
                        }
                        if constexpr (H) {
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                x[r] *= s_mul[n];
                        }
                        split8<H>(x, f[n]);
                    }
#pragma unroll
                    for (int m = 0; m < kTerms<H>; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int n = 0; n < NV; ++n)
                                acc[i][n] = mma16<H>(f[n][m], qf[i], acc[i][n]);
                }
                if constexpr (H) {
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float b = of_row(s_back[n], r);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[i][n][r] *= b;
                        }
                }
                __syncthreads();
                // + scores V; a token's FP16 scores carry a power of two, into which its sum is brought: exact, and
                // finite for states below 2^58 (see linear_scales.h)
                float back[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    back[i] = 1.0f;
                    float f = d.grown[16 * i + (lane & 15)] * a.scale;
                    if constexpr (H) {
                        back[i] = score_back[i][0][lane & 15];
                        f *= inverse_power(back[i]);
                    }
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][n][r] *= f;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    u32x4 vf[NV];
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        vf[n] = column_operand<NV>(vs + 16 * NV * wave, L::kVPitch, n, j);
#pragma unroll
                    for (int i = 2 * j; i < 4; ++i) {
                        if constexpr (H) {
                            if (j) {
                                const float next = score_back[i][1][lane & 15], f = back[i] * inverse_power(next);
#pragma unroll
                                for (int n = 0; n < NV; ++n)
#pragma unroll
                                    for (int r = 0; r < 4; ++r)
                                        acc[i][n][r] *= f;
                                back[i] = next;
                            }
                        }
#pragma unroll
                        for (int m = 0; m < kTerms<H>; ++m) {
                            const u32x4 pf = scores[(score_slot(i, j) * kTerms<H> + m) * 64 + lane];
#pragma unroll
                            for (int n = 0; n < NV; ++n)
                                acc[i][n] = mma16<H>(vf[n], pf, acc[i][n]);
                        }
                    }
                }
                if (more)
                    tv.load(vp + at * a.v_token, left);
                // a sum is finite only if all of it is
                float sums[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sums[i] = 0.0f;
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        sums[i] += (acc[i][n][0] + acc[i][n][1]) + (acc[i][n][2] + acc[i][n][3]);
                }
                unsigned short *o = op + (long long)c * kChunk * a.out_token;
                if (!slow && wave_any_nan(((sums[0] + sums[1]) + (sums[2] + sums[3])) * 0.0f)) {
                    slow = true;
#pragma unroll
                    for (int i = 0; i < NV * (DK / 16); ++i)
                        T[i] = S[i / (DK / 16)][i % (DK / 16)];
                }
                if (slow) {
                    recur<H, DK, WAVES, NV, OUT>(a, lds, d, rows, T, o, col0);
                } else {
                    const __amdgpu_buffer_rsrc_t dst = make_rsrc(o);
                    unsigned first = out_off;
                    asm volatile("" : "+v"(first));     // kept over the chunks alone, not with every row's
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        unsigned int w[2 * NV];
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            w[2 * n] = pack2<H>(acc[i][n][0] * back[i], acc[i][n][1] * back[i]);
                            w[2 * n + 1] = pack2<H>(acc[i][n][2] * back[i], acc[i][n][3] * back[i]);
                        }
                        // the whole offset per lane, none in a scalar register: the compiler may write the data
                        // registers of a store with a scalar offset in the very next instruction, and this chip was
                        // seen to store what that one wrote (16-byte stores; see the test of the built code)
                        const unsigned to = (lane & 15) < rows - 16 * i ? first + 16 * i * out_step : kSkip;
                        if constexpr (NV == 2)
                            __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, dst, to, 0, 0);
                        else
                            __builtin_amdgcn_raw_buffer_store_b64(u32x2{w[0], w[1]}, dst, to, 0, 0);
                    }
                }
            } else {
                if (more)
                    tv.load(vp + at * a.v_token, left);
                if (attempt)
                    recur<H, DK, WAVES, NV, OUT>(a, lds, d, rows, T, nullptr, col0);
            }
            update_state<H, DK, WAVES, NV, OUT>(lds, d, S);
            __syncthreads();
        }
        if constexpr (OUT)
            break;
        float odd = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * (DK / 16); ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                odd += S[i / (DK / 16)][i % (DK / 16)][r] * 0.0f;
        slow = attempt == 1;
        if (wave == kGateWave && lane == 0 && tile == 0) {
            a.ws_decay[next_at] = sum;
            if (p.part == 0)
                a.ws_serial[start_at] = 0x7FFFFFFF;
        }
        if (slow || !__syncthreads_or(odd != 0.0f))
            break;
    }
    float *to = a.ws_part + next_at * a.dk * a.dv;
    if constexpr (OUT) {
        if (!last || !a.state_out || slot < 0)
            return;
        to = a.state_out + slot * a.so_slot + head * a.so_head;
    }
    if (slow) {
#pragma unroll
        for (int i = 0; i < NV * (DK / 16); ++i)
            S[i / (DK / 16)][i % (DK / 16)] = T[i];
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
        store_state<DK>(a, to, wave_col + value_column<NV>(n, lane & 15), S[n]);
}

// State at the start of every part of the sequences that have several:
// S_0 = the old state, S_{j+1} = exp(G of part j) S_j + what part j adds.
// That is the recurrence only while the factor is finite, and not 0 on a state
// that is not: exp(g) (S + a) is neither inf S + inf a nor, where exp(G) has
// underflowed, 0 * inf.  Such a part takes the rest of its sequence in one go instead (ws_serial).
__global__ __launch_bounds__(kThreads) void linear_join(LArgs a)
{
    const int head = blockIdx.y, seq = blockIdx.z;
    Place p;
    const int start = a.starts[seq];
    place_of(start, a.starts[seq + 1], a.tokens, a.part, first_place(start, a.tokens, a.part, seq), seq, p);
    const int parts = parts_of(p.len, a.part);
    const int at = (blockIdx.x * kThreads + threadIdx.x) * 4, size = a.dk * a.dv;
    if (parts < 2 || at >= size)
        return;
    const int slot = slot_of(a, seq);
    f32x4 S = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (a.state_in && slot >= 0)
        S = *reinterpret_cast<const f32x4 *>(a.state_in + slot * a.in_slot + head * a.in_head + at);
    const long long start_at = (long long)start_state(p.first, a.tokens, a.part, a.sequences, seq) * a.heads + head;
    const long long part_at = (long long)part_state(p.first, a.tokens, a.part, 1) * a.heads + head;
    *reinterpret_cast<f32x4 *>(a.ws_start + start_at * size + at) = S;
    float *w = a.ws_part + part_at * size + at;
    const double *decay = a.ws_decay + part_at;
    const long long step = (long long)a.heads * size;
    constexpr int kAhead = 8;                   // parts whose loads are under way at once
    for (int j0 = 0; j0 + 1 < parts; j0 += kAhead) {
        f32x4 add[kAhead];
        double log2[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = min(j0 + u, parts - 2);
            add[u] = *reinterpret_cast<const f32x4 *>(w + j * step);
            log2[u] = decay[(long long)j * a.heads];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = j0 + u;
            if (j + 1 < parts) {
                const float f = __builtin_amdgcn_exp2f((float)log2[u]);
                const float odd = ((S[0] + S[1]) + (S[2] + S[3])) * 0.0f;
                if (!(f < INFINITY) || (f == 0.0f && odd != 0.0f))
                    atomicMin(&a.ws_serial[start_at], j);
                S = S * f + add[u];
                *reinterpret_cast<f32x4 *>(w + j * step) = S;
            }
        }
    }
}

// One new token of each sequence.  A workgroup takes 32 value columns of one
// (sequence, head): 8 threads of four columns by 32 rows of the state, so that
// every load of the state is under way at once and a single sequence still
// gives several workgroups a head.  Bound by the state's bytes, 8 dk dv a head.  64
// sequences of 12 heads of 128: 20.6 us, 4.9 TB/s of a copy's 4.8; one: 3.8 us.
template <bool H>
__global__ __launch_bounds__(kThreads, 4) void linear_step(LArgs a)
{
    __shared__ f32x4 part[4][8];
    const int head = blockIdx.y, seq = blockIdx.z;
    const int cq = threadIdx.x & 7, row0 = threadIdx.x >> 3, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned col = blockIdx.x * 32 + 4 * cq, dv = (unsigned)a.dv;
    const int khead = head / a.share, slot = slot_of(a, seq);
    const bool live = col < dv;
    const unsigned short *q = static_cast<const unsigned short *>(a.q) + seq * a.q_token + khead * a.q_head;
    const unsigned short *k = static_cast<const unsigned short *>(a.k) + seq * a.k_token + khead * a.k_head;
    const unsigned short *v = static_cast<const unsigned short *>(a.v) + seq * a.v_token + head * a.v_head;
    const float *in = slot >= 0 && a.state_in ? a.state_in + slot * a.in_slot + head * a.in_head : nullptr;
    float *so = slot >= 0 && a.state_out ? a.state_out + slot * a.so_slot + head * a.so_head : nullptr;
    constexpr int kRows = 8;                    // dk <= 256: at most 8 rows a thread
    f32x4 S[kRows];
    float kk[kRows], qq[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const unsigned row = row0 + 32 * i;
        S[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        kk[i] = qq[i] = 0.0f;
        if (row < (unsigned)a.dk && live) {
            if (in)
                S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(in + (row * dv + col)));
            kk[i] = to_float<H>(k[row]);
            qq[i] = to_float<H>(q[row]);
        }
    }
    const float e = expf(a.g[seq * a.g_token + head * a.g_head]);
    f32x4 vv = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, o = vv;
    if (live) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(v + col);
        const unsigned int w0 = w.x, w1 = w.y;
        float x0, x1, x2, x3;
        unpack2<H>(w0, x0, x1);
        unpack2<H>(w1, x2, x3);
        vv = f32x4{x0, x1, x2, x3};
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const unsigned row = row0 + 32 * i;
        if (row < (unsigned)a.dk && live) {
            S[i] = S[i] * e + kk[i] * vv;
            o += qq[i] * S[i];
            if (so)
                __builtin_nontemporal_store(S[i], reinterpret_cast<f32x4 *>(so + (row * dv + col)));
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float x = o[r];
        x += __shfl_xor(x, 8, 64);
        x += __shfl_xor(x, 16, 64);
        x += __shfl_xor(x, 32, 64);
        o[r] = x;
    }
    if (lane < 8)
        part[wave][lane] = o;
    __syncthreads();
    if (threadIdx.x < 8 && live) {
        const f32x4 s = ((part[0][cq] + part[1][cq]) + (part[2][cq] + part[3][cq])) * a.scale;
        u32x2 w;
        w.x = to_bits<H>(s[0]) | (unsigned)to_bits<H>(s[1]) << 16;
        w.y = to_bits<H>(s[2]) | (unsigned)to_bits<H>(s[3]) << 16;
        *reinterpret_cast<u32x2 *>(static_cast<unsigned short *>(a.out) + seq * a.out_token + head * a.out_head +
                                   col) = w;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// The workspace: states of parts and of starts, decays, the parts that go on.
struct Workspace {
    size_t parts, starts;       // states
    size_t state;               // bytes of one

    size_t bytes(int heads) const
    {
        return (parts + starts) * state + parts * heads * sizeof(double) + starts * heads * sizeof(int);
    }
};

Workspace workspace_of(int tokens, int sequences, int heads, int dk, int dv)
{
    const size_t parts = tokens > kOnePass ? (size_t)most_extra_parts(tokens, sequences, heads, dv) : 0;
    const size_t starts = parts < (size_t)sequences ? parts : (size_t)sequences;
    return Workspace{parts, starts, (size_t)heads * dk * dv * sizeof(float)};
}

hipError_t launch_one(void (*fn)(LArgs), dim3 grid, int threads, size_t lds, const LArgs &a, hipStream_t stream)
{
    LArgs copy = a;
    void *params[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void *>(fn), grid, dim3(threads), params, lds, stream);
}

// Dynamic LDS past 64 KiB has to be asked for, once on every device: `done` has a bit for each.
void raise_limit(void (*fn)(LArgs), int bytes, std::atomic<unsigned long long> &done)
{
    int device = 0;
    (void)hipGetDevice(&device);
    const unsigned long long bit = 1ull << (device & 63);
    if (done.load(std::memory_order_relaxed) & bit)
        return;
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    done.fetch_or(bit, std::memory_order_relaxed);
}

template <bool H, int DK, int WAVES, int NV>
hipError_t launch_prompt(const LArgs &a, hipStream_t stream)
{
    static std::atomic<unsigned long long> raised{0};
    raise_limit(linear_chunks<H, DK, WAVES, NV, true>, Layout<DK, WAVES, NV, true>::kBytes, raised);
    const dim3 grid((unsigned)(((long long)a.groups + 7) / 8 * 8 * a.share * a.col_tiles));
    hipError_t e = hipSuccess;
    if (a.multi) {
        e = launch_one(linear_chunks<H, DK, WAVES, NV, false>, grid, 64 * WAVES, Layout<DK, WAVES, NV, false>::kBytes, a,
                       stream);
        const dim3 jg((unsigned)((a.dk * a.dv / 4 + kThreads - 1) / kThreads), (unsigned)a.heads,
                      (unsigned)a.sequences);
        if (e == hipSuccess)
            e = launch_one(linear_join, jg, kThreads, 0, a, stream);
    }
    if (e == hipSuccess)
        e = launch_one(linear_chunks<H, DK, WAVES, NV, true>, grid, 64 * WAVES, Layout<DK, WAVES, NV, true>::kBytes, a, stream);
    return e;
}

template <bool H>
hipError_t launch_prompt_type(const LArgs &a, const Shape &s, hipStream_t stream)
{
    const bool wide = s.cols == 128;
    if (a.dk > 128)
        return wide ? launch_prompt<H, 256, 8, 1>(a, stream) : launch_prompt<H, 256, 4, 1>(a, stream);
    if (a.dk > 64)
        return s.eight ? launch_prompt<H, 128, 8, 1>(a, stream)
               : wide  ? launch_prompt<H, 128, 4, 2>(a, stream) : launch_prompt<H, 128, 4, 1>(a, stream);
    if (a.dk > 32)
        return wide ? launch_prompt<H, 64, 8, 1>(a, stream) : launch_prompt<H, 64, 4, 1>(a, stream);
    return wide ? launch_prompt<H, 32, 8, 1>(a, stream) : launch_prompt<H, 32, 4, 1>(a, stream);
}

// Threads of a workgroup of the form that launch_prompt_type takes.
int threads_of(const Shape &s, int dk)
{
    const bool wide_waves = dk > 64 && dk <= 128 && !s.eight;
    return s.cols == 128 && !wide_waves ? 512 : 256;
}

constexpr long long kMaxTokenStride = 1 << 24;

skinny_status bad(skinny_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
skinny_status bad(skinny_status s, const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error("%s", buf);
    return s;
}

skinny_status check_linear(const skinny_linear_args *p, bool prompt)
{
    if (!p)
        return bad(SKINNY_ERR_INVALID_ARG, "args is NULL");
    if (p->type != SKINNY_IN_BF16 && p->type != SKINNY_IN_F16)
        return bad(SKINNY_ERR_INVALID_ARG, "type %d is neither BF16 nor FP16", p->type);
    if (p->tokens < 0 || p->sequences < 0 || p->pool < 0)
        return bad(SKINNY_ERR_INVALID_ARG, "tokens=%d, sequences=%d and pool=%d must not be negative", p->tokens,
                   p->sequences, p->pool);
    if (p->heads < 1 || p->heads > 65535 || p->key_heads < 1 || p->heads % p->key_heads)
        return bad(SKINNY_ERR_SHAPE, "heads=%d must be 1..65535 and a multiple of key_heads=%d", p->heads,
                   p->key_heads);
    if (p->tokens > 0x7FFFF000)
        return bad(SKINNY_ERR_SHAPE, "tokens=%d: at most %d", p->tokens, 0x7FFFF000);
    if (p->sequences > 65535)
        return bad(SKINNY_ERR_SHAPE, "sequences=%d: at most 65535", p->sequences);
    if (p->dk < 8 || p->dk > 256 || p->dk % 8 || p->dv < 8 || p->dv > 1024 || p->dv % 8)
        return bad(SKINNY_ERR_SHAPE, "dk=%d and dv=%d must be multiples of 8, dk <= 256, dv <= 1024", p->dk, p->dv);
    if (!prompt && p->tokens != p->sequences)
        return bad(SKINNY_ERR_SHAPE, "a step has one token a sequence: tokens=%d, sequences=%d", p->tokens,
                   p->sequences);
    if (p->tokens > 0 && (!p->q || !p->k || !p->v || !p->log_decay || !p->out))
        return bad(SKINNY_ERR_INVALID_ARG, "q, k, v, log_decay or out is NULL");
    if (prompt && p->sequences > 0 && !p->starts)
        return bad(SKINNY_ERR_INVALID_ARG, "starts is NULL");
    if (prompt && p->sequences == 0 && p->tokens > 0)
        return bad(SKINNY_ERR_SHAPE, "%d tokens but no sequence", p->tokens);
    if (!p->slots && (p->state_in || p->state_out) && p->pool < p->sequences)
        return bad(SKINNY_ERR_SHAPE, "pool=%d holds fewer states than sequences=%d", p->pool, p->sequences);
    const long long token[] = {p->q_token, p->k_token, p->v_token, p->out_token};
    const long long per_head[] = {p->q_head, p->k_head, p->v_head, p->out_head};
    static const char *const names[] = {"q", "k", "v", "out"};
    const void *const ptr[] = {p->q, p->k, p->v, p->out};
    for (int i = 0; i < 4; ++i) {
        if (token[i] % 8 || per_head[i] % 8 || token[i] < 0 || per_head[i] < 0 || token[i] >= kMaxTokenStride)
            return bad(SKINNY_ERR_SHAPE, "%s strides (%lld, %lld) must be multiples of 8 in [0, 2^24)", names[i],
                       token[i], per_head[i]);
        if ((uintptr_t)ptr[i] & 15)
            return bad(SKINNY_ERR_ALIGN, "%s must be 16-byte aligned", names[i]);
    }
    if (p->decay_token < 0 || p->decay_head < 0)
        return bad(SKINNY_ERR_SHAPE, "log_decay strides must not be negative");
    if (((uintptr_t)p->log_decay & 3) || ((uintptr_t)p->starts & 3) || ((uintptr_t)p->slots & 3))
        return bad(SKINNY_ERR_ALIGN, "log_decay, starts and slots must be 4-byte aligned");
    if (((uintptr_t)p->state_in & 15) || ((uintptr_t)p->state_out & 15))
        return bad(SKINNY_ERR_ALIGN, "state_in and state_out must be 16-byte aligned");
    if (p->in_state_slot % 4 || p->in_state_head % 4 || p->out_state_slot % 4 || p->out_state_head % 4 || p->in_state_slot < 0 ||
        p->in_state_head < 0 || p->out_state_slot < 0 || p->out_state_head < 0)
        return bad(SKINNY_ERR_SHAPE, "state strides must be multiples of 4 and not negative");
    return SKINNY_OK;
}

LArgs kernel_args(const skinny_linear_args *p)
{
    LArgs a{};
    a.q = p->q;
    a.k = p->k;
    a.v = p->v;
    a.out = p->out;
    a.g = p->log_decay;
    a.state_in = p->state_in;
    a.state_out = p->state_out;
    a.starts = p->starts;
    a.slots = p->slots;
    a.q_token = p->q_token;
    a.q_head = p->q_head;
    a.k_token = p->k_token;
    a.k_head = p->k_head;
    a.v_token = p->v_token;
    a.v_head = p->v_head;
    a.out_token = p->out_token;
    a.out_head = p->out_head;
    a.g_token = p->decay_token;
    a.g_head = p->decay_head;
    a.in_slot = p->in_state_slot;
    a.in_head = p->in_state_head;
    a.so_slot = p->out_state_slot;
    a.so_head = p->out_state_head;
    a.tokens = p->tokens;
    a.sequences = p->sequences;
    a.heads = p->heads;
    a.share = p->heads / p->key_heads;
    a.dk = p->dk;
    a.dv = p->dv;
    a.pool = p->pool;
    a.scale = p->scale;
    return a;
}

skinny_status launched(hipError_t e)
{
    return e == hipSuccess ? SKINNY_OK : bad(SKINNY_ERR_HIP, "linear attention launch: %s", hipGetErrorString(e));
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

size_t skinny_linear_workspace(int tokens, int sequences, int heads, int dk, int dv)
{
    if (tokens < 0 || tokens > 0x7FFFF000 || sequences < 0 || heads < 1 || dk < 8 || dk > 256 || dv < 8 || dv > 1024)
        return 0;
    return workspace_of(tokens, sequences, heads, dk, dv).bytes(heads);
}

skinny_status skinny_linear_prompt(const skinny_linear_args *p, void *stream)
{
    skinny_status st = check_linear(p, true);
    if (st != SKINNY_OK)
        return st;
    if (p->sequences == 0)
        return SKINNY_OK;
    const Shape s = shape_of(p->tokens, p->sequences, p->heads, p->dk, p->dv);
    // a launch of 2^32 threads or more runs a part of them and reports nothing; 8 more key heads' fill the last XCDs
    const long long most = 0xFFFFFFFFLL / threads_of(s, p->dk);
    if (((long long)s.places * p->key_heads + 8) * (p->heads / p->key_heads) * s.col_tiles > most)
        return bad(SKINNY_ERR_SHAPE, "tokens=%d, sequences=%d and heads=%d are too many for one call", p->tokens,
                   p->sequences, p->heads);
    const Workspace w = workspace_of(p->tokens, p->sequences, p->heads, p->dk, p->dv);
    const size_t need = s.multi ? w.bytes(p->heads) : 0;
    if (need && (!p->workspace || p->workspace_bytes < need))
        return bad(SKINNY_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu are needed",
                   p->workspace ? p->workspace_bytes : (size_t)0, need);
    if (need && ((uintptr_t)p->workspace & 15))
        return bad(SKINNY_ERR_ALIGN, "workspace must be 16-byte aligned");
    LArgs a = kernel_args(p);
    a.part = s.part;
    a.places = s.places;
    a.col_tiles = s.col_tiles;
    a.groups = s.places * p->key_heads;
    // a sequence leaves one place empty at most; an XCD whose parts lie together in memory is faster on them (one
    // prompt of 32768 tokens: 194 against 201 us), one that has an empty run is not (7 of 18686 tokens: 178 against
    // 170 us)
    a.runs = s.places >= 16 * (long long)p->sequences;
    a.multi = s.multi;
    if (s.multi) {
        char *ws = static_cast<char *>(p->workspace);
        a.ws_part = reinterpret_cast<float *>(ws);
        a.ws_start = reinterpret_cast<float *>(ws += w.parts * w.state);
        a.ws_decay = reinterpret_cast<double *>(ws += w.starts * w.state);
        a.ws_serial = reinterpret_cast<int *>(ws + w.parts * p->heads * sizeof(double));
    }
    return launched(p->type == SKINNY_IN_F16 ? launch_prompt_type<true>(a, s, (hipStream_t)stream)
                                             : launch_prompt_type<false>(a, s, (hipStream_t)stream));
}

skinny_status skinny_linear_step(const skinny_linear_args *p, void *stream)
{
    skinny_status st = check_linear(p, false);
    if (st != SKINNY_OK)
        return st;
    if (p->sequences == 0)
        return SKINNY_OK;
    const LArgs a = kernel_args(p);
    const dim3 grid((unsigned)((a.dv + 31) / 32), (unsigned)a.heads, (unsigned)a.sequences);
    return launched(launch_one(p->type == SKINNY_IN_F16 ? linear_step<true> : linear_step<false>, grid, kThreads, 0, a,
                               (hipStream_t)stream));
}

}  // extern "C"
