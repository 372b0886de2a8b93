// HIP kernels and entry points of blocks of 32 values with a power of two
// (microscaled floating point), and of products with weights in them, for
// gfx950 (CDNA4):
//
//   byte = power + 127, power = floor(log2 max |v|) - top,  q = nearest(v 2^-power)
//   out[m][n] = sum over blocks b of 2^(xs[m][b] + ws[n][b] - 254) sum_{k in b} x[m][k] W[n][k]  (+ residual[m][n])
//
// W in 4 bits (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), x in 4 or
// 8 (e4m3).  The matrix units take codes and powers as they are
// (v_mfma_scale_f32_16x16x128_f8f6f4) and sum in fp32.
#include <hip/hip_runtime.h>

#include <new>

#include "mxfp4_tiles.h"
#include "operators.h"
#include "rows.h"
#include "skinny_internal.h"

// A prepared 4-bit weight.
struct skinny_mxfp4_plan {
    int N, K;
    int units;                  // of 256 k, in w: the last one filled with zeros
    skinny_type out;
    int device;
    void *w;                    // [N / 16][units][2 steps][64 lanes][16 bytes], zero past N and K
    unsigned *w_scale;          // [N / 32][units][64 lanes]: bytes of two row tiles at two steps
};

namespace skinny {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

constexpr long long kMostThreads = 0xFFFFFFFFLL;    // a launch may have

// ---------------------------------------------------------------------------
// Rows to blocks, and back
// ---------------------------------------------------------------------------

struct BArgs {
    const void *x, *gate;       // gate: or NULL
    unsigned char *q, *scale;
    long long ldx, ldg, ldq, lds;
    unsigned octets;            // in all rows of the launch
    unsigned per_row;
    FastDiv by_row;
};

__device__ __forceinline__ unsigned quotient(unsigned x, const FastDiv &f)
{
    const unsigned t = __umulhi(x, f.mul);
    return (t + ((x - t) >> f.s1)) >> f.s2;
}

// Eight values a thread, four threads a block, U times 256 threads a workgroup; no
// barrier and no LDS: the largest of a block goes around its four lanes.  Rows one
// after the other are taken as one.  Bound by bytes: 6001 x 7168 in BF16 to 4
// bits 23.3 us, 4.7 TB/s, to 8 bits 26.6; 1000 x 18432 gated, in FP16 to 8 bits,
// 18.6 us, 5.0 TB/s; 4 rows 1.9 us.
template <int TYPE, int BITS, bool GATE, bool VEC, int U>
__global__ __launch_bounds__(256) void quantize_octets(BArgs a)
{
    constexpr int kBytes = sizeof(typename Elem<TYPE>::raw);
    const unsigned first = blockIdx.x * (256u * U) + threadIdx.x;
    Octet x[U], g[U];
    long long row[U];
    unsigned o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned i = first + 256u * u;
        const unsigned r = quotient(i, a.by_row);
        row[u] = r;
        o[u] = i - r * a.per_row;
        if (i < a.octets) {
            const long long K = 8LL * a.per_row;
            x[u] = load_octet<VEC>(static_cast<const char *>(a.x) + row[u] * a.ldx * kBytes, TYPE, (int)o[u], K);
            if (GATE)
                g[u] = load_octet<VEC>(static_cast<const char *>(a.gate) + row[u] * a.ldg * kBytes, TYPE, (int)o[u], K);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (first + 256u * u >= a.octets)
            continue;                           // whole blocks: all four lanes of a quad or none
        float f[8];
        unpack_octet(x[u], TYPE, f);
        if (GATE) {
            float h[8];
            float gate[8];
            unpack_octet(g[u], TYPE, gate);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = gate[e];
            sigmoid(h);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] *= gate[e] * h[e];
        }
        unsigned byte;
        const u32x2 codes = block_codes<BITS>(f, byte);
        store_codes<VEC, BITS>(a.q + row[u] * a.ldq, (int)o[u], codes);
        if ((o[u] & 3) == 0)
            a.scale[row[u] * a.lds + (o[u] >> 2)] = (unsigned char)byte;
    }
}

struct XArgs {
    const unsigned char *q, *scale;
    void *out;
    long long ldq, lds, ldo;
    int type;
    unsigned octets, per_row;
    FastDiv by_row;
};

// Eight values a thread.  Bound by bytes: 6001 x 7168 from 4 bits to BF16 26 us alone
// (4.2 TB/s), 17.8 where the codes were just written and lie in the caches.
template <int BITS, bool VEC>
__global__ __launch_bounds__(256) void expand_octets(XArgs a)
{
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    if (i >= a.octets)
        return;
    const unsigned r = quotient(i, a.by_row), o = i - r * a.per_row;
    const unsigned char *p = a.q + r * a.ldq + (long long)o * BITS;
    const float scale = power_of(a.scale[r * a.lds + (o >> 2)]);
    unsigned w[BITS / 4];
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < BITS / 4; ++j)
            w[j] = reinterpret_cast<const unsigned *>(p)[j];
    } else {
#pragma unroll
        for (int j = 0; j < BITS / 4; ++j)
            w[j] = p[4 * j] | (unsigned)p[4 * j + 1] << 8 | (unsigned)p[4 * j + 2] << 16 | (unsigned)p[4 * j + 3] << 24;
    }
    float f[8];
    if constexpr (BITS == 8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
            f[4 * j] = lo[0] * scale;
            f[4 * j + 1] = lo[1] * scale;
            f[4 * j + 2] = hi[0] * scale;
            f[4 * j + 3] = hi[1] * scale;
        }
    } else {
        const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 0),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 2),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 3)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = v[j][0] * scale;
            f[2 * j + 1] = v[j][1] * scale;
        }
    }
    const Octet y = pack_octet(a.type, f);
    store_octet<VEC>(static_cast<char *>(a.out) + r * a.ldo * (a.type == SKINNY_TYPE_F32 ? 4 : 2), a.type, (int)o,
                     8LL * a.per_row, y);
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

constexpr int kUnitBlocks = 8;  // blocks of a unit: 256 k, two MFMAs of 128

struct PArgs {
    const u32x4 *w;             // laid out by lay_out
    const unsigned *w_scale;    // by lay_out_scales
    const unsigned char *x, *x_scale;
    const void *res;
    void *out;
    long long ldx, ldxs, ldr, ldo;      // in bytes, bytes, elements, elements
    int M, N;
    int x_bytes;                // of a row of x
    int blocks;                 // K / 32
    int units;                  // of 256 k
    int type;                   // skinny_type of out and res
    int vec;                    // out and res take four columns at once
    int words;                  // rows of x's powers are whole aligned dwords
    int m_tiles;                // token tiles of the launch
    int n_tiles;                // tiles of weight rows
};

// Weight rows into MFMA operands: at step s of unit u, lane l of row tile t
// takes block 8 u + 4 s + l / 16 of row 16 t + l % 16, so that a wave's load of
// an operand is 1 KiB in a row.  16-byte vectors `first` .. count - 1.
__global__ __launch_bounds__(256) void lay_out(const unsigned char *w, long long ldw, int N, int blocks, int units,
                                               u32x4 *out, long long first, long long count)
{
    const long long i = first + (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    const int lane = (int)(i & 63), s = (int)(i >> 6) & 1;
    const long long tu = i >> 7;
    const long long n = tu / units * 16 + (lane & 15);
    const int b = (int)(tu % units) * kUnitBlocks + 4 * s + (lane >> 4);
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (n < N && b < blocks) {
        const unsigned char *p = w + n * ldw + 16LL * b;
        if (((uintptr_t)p & 15) == 0) {
            v = *reinterpret_cast<const u32x4 *>(p);
        } else {
            for (int j = 0; j < 16; ++j)
                v[j / 4] |= (unsigned)p[j] << (8 * (j % 4));
        }
    }
    out[i] = v;
}

// Their powers: lane l of unit u of row tiles 2 p and 2 p + 1 has one dword,
// the bytes of (2 p, step 0), (2 p, step 1), (2 p + 1, step 0), (2 p + 1, step 1).
__global__ __launch_bounds__(256) void lay_out_scales(const unsigned char *s, long long lds, int N, int blocks,
                                                      int units, unsigned *out, long long first, long long count)
{
    const long long i = first + (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    const int lane = (int)(i & 63);
    const long long pu = i >> 6;
    unsigned v = 0;
    for (int j = 0; j < 4; ++j) {
        const long long n = pu / units * 32 + 16 * (j >> 1) + (lane & 15);
        const int b = (int)(pu % units) * kUnitBlocks + 4 * (j & 1) + (lane >> 4);
        if (n < N && b < blocks)
            v |= (unsigned)s[n * lds + b] << (8 * j);
    }
    out[i] = v;
}

// Four outputs of one token, columns n .. n + 3.
template <int OUT>
__device__ __forceinline__ void store4_as(const PArgs &a, int m, int n, f32x4 v)
{
    using E = Elem<OUT>;
    typedef __attribute__((ext_vector_type(4))) typename E::raw raw4;
    typename E::raw *o = static_cast<typename E::raw *>(a.out) + m * a.ldo + n;
    const typename E::raw *res = a.res ? static_cast<const typename E::raw *>(a.res) + m * a.ldr + n : nullptr;
    if (a.vec && n + 4 <= a.N) {
        if (res) {
            const raw4 x = *reinterpret_cast<const raw4 *>(res);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] += E::get(x[r]);
        }
        raw4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            y[r] = E::put(v[r]);
        *reinterpret_cast<raw4 *>(o) = y;
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (n + r < a.N)
            o[r] = E::put(res ? v[r] + E::get(res[r]) : v[r]);
}

__device__ __forceinline__ void store4(const PArgs &a, int m, int n, f32x4 v)
{
    if (a.type == SKINNY_TYPE_BF16)
        store4_as<SKINNY_TYPE_BF16>(a, m, n, v);
    else if (a.type == SKINNY_TYPE_F32)
        store4_as<SKINNY_TYPE_F32>(a, m, n, v);
    else
        store4_as<SKINNY_TYPE_F16>(a, m, n, v);
}

// An operand of x: one vector of 32 4-bit values, or two of 16 8-bit ones.
template <int BITS>
struct XOp {
    u32x4 v[BITS / 4];
};

__device__ __forceinline__ i32x8 widened(u32x4 v)
{
    const i32x4 w = __builtin_bit_cast(i32x4, v);
    return __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
}

template <int V>
struct Const {
    static constexpr int value = V;
};

// 16 rows of w by 16 tokens over 128 k, both in 4 bits; byte WB of ws and the
// lowest of xs are the lanes' powers.
template <int WB>
__device__ __forceinline__ f32x4 mma128(u32x4 w, u32x4 x, f32x4 c, unsigned ws, unsigned xs)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widened(w), widened(x), c, 4, 4, WB, (int)ws, 0, (int)xs);
}

// Eight values times their power in BF16, whose subnormals reach down to 2^-133 and are
// kept: exact for codes of 4 bits with powers of 2^-127 to 2^125 and of 8 with 2^-124
// to 2^119.  Blocks of finite fp32 values get no larger ones; 8-bit blocks with nothing above
// 2^-116 may get smaller ones, and their values are rounded to multiples of 2^-133.
__device__ __forceinline__ bf16x8 bf16_of_4(unsigned w, float power)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 3);
    return __builtin_shufflevector(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3),
                                   0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ bf16x8 bf16_of_8(unsigned lo, unsigned hi, float power)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, power, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, power, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, power, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, power, true);
    return __builtin_shufflevector(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3),
                                   0, 1, 2, 3, 4, 5, 6, 7);
}

// Where a row's 16-byte chunks lie in LDS, before the row's own order (^ row % 8):
// part `part` of lane group g's operand at step s, block 4 s + g, at 4 s + g in 4
// bits and at 8 s + 4 part + g in 8, so that the four lane groups read side by
// side (memory's order has bank conflicts in a thirteenth of the cycles).
template <int BITS>
__device__ __forceinline__ int place_in_row(int g, int s, int part)
{
    return BITS == 4 ? 4 * s + g : 8 * s + 4 * part + g;
}

// The same of chunk c in memory.
template <int BITS>
__device__ __forceinline__ int place_of_chunk(int c)
{
    return BITS == 4 ? c : (c & 8) + 4 * (c & 1) + (c >> 1 & 3);
}

// A buffer load whose offset is past its resource reads zero and touches no
// memory; loads to be skipped take this one (resources are smaller: 256 rows of
// x at pitches below 2^22).  Offsets are all in the per-lane part, the one that
// is checked whatever its value.
constexpr unsigned kSkip = 0x7FF00000u;
constexpr long long kMaxPitch = 1 << 22;
constexpr int kMaxRows = 0x7FFFF000;     // of x and w: tiles are counted in 32 bits

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, unsigned bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

// Consecutive logical ids on one XCD (the dispatcher deals workgroups over 8).
__device__ __forceinline__ unsigned logical_id()
{
    const unsigned xcd = blockIdx.x & 7u, turn = blockIdx.x >> 3, q = gridDim.x >> 3, r = gridDim.x & 7u;
    return xcd * q + (xcd < r ? xcd : r) + turn;
}

// The products of a unit: RT row tiles by MT token tiles, 256 k.  4-bit tokens
// go into the scaled MFMA as they are.  8-bit ones could, but that one adds
// neighbouring products of 8-bit codes in a fixed window: what is below 2^-13 of
// the largest of them is lost (K = 7168, channels that differ as exp(n / 2): 0.73 % of
// BF16 outputs are another value, and 0.01 % by the way taken).  They go in BF16, as
// does w then, at two values an instruction and four cycles, and every product is added in fp32.
template <int RT, int MT, int BITS>
__device__ __forceinline__ void multiply(f32x4 (&acc)[RT][MT], const u32x4 (&w)[2][RT], const XOp<BITS> (&x)[2][MT],
                                         const unsigned *ws, const unsigned (&xs)[2][MT])
{
    if constexpr (BITS == 4) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (r % 2 == 0) {
                    acc[r][t] = mma128<0>(w[0][r], x[0][t].v[0], acc[r][t], ws[r / 2], xs[0][t]);
                    acc[r][t] = mma128<1>(w[1][r], x[1][t].v[0], acc[r][t], ws[r / 2], xs[1][t]);
                } else {
                    acc[r][t] = mma128<2>(w[0][r], x[0][t].v[0], acc[r][t], ws[r / 2], xs[0][t]);
                    acc[r][t] = mma128<3>(w[1][r], x[1][t].v[0], acc[r][t], ws[r / 2], xs[1][t]);
                }
            }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float wp[RT], xp[MT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wp[r] = power_of(ws[r / 2] >> (16 * (r % 2) + 8 * k) & 0xFFu);
#pragma unroll
            for (int t = 0; t < MT; ++t)
                xp[t] = power_of(xs[k][t] & 0xFFu);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bf16x8 wv[RT], xv[MT];
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    wv[r] = bf16_of_4(w[k][r][j], wp[r]);
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    xv[t] = bf16_of_8(x[k][t].v[j / 2][2 * j % 4], x[k][t].v[j / 2][2 * j % 4 + 1], xp[t]);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[r], xv[t], acc[r][t], 0, 0, 0);
            }
        }
    }
}

// 16 RT weight rows by 16 MT tokens a workgroup, its eight waves taking every
// eighth unit of 256 k: each holds all sums of the tile, which are added at the
// end through LDS in a fixed order.  Loads go into registers, D units ahead.  x
// is read in whole lines, XR rows of a tile (the tokens that there are), and passes
// through the wave's own LDS on its way into operands, a token tile at a time.
// Bound by the loads' way from memory: with none of x 6288 x 7168 takes one token
// 6.0 us of 6.3, 7168 x 18432 64 tokens 14.3 of 17.1.  One token of 6288 x 7168 takes
// 6.2 us in 4 bits and 6.5 in 8 (24 MB at 3.8 TB/s, with a launch's 2 us), of 7168 x
// 18432 12.5 us (5.6 TB/s).  Units past the last are not loaded, which made 8.5 us
// of 6.9; four units ahead cost as much again, two with more tokens up to a quarter
// (64 x 6288 x 7168 in 8 bits 12.2 against 13.1 us, at 64 rows by 16 tokens 13.8 against
// 16.8), and so does x asked for before the products and w after them.  NT: the weight passes by once (a
// single token tile) and need not stay in the caches: with more weights than these
// hold 6.2 against 6.6 us for one token, 8.4 against 8.9 for 16; where a few weights
// are read again and again it is up to 1.3 us slower (2048 x 7168).
template <int RT, int MT, int BITS, int D, int XR, bool NT>
__global__ __launch_bounds__(512) void product_rows(PArgs a)
{
    constexpr int kWaves = 8, kV = RT * MT;
    constexpr int kLine = 32 * BITS;                    // bytes of a row's unit
    constexpr int kPerRow = kLine / 16, kRows = 64 / kPerRow;   // vectors of a row's unit, rows of a load
    constexpr int kLoads = (XR + kRows - 1) / kRows;    // loads of a token tile's unit
    constexpr int kTile = 16 * kPerRow;                 // vectors of a token tile's unit
    constexpr int kS = (RT + 1) / 2;
    __shared__ u32x4 shared[kWaves * kTile > 256 * kV ? kWaves * kTile : 256 * kV];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const unsigned id = logical_id();
    const int mt = (int)(id % (unsigned)a.m_tiles), block = (int)(id / (unsigned)a.m_tiles);
    const int n0 = block * 16 * RT, m0 = mt * 16 * MT;
    const int row_tiles = min(RT, (a.N - n0 + 15) / 16), rows = min(16 * MT, a.M - m0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (long long)block * RT * a.units * 128,
                                                (unsigned)(row_tiles * a.units) * 2048u);
    const int pair = block * RT / 2;
    const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.w_scale + (long long)pair * a.units * 64,
                                                 (unsigned)((row_tiles + 1) / 2 * a.units) * 256u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + m0 * a.ldx, (unsigned)((rows - 1) * a.ldx) + (unsigned)a.x_bytes);
    const __amdgpu_buffer_rsrc_t xsr = make_rsrc(a.x_scale + m0 * a.ldxs,
                                                 (unsigned)((rows - 1) * a.ldxs) + (unsigned)a.blocks);
    unsigned w_off[RT], x_off[MT * kLoads], xs_off[MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        w_off[r] = (unsigned)(r * a.units) * 2048u + 16u * lane;
    const int sub = lane / kPerRow, slot = lane % kPerRow;      // a load's row and 16-byte chunk of this lane
#pragma unroll
    for (int t = 0; t < MT * kLoads; ++t) {
        const int row = kRows * t + sub;
        x_off[t] = row < rows ? (unsigned)(row * a.ldx) + 16u * slot : kSkip;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + (lane & 15);
        xs_off[t] = row < rows ? (unsigned)(row * a.ldxs) + (a.words ? 0u : (unsigned)g) : kSkip;
    }
    f32x4 acc[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 wf[D][2][RT], xf[D][MT * kLoads];
    unsigned ws[D][kS], xs[D][2][MT];
    // Past K neither codes nor powers of x may be read, which are other rows' and
    // may stand for NaN.  Units past the last are not loaded, which a load of
    // nothing would pay for like any other.
    const auto load = [&](int d, int u) {
        if (u >= a.units)
            return;
        const unsigned wo = (unsigned)u * 2048u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wf[d][k][r] = __builtin_amdgcn_raw_buffer_load_b128(wr, w_off[r] + wo + 1024u * k, 0, NT ? 2 : 0);
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            const unsigned at = (unsigned)(r * a.units) * 256u + 4u * lane + (unsigned)u * 256u;
            if constexpr (RT == 1)
                ws[d][r] = __builtin_amdgcn_raw_buffer_load_b16(wsr, at + 2u * (block & 1), 0, NT ? 2 : 0);
            else
                ws[d][r] = __builtin_amdgcn_raw_buffer_load_b32(wsr, at, 0, NT ? 2 : 0);
        }
        const unsigned xo = u * kLine + 16 * slot < a.x_bytes ? (unsigned)u * kLine : kSkip;
#pragma unroll
        for (int t = 0; t < MT * kLoads; ++t)
            xf[d][t] = __builtin_amdgcn_raw_buffer_load_b128(xr, x_off[t] + xo, 0, 0);
        const unsigned so = (unsigned)(kUnitBlocks * u);
        if (a.words) {
            if (kUnitBlocks * u + 4 < a.blocks) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(xsr, xs_off[t] + so, 0, 0);
                    xs[d][0][t] = v[0];
                    xs[d][1][t] = v[1];
                }
            } else {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    xs[d][0][t] = __builtin_amdgcn_raw_buffer_load_b32(xsr, xs_off[t] + so, 0, 0);
                    xs[d][1][t] = 0u;
                }
            }
        } else {
            const int b = kUnitBlocks * u + g;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    xs[d][k][t] = __builtin_amdgcn_raw_buffer_load_b8(
                        xsr, xs_off[t] + (b + 4 * k < a.blocks ? so + 4u * k : kSkip), 0, 0);
        }
    };
    // written a row at a time and read a column at a time without bank conflicts
    u32x4 *mine = shared + wave * kTile;
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(d, wave + kWaves * d);
    for (int u = wave; u < a.units; u += kWaves * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + kWaves * d >= a.units)
                break;
            XOp<BITS> x[2][MT];
            unsigned xp[2][MT];                 // the lanes' own bytes
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    xp[k][t] = a.words ? xs[d][k][t] >> (8 * g) : xs[d][k][t];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const int row = kRows * j + sub;
                    mine[row * kPerRow + (place_of_chunk<BITS>(slot) ^ (row & 7))] = xf[d][t * kLoads + j];
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int p = 0; p < BITS / 4; ++p)
                        x[k][t].v[p] = mine[(lane & 15) * kPerRow + (place_in_row<BITS>(g, k, p) ^ (lane & 7))];
                __builtin_amdgcn_wave_barrier();
            }
            multiply<RT, MT, BITS>(acc, wf[d], x, ws[d], xp);
            load(d, u + kWaves * (d + D));
        }
    }
    // waves 4..7 to LDS, 0..3 add theirs, all add the four
    f32x4(*part)[kV][64] = reinterpret_cast<f32x4(*)[kV][64]>(shared);
    __syncthreads();
    if (wave >= 4) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            part[wave - 4][v][lane] = acc[v / MT][v % MT];
    }
    __syncthreads();
    if (wave < 4) {
#pragma unroll
        for (int v = 0; v < kV; ++v)
            part[wave][v][lane] += acc[v / MT][v % MT];
    }
    __syncthreads();
    for (int v = wave; v < kV; v += kWaves) {
        const f32x4 sum = (part[0][v][lane] + part[1][v][lane]) + (part[2][v][lane] + part[3][v][lane]);
        const int m = m0 + 16 * (v % MT) + (lane & 15), n = n0 + 16 * (v / MT) + 4 * g;
        if (m < a.M && n < a.N)
            store4(a, m, n, sum);
    }
}

// s_waitcnt for at most `vm` vector memory and `lgkm` LDS operations under way.
constexpr int wait_for(int vm, int lgkm) { return (vm & 15) | (vm >> 4) << 14 | 0x70 | lgkm << 8; }

// Waits until at most VM of this wave's copies to LDS and LGKM of its LDS reads
// are under way, then for the workgroup.  Not __syncthreads, which may wait for
// every copy.
template <int VM, int LGKM>
__device__ __forceinline__ void landed()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_for(VM, LGKM));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 1 KiB, or 64 dwords, from global memory to LDS without passing through
// registers: lane l's 16 or 4 bytes land at `lds` + 16 l or 4 l.
typedef __attribute__((address_space(3))) void *lds_ptr;

__device__ __forceinline__ void copy_vectors(__amdgpu_buffer_rsrc_t r, u32x4 *lds, unsigned offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, offset, 0, 0, 0);
}

__device__ __forceinline__ void copy_words(__amdgpu_buffer_rsrc_t r, u32x4 *lds, unsigned offset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 4, offset, 0, 0, 0);
}

// LDS of product_tiles, in 16-byte vectors: stages of a step (128 k) of w and x,
// and rings of units (256 k) of powers.
template <int T0>
struct TilesLayout {
    static constexpr int kXCopies = (T0 + 3) / 4;       // a wave's copies of x a step, 16 rows each
    static constexpr int kX = 16 * 64, kVecs = kX + 8 * kXCopies * 64;
    static constexpr int kStages = T0 <= 4 ? 5 : 4;
    static constexpr int kUnits = kStages / 2 + 1 + kStages % 2;    // of powers: read and under way
    static constexpr int kUnitVecs = 2 * 8 * 16;        // of w, then of x
    static constexpr int kPowers = kStages * kVecs;
    static constexpr int kBytes = (kPowers + kUnits * kUnitVecs) * 16;
};

// Many 4-bit tokens: 256 weight rows by 32 T0 tokens a workgroup of eight
// waves, each a quarter of the rows by half of the tokens, 4 x T0 products of 128 k
// a step.  All operands are copied to LDS, three or four steps ahead -- w and its
// powers lie in MFMA order, x goes by 64 bytes of a row, its 16-byte chunks in an
// order without bank conflicts -- and read into registers one step ahead of the
// products.  WORDS: rows of x's powers are whole aligned dwords, two a row and
// unit; otherwise the three aligned dwords around them are copied (each holds a
// byte of the row, so that none lies outside its memory's page).
//
// 4000 x 6288 x 7168: 100 to 105 us, 3.4 to 3.6 PFLOP/s (a library product of 4096 x
// 6400 x 7168 147 to 149 us); 8192 x 8192 x 8192 295 us, 3.7 PFLOP/s.  Bound by the matrix units,
// which are busy for half of the time, and what a step of theirs waits for: of the
// 1650 cycles of a step of 256 tokens, 1024 are products and 320 the barrier.  The
// units alone, on random data, reach 7.5 PFLOP/s at the clock that they leave.
// Copies and reads all at the start of a step: 5 % slower.  Steps of 256 k in two
// stages: the same.  Four waves of 128 rows: 40 % slower (sums go back and forth
// between register files); two workgroups of 128 rows a CU: 16 % slower.
template <int T0, bool WORDS>
__global__ __launch_bounds__(512, 2) void product_tiles(PArgs a)
{
    using L = TilesLayout<T0>;
    constexpr int kStages = L::kStages, kCopies = 3 + L::kXCopies;
    extern __shared__ u32x4 ring[];             // [kStages][L::kVecs], [L::kUnits][L::kUnitVecs]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int half = wave >> 2, quarter = wave & 3;
    // four token tiles by all row tiles at a time: the 32 workgroups of an XCD
    // then share 8 x 256 rows and 4 token tiles
    const unsigned id = logical_id();
    const unsigned per = 4u * (unsigned)a.n_tiles, grp = id / per, in = id - grp * per;
    const unsigned width = min(4u, (unsigned)a.m_tiles - 4u * grp);
    const int mt = (int)(4u * grp + in % width), nt = (int)(in / width);
    const int n0 = nt * 256, m0 = mt * 32 * T0;
    const int row_tiles = min(16, (a.N - n0 + 15) / 16), rows = min(32 * T0, a.M - m0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (long long)nt * 16 * a.units * 128,
                                                (unsigned)(row_tiles * a.units) * 2048u);
    const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.w_scale + (long long)nt * 8 * a.units * 64,
                                                 (unsigned)((row_tiles + 1) / 2 * a.units) * 256u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + m0 * a.ldx, (unsigned)((rows - 1) * a.ldx) + (unsigned)a.x_bytes);
    const unsigned char *xs0 = a.x_scale + m0 * a.ldxs;
    const unsigned shift = WORDS ? 0u : (unsigned)((uintptr_t)xs0 & 3);
    const __amdgpu_buffer_rsrc_t xsr =
        make_rsrc(xs0 - shift, (shift + (unsigned)((rows - 1) * a.ldxs) + (unsigned)a.blocks + 3u) & ~3u);
    // this wave's copies of a step: row tiles 2 wave, 2 wave + 1 of w, every eighth
    // 16 rows of x, 16-byte chunk c of row r at c ^ (r / 2 % 4); of a unit: the powers
    // of those row tiles and of 32 (WORDS) or 16 rows of x
    unsigned w_off[2], ws_off, x_off[L::kXCopies], xs_off, xs_block;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w_off[j] = (unsigned)((2 * wave + j) * a.units) * 2048u + 16u * lane;
    ws_off = (unsigned)(wave * a.units) * 256u + 4u * lane;
#pragma unroll
    for (int j = 0; j < L::kXCopies; ++j) {
        const int row = 16 * (wave + 8 * j) + (lane >> 2);
        x_off[j] = row < rows ? (unsigned)(row * a.ldx) + 16u * ((lane & 3) ^ (lane >> 3 & 3)) : kSkip;
    }
    if constexpr (WORDS) {
        const int row = 32 * wave + (lane >> 1);
        xs_block = 4u * (lane & 1);
        xs_off = row < rows ? (unsigned)(row * a.ldxs) + xs_block : kSkip;
    } else {
        const int row = 16 * wave + (lane >> 2);
        const unsigned at = shift + (unsigned)(row * a.ldxs), word = lane & 3;
        xs_off = row < rows && word < 3 ? (at & ~3u) + 4u * word : kSkip;
        // the word's first byte that is the row's own
        xs_block = 4u * word > (at & 3u) ? 4u * word - (at & 3u) : 0u;
    }
    const int steps = 2 * a.units;
    // Copy c of the kCopies of step st: w, x, then a unit's powers (of w with even
    // steps, of x with odd ones).  The same count for every step, past the last one
    // too: the waits below count them.
    const auto copy_xs = [&](int unit, int place) __attribute__((always_inline)) {
        const unsigned b = (unsigned)unit * kUnitBlocks;
        copy_words(xsr, ring + L::kPowers + place * L::kUnitVecs + 128 + wave * 16,
                   xs_off + (b + xs_block < (unsigned)a.blocks ? b : kSkip));
    };
    const auto copy = [&](int c, int st, int buf, int place) __attribute__((always_inline)) {
        u32x4 *base = ring + buf * L::kVecs;
        if (c < 2)
            copy_vectors(wr, base + (2 * wave + c) * 64, w_off[c] + (st < steps ? (unsigned)st * 1024u : kSkip));
        else if (c < 2 + L::kXCopies)
            copy_vectors(xr, base + L::kX + (wave + 8 * (c - 2)) * 64,
                         x_off[c < 2 ? 0 : c - 2 < L::kXCopies ? c - 2 : 0] + (st < steps ? (unsigned)st * 64u : kSkip));
        else if (st % 2 == 0)
            copy_words(wsr, ring + L::kPowers + place * L::kUnitVecs + wave * 16,
                       ws_off + (st < steps ? (unsigned)st * 128u : kSkip));
        else
            copy_xs(st / 2 + 1, place);
    };
    f32x4 acc[4][T0];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < T0; ++t)
            acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 wf[2][4], xf[2][T0];
    unsigned ws[2], ws_next[2], xs[2][T0];
    // Part t of the operands of a step, k its parity, in registers one step ahead of their products.
    const auto read = [&](int t, int buf, int k, int unit, int place) __attribute__((always_inline)) {
        const u32x4 *base = ring + buf * L::kVecs;
        const u32x4 *at = base + lane;
        const u32x4 *xat = base + L::kX + T0 * half * 64 + 4 * (lane & 15) + (g ^ (lane >> 1 & 3));
        const u32x4 *powers = ring + L::kPowers + place * L::kUnitVecs;
        if (k == 0 && t == 0) {
            const unsigned *wp = reinterpret_cast<const unsigned *>(powers) + 2 * quarter * 64 + lane;
            ws_next[0] = wp[0];
            ws_next[1] = wp[64];
        }
        xf[k][t] = xat[t * 64];
#pragma unroll
        for (int i = t; i < 4; i += T0)
            wf[k][i] = at[(4 * quarter + i) * 64];
        const int row = 16 * T0 * half + (lane & 15);
        // rows 16 apart begin at the same place in a dword
        const unsigned off = WORDS ? 0u : (shift + (unsigned)(row * (int)a.ldxs)) & 3u;
        const unsigned char *xp = reinterpret_cast<const unsigned char *>(powers + 128) + (WORDS ? 8 : 16) * row + off +
                                  4 * k + g;
        const bool own = WORDS || kUnitBlocks * unit + 4 * k + g < a.blocks;    // else the next row's byte
        xs[k][t] = own ? (unsigned)xp[(WORDS ? 128 : 256) * t] : 0u;
    };
    // A step's products, k its parity, with the copies of step `st` and the reads of
    // the next step between them: all at the start, the waves of a SIMD wait for the
    // memory path and LDS together.
    const auto run = [&](auto parity, int st, int buf, int st_place, int next, int unit, int place)
                         __attribute__((always_inline)) {
        constexpr int k = decltype(parity)::value;
#pragma unroll
        for (int t = 0; t < T0; ++t) {
#pragma unroll
            for (int c = t; c < kCopies; c += T0)
                copy(c, st, buf, st_place);
            read(t, next, 1 - k, unit, place);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                acc[i][t] = mma128<k>(wf[k][i], xf[k][t], acc[i][t], ws[i / 2], xs[k][t]);
                acc[i + 1][t] = mma128<2 + k>(wf[k][i + 1], xf[k][t], acc[i + 1][t], ws[i / 2], xs[k][t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // step st takes buffer st % kStages, unit u place u % kUnits
    copy_xs(0, 0);
#pragma unroll
    for (int st = 0; st < kStages; ++st)
#pragma unroll
        for (int c = 0; c < kCopies; ++c)
            copy(c, st, st, (st + 1) / 2 % L::kUnits);
    landed<(kStages - 1) * kCopies, 15>();
#pragma unroll
    for (int t = 0; t < T0; ++t)
        read(t, 0, 0, 0, 0);
    ws[0] = ws_next[0];
    ws[1] = ws_next[1];
    int buf = 0, place = 0;                     // of step st and of its unit
    int ahead = (kStages + 1) / 2 % L::kUnits;  // of the unit whose powers go with step st + kStages
    for (int st = 0; st < steps; st += 2) {
        const int unit = st / 2, next_place = place + 1 < L::kUnits ? place + 1 : 0;
        const int next_ahead = ahead + 1 < L::kUnits ? ahead + 1 : 0;
        int next = buf + 1 < kStages ? buf + 1 : 0;
        // this wave's copies of the next step have landed, and it has read all of this one
        landed<(kStages - 2) * kCopies, 0>();
        run(Const<0>{}, st + kStages, buf, ahead, next, unit, place);
        buf = next;
        next = buf + 1 < kStages ? buf + 1 : 0;
        landed<(kStages - 2) * kCopies, 0>();
        // the reads after the last step: what lies in LDS, and is not used
        run(Const<1>{}, st + 1 + kStages, buf, kStages % 2 ? ahead : next_ahead, next, unit + 1, next_place);
        buf = next;
        place = next_place;
        ahead = next_ahead;
        ws[0] = ws_next[0];
        ws[1] = ws_next[1];
    }
    __builtin_amdgcn_s_waitcnt(wait_for(0, 15));        // no copy outlives its workgroup's LDS
#pragma unroll
    for (int t = 0; t < T0; ++t) {
        const int m = m0 + 16 * (T0 * half + t) + (lane & 15);
        if (m >= a.M)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 64 * quarter + 16 * i + 4 * g;
            if (n < a.N)
                store4(a, m, n, acc[i][t]);
        }
    }
}

// LDS of product_tiles8, in 16-byte vectors, as TilesLayout.
template <int T0>
struct Tiles8Layout {
    static constexpr int kXCopies = (T0 + 1) / 2;       // a wave's copies of x a step, 8 rows each
    static constexpr int kX = 16 * 64, kVecs = kX + 8 * kXCopies * 64;
    static constexpr int kStages = T0 <= 4 ? 4 : 3;
    static constexpr int kUnits = kStages / 2 + 1 + kStages % 2;
    static constexpr int kUnitVecs = 2 * 8 * 16;
    static constexpr int kPowers = kStages * kVecs;
    static constexpr int kBytes = (kPowers + kUnits * kUnitVecs) * 16;
};

// Many 8-bit tokens: product_tiles' workgroup, with both operands converted to
// BF16 on their way from LDS to the matrix units (see multiply): a wave's w once for
// its 16 T0 tokens, x once for its 64 rows.  1501 x 6288 x 7168: 105 to 112 us, 1.2 to
// 1.29 PFLOP/s (BF16 units alone: 2.0 on random data, a library product in BF16
// 1.48 to 1.5).  The matrix units are busy for 60 % of the time; a step's conversions, some
// 150 a wave, run beside the other wave's products but for its first ones.  With
// two barriers a step and operands read in it 124 us; waves of other priorities: no
// change, or 10 % slower.
template <int T0, bool WORDS>
__global__ __launch_bounds__(512, 2) void product_tiles8(PArgs a)
{
    using L = Tiles8Layout<T0>;
    constexpr int kStages = L::kStages, kCopies = 3 + L::kXCopies;
    extern __shared__ u32x4 ring[];             // [kStages][L::kVecs], [L::kUnits][L::kUnitVecs]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const int half = wave >> 2, quarter = wave & 3;
    const unsigned id = logical_id();
    const unsigned per = 4u * (unsigned)a.n_tiles, grp = id / per, in = id - grp * per;
    const unsigned width = min(4u, (unsigned)a.m_tiles - 4u * grp);
    const int mt = (int)(4u * grp + in % width), nt = (int)(in / width);
    const int n0 = nt * 256, m0 = mt * 32 * T0;
    const int row_tiles = min(16, (a.N - n0 + 15) / 16), rows = min(32 * T0, a.M - m0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (long long)nt * 16 * a.units * 128,
                                                (unsigned)(row_tiles * a.units) * 2048u);
    const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.w_scale + (long long)nt * 8 * a.units * 64,
                                                 (unsigned)((row_tiles + 1) / 2 * a.units) * 256u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + m0 * a.ldx, (unsigned)((rows - 1) * a.ldx) + (unsigned)a.x_bytes);
    const unsigned char *xs0 = a.x_scale + m0 * a.ldxs;
    const unsigned shift = WORDS ? 0u : (unsigned)((uintptr_t)xs0 & 3);
    const __amdgpu_buffer_rsrc_t xsr =
        make_rsrc(xs0 - shift, (shift + (unsigned)((rows - 1) * a.ldxs) + (unsigned)a.blocks + 3u) & ~3u);
    unsigned w_off[2], ws_off, x_off[L::kXCopies], xs_off, xs_block;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w_off[j] = (unsigned)((2 * wave + j) * a.units) * 2048u + 16u * lane;
    ws_off = (unsigned)(wave * a.units) * 256u + 4u * lane;
    const int at = (lane & 7) ^ (lane >> 3), chunk = 2 * (at & 3) + (at >> 2);  // of a row's 128 bytes: as place_of_chunk
#pragma unroll
    for (int j = 0; j < L::kXCopies; ++j) {
        const int row = 8 * (wave + 8 * j) + (lane >> 3);
        x_off[j] = row < rows ? (unsigned)(row * a.ldx) + 16u * chunk : kSkip;
    }
    if constexpr (WORDS) {
        const int row = 32 * wave + (lane >> 1);
        xs_block = 4u * (lane & 1);
        xs_off = row < rows ? (unsigned)(row * a.ldxs) + xs_block : kSkip;
    } else {
        const int row = 16 * wave + (lane >> 2);
        const unsigned from = shift + (unsigned)(row * a.ldxs), word = lane & 3;
        xs_off = row < rows && word < 3 ? (from & ~3u) + 4u * word : kSkip;
        xs_block = 4u * word > (from & 3u) ? 4u * word - (from & 3u) : 0u;
    }
    const int steps = 2 * a.units;
    const auto copy_xs = [&](int unit, int place) __attribute__((always_inline)) {
        const unsigned b = (unsigned)unit * kUnitBlocks;
        copy_words(xsr, ring + L::kPowers + place * L::kUnitVecs + 128 + wave * 16,
                   xs_off + (b + xs_block < (unsigned)a.blocks ? b : kSkip));
    };
    const auto copy = [&](int c, auto parity, int st, int buf, int place) __attribute__((always_inline)) {
        u32x4 *base = ring + buf * L::kVecs;
        if (c < 2)
            copy_vectors(wr, base + (2 * wave + c) * 64, w_off[c] + (st < steps ? (unsigned)st * 1024u : kSkip));
        else if (c < 2 + L::kXCopies)           // past K the codes are the next row's and may be NaN
            copy_vectors(xr, base + L::kX + (wave + 8 * (c - 2)) * 64,
                         x_off[c < 2 ? 0 : c - 2 < L::kXCopies ? c - 2 : 0] +
                             (st * 128 + 16 * chunk < a.x_bytes ? (unsigned)st * 128u : kSkip));
        else if (decltype(parity)::value == 0)
            copy_words(wsr, ring + L::kPowers + place * L::kUnitVecs + wave * 16,
                       ws_off + (st < steps ? (unsigned)st * 128u : kSkip));
        else
            copy_xs(st / 2 + 1, place);
    };
    f32x4 acc[4][T0];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < T0; ++t)
            acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 wf[4], xf[2][T0];
    unsigned ws[2], xs[T0];
    // A wave's operands of a step, each read one step ahead, into the registers
    // that the step before has just converted from.
    const auto read_w = [&](int i, int buf, int place) __attribute__((always_inline)) {
        wf[i] = (ring + buf * L::kVecs + lane + 4 * quarter * 64)[i * 64];
        if (i % 2 == 0)
            ws[i / 2] = (reinterpret_cast<const unsigned *>(ring + L::kPowers + place * L::kUnitVecs) + 2 * quarter * 64 +
                         lane)[i / 2 * 64];
    };
    const auto read_powers = [&](int t, int k, int unit, int place) __attribute__((always_inline)) {
        const int row = 16 * T0 * half + (lane & 15);
        const unsigned off = WORDS ? 0u : (shift + (unsigned)(row * (int)a.ldxs)) & 3u;
        const unsigned char *p = reinterpret_cast<const unsigned char *>(ring + L::kPowers + place * L::kUnitVecs + 128) +
                                 (WORDS ? 8 : 16) * row + off + 4 * k + g;
        const bool own = WORDS || kUnitBlocks * unit + 4 * k + g < a.blocks;
        xs[t] = own ? (unsigned)p[(WORDS ? 128 : 256) * t] : 0u;
    };
    // Half h (16 values of its block for each lane) of token tile t.
    const auto read_x = [&](int t, int buf, int h) __attribute__((always_inline)) {
        xf[h][t] =
            (ring + buf * L::kVecs + L::kX + T0 * half * 128 + 8 * (lane & 15) + (place_in_row<8>(g, 0, h) ^ (lane & 7)))[t * 128];
    };
    copy_xs(0, 0);
#pragma unroll
    for (int st = 0; st < kStages; ++st)
#pragma unroll
        for (int c = 0; c < kCopies; ++c)
            if (st % 2 == 0)
                copy(c, Const<0>{}, st, st, (st + 1) / 2 % L::kUnits);
            else
                copy(c, Const<1>{}, st, st, (st + 1) / 2 % L::kUnits);
    landed<(kStages - 1) * kCopies, 15>();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        read_w(i, 0, 0);
#pragma unroll
    for (int t = 0; t < T0; ++t) {
        read_x(t, 0, 0);
        read_x(t, 0, 1);
        read_powers(t, 0, 0, 0);
    }
    // A step's products, k its parity, with the copies of step `st` and the reads of
    // the next step between them.
    const auto run = [&](auto parity, int st, int buf, int st_place, int next, int unit, int place)
                         __attribute__((always_inline)) {
        constexpr int k = decltype(parity)::value;
        float wp[4], xp[T0];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            wp[i] = power_of(ws[i / 2] >> (16 * (i & 1) + 8 * k) & 0xFFu);
#pragma unroll
        for (int t = 0; t < T0; ++t)
            xp[t] = power_of(xs[t]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 wb[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    wb[j][i] = bf16_of_4(wf[i][2 * h + j], wp[i]);
#pragma unroll
            for (int t = 0; t < T0; ++t) {
                bf16x8 xb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    xb[j] = bf16_of_8(xf[h][t][2 * j], xf[h][t][2 * j + 1], xp[t]);
#pragma unroll
                for (int c = h * T0 + t; c < kCopies; c += 2 * T0)
                    copy(c, Const<(k + kStages) % 2>{}, st, buf, st_place);
                read_x(t, next, h);
                if (h == 1) {
#pragma unroll
                    for (int i = t; i < 4; i += T0)
                        read_w(i, next, place);
                    read_powers(t, 1 - k, unit, place);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][i], xb[j], acc[i][t], 0, 0, 0);
            }
        }
    };
    // step st takes buffer st % kStages, unit u place u % kUnits
    int buf = 0, place = 0;
    int ahead = (kStages + 1) / 2 % L::kUnits;  // of the unit whose powers go with step st + kStages
    for (int st = 0; st < steps; st += 2) {
        const int unit = st / 2, next_place = place + 1 < L::kUnits ? place + 1 : 0;
        const int next_ahead = ahead + 1 < L::kUnits ? ahead + 1 : 0;
        int next = buf + 1 < kStages ? buf + 1 : 0;
        // this wave's copies of the next step have landed, and it has read all of this one
        landed<(kStages - 2) * kCopies, 0>();
        run(Const<0>{}, st + kStages, buf, ahead, next, unit, place);
        buf = next;
        next = buf + 1 < kStages ? buf + 1 : 0;
        landed<(kStages - 2) * kCopies, 0>();
        run(Const<1>{}, st + 1 + kStages, buf, kStages % 2 ? ahead : next_ahead, next, unit + 1, next_place);
        buf = next;
        place = next_place;
        ahead = next_ahead;
    }
    __builtin_amdgcn_s_waitcnt(wait_for(0, 15));        // no copy outlives its workgroup's LDS
#pragma unroll
    for (int t = 0; t < T0; ++t) {
        const int m = m0 + 16 * (T0 * half + t) + (lane & 15);
        if (m >= a.M)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 64 * quarter + 16 * i + 4 * g;
            if (n < a.N)
                store4(a, m, n, acc[i][t]);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

bool is_bits(int bits) { return bits == 4 || bits == 8; }

// Rows of a launch whose octets are counted in 31 bits.
int rows_of_launch(int per_row) { return per_row >= 1 << 30 ? 1 : (1 << 30) / per_row; }

template <int TYPE, int BITS>
const void *quantize_kernel(bool gate, bool vec, bool many)
{
    if (!vec)
        return gate ? reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, true, false, 1>)
                    : reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, false, false, 1>);
    if (gate)
        return many ? reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, true, true, 2>)
                    : reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, true, true, 1>);
    return many ? reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, false, true, 4>)
                : reinterpret_cast<const void *>(quantize_octets<TYPE, BITS, false, true, 1>);
}

template <int BITS>
const void *quantize_kernel_of(int type, bool gate, bool vec, bool many)
{
    return type == SKINNY_TYPE_F32   ? quantize_kernel<SKINNY_TYPE_F32, BITS>(gate, vec, many)
           : type == SKINNY_TYPE_F16 ? quantize_kernel<SKINNY_TYPE_F16, BITS>(gate, vec, many)
                                     : quantize_kernel<SKINNY_TYPE_BF16, BITS>(gate, vec, many);
}

// Two units ahead for up to four 8-bit tokens, whose loads and registers are
// few (6288 x 7168: 6.8 against 7.2 us); one elsewhere.
template <int RT, int MT, int BITS, int XR, bool NT>
const void *rows_fn()
{
    return reinterpret_cast<const void *>(product_rows<RT, MT, BITS, BITS == 8 && XR == 4 && RT <= 2 ? 2 : 1, XR, NT>);
}

// A single token tile takes the weight past by; several have whole tiles of x.
template <int RT, int BITS>
const void *rows_kernel_of(const Product &p)
{
    if constexpr (RT > 1)
        if (p.t == 2)
            return p.once ? rows_fn<RT, 2, BITS, 16, true>() : rows_fn<RT, 2, BITS, 16, false>();
    return !p.once          ? rows_fn<RT, 1, BITS, 16, false>()
           : p.x_rows == 4  ? rows_fn<RT, 1, BITS, 4, true>()
           : p.x_rows == 8  ? rows_fn<RT, 1, BITS, 8, true>()
                            : rows_fn<RT, 1, BITS, 16, true>();
}

template <int BITS>
const void *rows_kernel(const Product &p)
{
    return p.r == 1 ? rows_kernel_of<1, BITS>(p) : p.r == 2 ? rows_kernel_of<2, BITS>(p) : rows_kernel_of<4, BITS>(p);
}

template <int T0>
const void *tiles_fn(int bits, bool words)
{
    if constexpr (T0 <= kAnyTiles)
        if (!words)
            return bits == 4 ? reinterpret_cast<const void *>(product_tiles<T0, false>)
                             : reinterpret_cast<const void *>(product_tiles8<T0, false>);
    if constexpr (T0 <= kTiles8)
        if (bits == 8)
            return reinterpret_cast<const void *>(product_tiles8<T0, true>);
    return reinterpret_cast<const void *>(product_tiles<T0, true>);
}

// t0 from kFewest to most_tiles(bits, words).
const void *tiles_kernel(int t0, int bits, bool words)
{
    return t0 == 2 ? tiles_fn<2>(bits, words) : t0 == 3 ? tiles_fn<3>(bits, words) : t0 == 4 ? tiles_fn<4>(bits, words)
         : t0 == 5 ? tiles_fn<5>(bits, words) : t0 == 6 ? tiles_fn<6>(bits, words) : t0 == 7 ? tiles_fn<7>(bits, words)
                                                                                           : tiles_fn<8>(bits, words);
}

template <int T0>
int tiles_lds_of(int bits)
{
    return bits == 4 ? TilesLayout<T0>::kBytes : Tiles8Layout<T0>::kBytes;
}

int tiles_lds(int t0, int bits)
{
    return t0 == 2 ? tiles_lds_of<2>(bits) : t0 == 3 ? tiles_lds_of<3>(bits) : t0 == 4 ? tiles_lds_of<4>(bits)
         : t0 == 5 ? tiles_lds_of<5>(bits) : t0 == 6 ? tiles_lds_of<6>(bits) : t0 == 7 ? tiles_lds_of<7>(bits)
                                                                                     : tiles_lds_of<8>(bits);
}

hipError_t launch_product(PArgs a, int bits, hipStream_t stream)
{
    constexpr unsigned kThreads = 512;
    constexpr int kSplit = 256;                 // rows and tokens of the largest tile: both halves begin on one
    void *params[] = {&a};
    const bool words = a.words != 0;
    const Product p = product_of(a.M, a.N, bits, words);
    if (p.n_tiles * p.m_tiles > kMostThreads / kThreads) {
        // more threads than a launch may have: the two halves of the longer side, one after the other
        const int bytes = type_bytes(a.type);
        PArgs second = a;
        if (a.M >= a.N) {
            const int first = a.M / 2 / kSplit * kSplit;
            second.M = a.M - first;
            second.x += first * a.ldx;
            second.x_scale += first * a.ldxs;
            second.out = static_cast<char *>(a.out) + first * a.ldo * bytes;
            if (a.res)
                second.res = static_cast<const char *>(a.res) + first * a.ldr * bytes;
            a.M = first;
        } else {
            const int first = a.N / 2 / kSplit * kSplit;
            second.N = a.N - first;
            second.w += (long long)(first / 16) * a.units * 128;
            second.w_scale += (long long)(first / 32) * a.units * 64;
            second.out = static_cast<char *>(a.out) + (long long)first * bytes;
            if (a.res)
                second.res = static_cast<const char *>(a.res) + (long long)first * bytes;
            a.N = first;
        }
        const hipError_t e = launch_product(a, bits, stream);
        return e == hipSuccess ? launch_product(second, bits, stream) : e;
    }
    a.n_tiles = (int)p.n_tiles;
    a.m_tiles = (int)p.m_tiles;
    const void *fn = p.many ? tiles_kernel(p.t, bits, words) : bits == 4 ? rows_kernel<4>(p) : rows_kernel<8>(p);
    return hipLaunchKernel(fn, dim3((unsigned)(p.n_tiles * p.m_tiles)), dim3(kThreads), params,
                           p.many ? (size_t)tiles_lds(p.t, bits) : 0, stream);
}

// Dynamic LDS past 64 KiB has to be asked for, on every device that the kernels run on.
hipError_t raise_limits()
{
    for (const int bits : {4, 8})
        for (const bool words : {false, true})
            for (int t0 = kFewest; t0 <= most_tiles(bits, words); ++t0) {
                const hipError_t e = hipFuncSetAttribute(
                    tiles_kernel(t0, bits, words), hipFuncAttributeMaxDynamicSharedMemorySize, tiles_lds(t0, bits));
                if (e != hipSuccess)
                    return e;
            }
    return hipSuccess;
}

// fn(first vector, launch's end) over count vectors of 256-thread workgroups, in launches of fewer than 2^32 threads.
template <typename F>
hipError_t over_launches(long long count, F launch)
{
    constexpr long long kMost = 1LL << 31;
    hipError_t e = hipSuccess;
    for (long long first = 0; e == hipSuccess && first < count; first += kMost) {
        const long long left = count - first < kMost ? count - first : kMost;
        e = launch(first, dim3((unsigned)((left + 255) / 256)));
    }
    return e;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

skinny_status skinny_quantize_blocks(const void *x, skinny_type type, int M, int K, long long ldx, const void *gate,
                                     long long ldg, int bits, void *q, long long ldq, void *scale, long long lds,
                                     void *stream)
{
    if (!is_type((int)type))
        return bad(SKINNY_ERR_INVALID_ARG, "type %d is none of BF16, F32 and F16", (int)type);
    if (!is_bits(bits))
        return bad(SKINNY_ERR_INVALID_ARG, "bits=%d is neither 4 nor 8", bits);
    if (M < 0 || K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d and K=%d: M >= 0 and K >= 1 are needed", M, K);
    if (K % kBlock)
        return bad(SKINNY_ERR_SHAPE, "K=%d must be a multiple of 32, whole blocks", K);
    if (M == 0)
        return SKINNY_OK;
    if (!x || !q || !scale)
        return bad(SKINNY_ERR_INVALID_ARG, "x, q or scale is NULL");
    const int row_bytes = K / 8 * bits, blocks = K / kBlock;
    if (ldx < K || (gate && ldg < K) || ldq < row_bytes || lds < blocks)
        return bad(SKINNY_ERR_SHAPE, "ldx=%lld and ldg=%lld must be at least K=%d, ldq=%lld %d and lds=%lld %d", ldx, ldg,
                   K, ldq, row_bytes, lds, blocks);
    const int eb = type_bytes((int)type);
    if ((uintptr_t)x % eb || (uintptr_t)gate % eb)
        return bad(SKINNY_ERR_ALIGN, "x and gate must be aligned to their elements");
    const bool vec = (uintptr_t)x % 16 == 0 && ldx * eb % 16 == 0 &&
                     (!gate || ((uintptr_t)gate % 16 == 0 && ldg * eb % 16 == 0)) && (uintptr_t)q % bits == 0 &&
                     ldq % bits == 0;
    const int per_row = K / 8, most = rows_of_launch(per_row);
    const bool whole = ldx == K && (!gate || ldg == K) && ldq == row_bytes && lds == blocks;
    for (int done = 0; done < M;) {
        const int rows = M - done < most ? M - done : most;
        BArgs a{};
        a.x = static_cast<const char *>(x) + done * ldx * eb;
        a.gate = gate ? static_cast<const char *>(gate) + done * ldg * eb : nullptr;
        a.q = static_cast<unsigned char *>(q) + done * ldq;
        a.scale = static_cast<unsigned char *>(scale) + done * lds;
        a.ldx = ldx;
        a.ldg = ldg;
        a.ldq = ldq;
        a.lds = lds;
        a.octets = (unsigned)rows * (unsigned)per_row;
        // rows one after the other are one long row
        a.per_row = whole ? a.octets : (unsigned)per_row;
        a.by_row = make_fastdiv(a.per_row);
        // several octets a thread once they fill the chip's threads all the same: more loads under way
        const bool many = a.octets >= 1u << 20;
        const unsigned per_group = 256u * (!vec || !many ? 1u : gate ? 2u : 4u);
        const void *fn = bits == 4 ? quantize_kernel_of<4>((int)type, gate != nullptr, vec, many)
                                   : quantize_kernel_of<8>((int)type, gate != nullptr, vec, many);
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(fn, dim3((a.octets + per_group - 1) / per_group), dim3(256), params, 0,
                                             (hipStream_t)stream);
        if (e != hipSuccess)
            return hip_bad(e, "quantize launch");
        done += rows;
    }
    return SKINNY_OK;
}

skinny_status skinny_expand_blocks(const void *q, int bits, int M, int K, long long ldq, const void *scale,
                                   long long lds, void *out, skinny_type type, long long ldo, void *stream)
{
    if (!is_type((int)type))
        return bad(SKINNY_ERR_INVALID_ARG, "type %d is none of BF16, F32 and F16", (int)type);
    if (!is_bits(bits))
        return bad(SKINNY_ERR_INVALID_ARG, "bits=%d is neither 4 nor 8", bits);
    if (M < 0 || K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d and K=%d: M >= 0 and K >= 1 are needed", M, K);
    if (K % kBlock)
        return bad(SKINNY_ERR_SHAPE, "K=%d must be a multiple of 32, whole blocks", K);
    if (M == 0)
        return SKINNY_OK;
    if (!q || !scale || !out)
        return bad(SKINNY_ERR_INVALID_ARG, "q, scale or out is NULL");
    const int row_bytes = K / 8 * bits, blocks = K / kBlock;
    if (ldo < K || ldq < row_bytes || lds < blocks)
        return bad(SKINNY_ERR_SHAPE, "ldo=%lld must be at least K=%d, ldq=%lld %d and lds=%lld %d", ldo, K, ldq,
                   row_bytes, lds, blocks);
    const int eb = type_bytes((int)type);
    if ((uintptr_t)out % eb)
        return bad(SKINNY_ERR_ALIGN, "out must be aligned to its elements");
    const bool vec = (uintptr_t)out % 16 == 0 && ldo * eb % 16 == 0 && (uintptr_t)q % bits == 0 && ldq % bits == 0;
    const int per_row = K / 8, most = rows_of_launch(per_row);
    const bool whole = ldo == K && ldq == row_bytes && lds == blocks;
    for (int done = 0; done < M;) {
        const int rows = M - done < most ? M - done : most;
        XArgs a{};
        a.q = static_cast<const unsigned char *>(q) + done * ldq;
        a.scale = static_cast<const unsigned char *>(scale) + done * lds;
        a.out = static_cast<char *>(out) + done * ldo * eb;
        a.ldq = ldq;
        a.lds = lds;
        a.ldo = ldo;
        a.type = (int)type;
        a.octets = (unsigned)rows * (unsigned)per_row;
        a.per_row = whole ? a.octets : (unsigned)per_row;
        a.by_row = make_fastdiv(a.per_row);
        const void *fn = bits == 4 ? (vec ? reinterpret_cast<const void *>(expand_octets<4, true>)
                                          : reinterpret_cast<const void *>(expand_octets<4, false>))
                                   : (vec ? reinterpret_cast<const void *>(expand_octets<8, true>)
                                          : reinterpret_cast<const void *>(expand_octets<8, false>));
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(fn, dim3((a.octets + 255) / 256), dim3(256), params, 0,
                                             (hipStream_t)stream);
        if (e != hipSuccess)
            return hip_bad(e, "expand launch");
        done += rows;
    }
    return SKINNY_OK;
}

skinny_status skinny_mxfp4_prepare(const void *Wq, int N, int K, long long ldw, const void *w_scale, long long ldws,
                                   skinny_type out_type, void *stream, skinny_mxfp4_plan **plan)
{
    if (!plan)
        return bad(SKINNY_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    if (!Wq || !w_scale || N < 1 || K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "Wq or w_scale is NULL, or N=%d, K=%d is not positive", N, K);
    if (!is_type((int)out_type))
        return bad(SKINNY_ERR_INVALID_ARG, "output type %d is none of BF16, F32 and F16", (int)out_type);
    if (N > kMaxRows)
        return bad(SKINNY_ERR_SHAPE, "N=%d: at most %d", N, kMaxRows);
    if (K % kBlock || K > kMaxPitch)
        return bad(SKINNY_ERR_SHAPE, "K=%d must be a multiple of 32, at most 2^22", K);
    const int blocks = K / kBlock, units = (blocks + kUnitBlocks - 1) / kUnitBlocks;
    if (ldw < K / 2 || ldws < blocks)
        return bad(SKINNY_ERR_SHAPE, "ldw=%lld must be at least %d bytes and ldws=%lld %d", ldw, K / 2, ldws, blocks);
    const long long tiles = ((long long)N + 15) / 16, count = tiles * units * 128;
    const long long pairs = (tiles + 1) / 2, scales = pairs * units * 64;
    if (count >= 1LL << 36)
        return bad(SKINNY_ERR_SHAPE, "N=%d by K=%d is too large", N, K);
    skinny_mxfp4_plan *p = new (std::nothrow) skinny_mxfp4_plan{N, K, units, out_type, 0, nullptr, nullptr};
    if (!p)
        return bad(SKINNY_ERR_NOMEM, "host allocation failed");
    int cus = 0;
    const skinny_status st = current_gfx950(&p->device, &cus);
    if (st != SKINNY_OK) {
        delete p;
        return st;
    }
    hipError_t e = raise_limits();
    if (e == hipSuccess)
        e = hipMalloc(&p->w, (size_t)count * 16);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&p->w_scale), (size_t)scales * 4);
    const hipStream_t s = (hipStream_t)stream;
    int n = N, b = blocks, us = units;
    if (e == hipSuccess)
        e = over_launches(count, [&](long long first, dim3 grid) {
            const unsigned char *src = static_cast<const unsigned char *>(Wq);
            u32x4 *dst = static_cast<u32x4 *>(p->w);
            long long ld = ldw, c = count;
            void *params[] = {&src, &ld, &n, &b, &us, &dst, &first, &c};
            return hipLaunchKernel(reinterpret_cast<const void *>(lay_out), grid, dim3(256), params, 0, s);
        });
    if (e == hipSuccess)
        e = over_launches(scales, [&](long long first, dim3 grid) {
            const unsigned char *src = static_cast<const unsigned char *>(w_scale);
            unsigned *dst = p->w_scale;
            long long ld = ldws, c = scales;
            void *params[] = {&src, &ld, &n, &b, &us, &dst, &first, &c};
            return hipLaunchKernel(reinterpret_cast<const void *>(lay_out_scales), grid, dim3(256), params, 0, s);
        });
    if (e == hipSuccess)
        e = hipStreamSynchronize(s);
    if (e != hipSuccess) {
        (void)hipFree(p->w);
        (void)hipFree(p->w_scale);
        delete p;
        return hip_bad(e, "mxfp4 prepare");
    }
    *plan = p;
    return SKINNY_OK;
}

skinny_status skinny_mxfp4_run(const skinny_mxfp4_plan *p, const void *xq, int bits, long long ldx, const void *x_scale,
                               long long ldxs, const void *residual, long long ldr, void *out, long long ldo, int M,
                               void *stream)
{
    if (!p)
        return bad(SKINNY_ERR_INVALID_ARG, "plan is NULL");
    if (!is_bits(bits))
        return bad(SKINNY_ERR_INVALID_ARG, "bits=%d is neither 4 nor 8", bits);
    if (M < 0)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d is negative", M);
    if (M > kMaxRows)
        return bad(SKINNY_ERR_SHAPE, "M=%d: at most %d", M, kMaxRows);
    if (M == 0)
        return SKINNY_OK;
    if (!xq || !x_scale || !out)
        return bad(SKINNY_ERR_INVALID_ARG, "xq, x_scale or out is NULL");
    const int row_bytes = p->K / 8 * bits, blocks = p->K / kBlock;
    if (ldx < row_bytes || ldx % 16 || ldx > kMaxPitch || ldxs < blocks || ldxs > kMaxPitch)
        return bad(SKINNY_ERR_SHAPE, "ldx=%lld must be a multiple of 16 bytes from %d to 2^22, ldxs=%lld from %d to 2^22",
                   ldx, row_bytes, ldxs, blocks);
    if (ldo < p->N || (residual && ldr < p->N))
        return bad(SKINNY_ERR_SHAPE, "ldo=%lld and ldr=%lld must be at least N=%d", ldo, ldr, p->N);
    const int eb = type_bytes((int)p->out);
    if ((uintptr_t)xq % 16 || (uintptr_t)out % eb || (uintptr_t)residual % eb)
        return bad(SKINNY_ERR_ALIGN, "xq must be 16-byte aligned, out and residual to their elements");
    PArgs a{};
    a.w = static_cast<const u32x4 *>(p->w);
    a.w_scale = p->w_scale;
    a.x = static_cast<const unsigned char *>(xq);
    a.x_scale = static_cast<const unsigned char *>(x_scale);
    a.res = residual;
    a.out = out;
    a.ldx = ldx;
    a.ldxs = ldxs;
    a.ldr = ldr;
    a.ldo = ldo;
    a.M = M;
    a.N = p->N;
    a.x_bytes = row_bytes;
    a.blocks = blocks;
    a.units = p->units;
    a.type = p->out;
    a.words = blocks % 4 == 0 && ldxs % 4 == 0 && (uintptr_t)x_scale % 4 == 0;
    a.vec = (uintptr_t)out % (4 * eb) == 0 && ldo % 4 == 0 && (uintptr_t)residual % (4 * eb) == 0 && ldr % 4 == 0;
    const hipError_t e = launch_product(a, bits, (hipStream_t)stream);
    return e == hipSuccess ? SKINNY_OK : hip_bad(e, "mxfp4 product launch");
}

void skinny_mxfp4_destroy(skinny_mxfp4_plan *p)
{
    if (!p)
        return;
    int cur = -1;
    (void)hipGetDevice(&cur);
    if (cur != p->device)
        (void)hipSetDevice(p->device);
    (void)hipDeviceSynchronize();
    (void)hipFree(p->w);
    (void)hipFree(p->w_scale);
    if (cur != p->device && cur >= 0)
        (void)hipSetDevice(cur);
    delete p;
}

}  // extern "C"
