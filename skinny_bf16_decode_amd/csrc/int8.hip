// HIP kernels and entry points of products in 8-bit integers for gfx950 (CDNA4):
//
//   q[m][k]   = round(x[m][k] 127 / max_k |x[m][k]|),  scale[m] = max_k |x[m][k]| / 127
//   out[m][n] = (sum_k q[m][k] Wq[n][k]) x_scale[m] w_scale[n] (+ residual[m][n])
//
// The sums run in 32-bit integers (v_mfma_i32_16x16x64_i8) and are exact, so
// neither the order of a sum nor a K split changes a result.
#include <hip/hip_runtime.h>

#include <new>
#include <stdarg.h>
#include <stdio.h>

#include "skinny_internal.h"

// A prepared 8-bit weight.
struct skinny_int8_plan {
    int N, K;
    int pitch;                  // steps of a row tile in w: K / 64, rounded up to an even number
    skinny_type out;
    int device;
    void *w;                    // [N / 16][pitch][64 lanes][16 bytes], zero past N and K
    float *w_scale;             // [N]
};

namespace skinny {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kStep = 64;       // bytes of K a 16x16x64 MFMA takes

// ---------------------------------------------------------------------------
// Rows to 8-bit integers
// ---------------------------------------------------------------------------

template <int TYPE>
struct Elem;
template <>
struct Elem<SKINNY_TYPE_BF16> {
    typedef unsigned short raw;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(raw v) { return __uint_as_float((unsigned)v << 16); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(raw, (__bf16)v); }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[2 * i] = __uint_as_float(w << 16);
            f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
};
template <>
struct Elem<SKINNY_TYPE_F16> {
    typedef unsigned short raw;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(raw, (_Float16)v); }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[2 * i] = get((raw)(w & 0xFFFFu));
            f[2 * i + 1] = get((raw)(w >> 16));
        }
    }
};
template <>
struct Elem<SKINNY_TYPE_F32> {
    typedef float raw;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(raw v) { return v; }
    static __device__ __forceinline__ raw put(float v) { return v; }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned int w = v[i];
            f[i] = __uint_as_float(w);
        }
    }
};

struct QArgs {
    const void *x;
    signed char *q;
    float *scale;
    long long ldx, ldq;
    int K;
};

// Magnitude bits of an fp32 value: ordered as unsigned integers like the
// values, with infinity and NaN (which a maximum of floats would drop) on top.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ unsigned wave_max_u(unsigned v)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const unsigned o = (unsigned)__shfl_xor((int)v, s, 64);
        v = o > v ? o : v;
    }
    return v;
}

// What a row's values are multiplied with, in two steps: lift (a power of
// two), then 127 / (lifted maximum), rounded to fp32 once.
struct RowScale {
    float lift, inverse;
    bool fine;                  // finite and not all zero
};

__device__ __forceinline__ RowScale row_scale(unsigned top_bits, float &scale)
{
    RowScale r;
    const float top = __uint_as_float(top_bits);
    const bool finite = top_bits < 0x7F800000u;
    r.fine = finite && top_bits != 0u;
    r.lift = top < 0x1p-60f ? 0x1p64f : 1.0f;
    r.inverse = r.fine ? __fdiv_rn(127.0f, top * r.lift) : 0.0f;
    scale = finite ? __fdiv_rn(top, 127.0f) : __uint_as_float(0x7FC00000u);
    return r;
}

__device__ __forceinline__ int to_int8(float v, const RowScale &r)
{
    return r.fine ? (int)rintf(__fmul_rn(__fmul_rn(v, r.lift), r.inverse)) : 0;
}

// One workgroup a row.  The row is read once: up to VECS 16-byte vectors a
// thread stay in registers between the maximum and the rounding (VECS = 0: the
// row is longer than that, and read again).  Bound by bytes: K (2 or 4 read +
// 1 1 written) a row.  6001 x 7168 in BF16: 23.2 us, 5.6 TB/s, in fp32 (4-byte
// stores) 38 us, 5.7 TB/s; 4 rows: 2.9 us.
template <int TYPE, int VECS>
__global__ __launch_bounds__(1024) void quantize_vector(QArgs a)
{
    using E = Elem<TYPE>;
    constexpr int kVec = E::kVec;
    __shared__ unsigned tops[16];
    const int threads = blockDim.x, tid = threadIdx.x;
    const typename E::raw *x = static_cast<const typename E::raw *>(a.x) + blockIdx.x * a.ldx;
    signed char *q = a.q + blockIdx.x * a.ldq;
    const int vecs = a.K / kVec;
    u32x4 keep[VECS ? VECS : 1];
    unsigned top = 0;
    const auto see = [&](u32x4 v) {
        float f[kVec];
        E::unpack(v, f);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const unsigned m = mag(f[e]);
            top = m > top ? m : top;
        }
    };
    if constexpr (VECS > 0) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            keep[i] = u32x4{0u, 0u, 0u, 0u};
            if (tid + i * threads < vecs)
                keep[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x) + tid + i * threads);
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            see(keep[i]);
    } else {
        for (int i = tid; i < vecs; i += threads)
            see(reinterpret_cast<const u32x4 *>(x)[i]);
    }
    top = wave_max_u(top);
    if (threads > 64) {
        if ((tid & 63) == 0)
            tops[tid >> 6] = top;
        __syncthreads();
        for (int w = 0; w < threads >> 6; ++w)
            top = tops[w] > top ? tops[w] : top;
    }
    float scale;
    const RowScale r = row_scale(top, scale);
    if (tid == 0)
        a.scale[blockIdx.x] = scale;
    const auto write = [&](u32x4 v, int i) {
        float f[kVec];
        E::unpack(v, f);
        unsigned w[kVec / 4];
#pragma unroll
        for (int e = 0; e < kVec; e += 4)
            w[e / 4] = (unsigned)(to_int8(f[e], r) & 0xFF) | (unsigned)(to_int8(f[e + 1], r) & 0xFF) << 8 |
                       (unsigned)(to_int8(f[e + 2], r) & 0xFF) << 16 | (unsigned)to_int8(f[e + 3], r) << 24;
        if constexpr (kVec == 8)
            *reinterpret_cast<u32x2 *>(q + (long long)i * 8) = u32x2{w[0], w[1]};
        else
            *reinterpret_cast<unsigned *>(q + (long long)i * 4) = w[0];
    };
    if constexpr (VECS > 0) {
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (tid + i * threads < vecs)
                write(keep[i], tid + i * threads);
    } else {
        for (int i = tid; i < vecs; i += threads)
            write(reinterpret_cast<const u32x4 *>(x)[i], i);
    }
}

// Any K, pitch and alignment, an element at a time.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_element(QArgs a)
{
    using E = Elem<TYPE>;
    __shared__ unsigned tops[4];
    const int tid = threadIdx.x;
    const typename E::raw *x = static_cast<const typename E::raw *>(a.x) + blockIdx.x * a.ldx;
    signed char *q = a.q + blockIdx.x * a.ldq;
    unsigned top = 0;
    for (int i = tid; i < a.K; i += 256) {
        const unsigned m = mag(E::get(x[i]));
        top = m > top ? m : top;
    }
    top = wave_max_u(top);
    if ((tid & 63) == 0)
        tops[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w)
        top = tops[w] > top ? tops[w] : top;
    float scale;
    const RowScale r = row_scale(top, scale);
    if (tid == 0)
        a.scale[blockIdx.x] = scale;
    for (int i = tid; i < a.K; i += 256)
        q[i] = (signed char)to_int8(E::get(x[i]), r);
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

struct PArgs {
    const u32x4 *w;             // laid out by lay_out
    const signed char *x;
    const float *x_scale, *w_scale;
    const void *res;
    void *out;
    long long ldx, ldr, ldo;
    int M, N, K;
    int pitch;                  // steps of 64 a row tile holds in w: even, zeros past K
    int type;                   // skinny_type of out and res
    int vec;                    // out and res take four columns at once
    int m_tiles;                // token tiles of the launch
    int n_tiles;                // tiles of weight rows
};

// Weight rows into MFMA operands: lane l of step s of row tile t takes row
// 16 t + l % 16, bytes 64 s + 16 (l / 16) .. + 15, so that a wave's load of an
// operand is 1 KiB in a row.
// Vectors `first` .. count - 1.
__global__ __launch_bounds__(256) void lay_out(const signed char *w, long long ldw, int N, int K, int pitch,
                                               u32x4 *out, long long first, long long count)
{
    const long long i = first + (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= count)
        return;
    const int lane = (int)(i & 63);
    const long long st = i >> 6;
    const long long n = st / pitch * 16 + (lane & 15);
    const int k = (int)(st % pitch) * kStep + 16 * (lane >> 4);
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (n < N && k < K) {                       // K % 16 == 0: a chunk is all in or all out
        const signed char *p = w + n * ldw + k;
        if (((uintptr_t)p & 15) == 0) {
            v = *reinterpret_cast<const u32x4 *>(p);
        } else {
            unsigned b[4] = {0, 0, 0, 0};
            for (int j = 0; j < 16; ++j)
                b[j / 4] |= (unsigned)(unsigned char)p[j] << (8 * (j % 4));
            v = u32x4{b[0], b[1], b[2], b[3]};
        }
    }
    out[i] = v;
}

// Four outputs of one token, columns n .. n + 3, from the exact sums.
template <int OUT>
__device__ __forceinline__ void store4_as(const PArgs &a, int m, int n, i32x4 sum, float xs, f32x4 ws)
{
    using E = Elem<OUT>;
    typedef __attribute__((ext_vector_type(4))) typename E::raw raw4;
    typename E::raw *o = static_cast<typename E::raw *>(a.out) + m * a.ldo + n;
    const typename E::raw *res = a.res ? static_cast<const typename E::raw *>(a.res) + m * a.ldr + n : nullptr;
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        v[r] = (float)sum[r] * xs * ws[r];
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

__device__ __forceinline__ void store4(const PArgs &a, int m, int n, i32x4 sum, float xs, f32x4 ws)
{
    if (a.type == SKINNY_TYPE_BF16)
        store4_as<SKINNY_TYPE_BF16>(a, m, n, sum, xs, ws);
    else if (a.type == SKINNY_TYPE_F32)
        store4_as<SKINNY_TYPE_F32>(a, m, n, sum, xs, ws);
    else
        store4_as<SKINNY_TYPE_F16>(a, m, n, sum, xs, ws);
}

__device__ __forceinline__ f32x4 channel_scales(const PArgs &a, int n)
{
    f32x4 s;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        s[r] = n + r < a.N ? a.w_scale[n + r] : 0.0f;
    return s;
}

__device__ __forceinline__ i32x4 mma64(u32x4 w, u32x4 x, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0,
                                                 0);
}

// A buffer load whose offset is past its resource reads zero and touches no
// memory; loads to be skipped take this one (resources are smaller: 256 rows of
// x at pitches below 2^22, four row tiles of w).  Offsets are all in the
// per-lane part, the one that is checked whatever its value.
constexpr unsigned kSkip = 0x7FF00000u;
constexpr long long kMaxPitch = 1 << 22;
constexpr int kMaxRows = 0x7FFFF000;     // of x and w: tiles are counted in 32 bits

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, unsigned bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

// 1 KiB from global memory to LDS without passing through registers: lane l's
// 16 bytes land at `lds` + 16 l.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t r, u32x4 *lds, unsigned offset)
{
    typedef __attribute__((address_space(3))) void *lds_ptr;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, offset, 0, 0, 0);
}

// Consecutive logical ids on one XCD (the dispatcher deals workgroups over 8).
__device__ __forceinline__ unsigned logical_id()
{
    const unsigned xcd = blockIdx.x & 7u, turn = blockIdx.x >> 3, q = gridDim.x >> 3, r = gridDim.x & 7u;
    return xcd * q + (xcd < r ? xcd : r) + turn;
}

// 16 RT weight rows by 16 MT tokens a workgroup, its eight waves taking every
// eighth unit of two K steps: each holds all sums of the tile, which are added
// at the end through LDS.  Loads go into registers, D units ahead.  x is read
// in whole lines, eight rows of 128 bytes a load, and passes through the wave's
// own LDS on its way into operands: gathered by the operands' lanes, 64 bytes
// of 16 rows a load, 64 x 7168 x 18432 took 53 against 36 us.  What bounds it is
// a workgroup's 16 K (RT + MT) bytes of loads: x alone takes 17 us there and w
// alone 22, so the two add (132 MB of w at 3.6 TB/s; 45 MB at 4.8 TB/s for one
// token of 6288 x 7168).  They come at some 21 bytes a cycle and CU; whether that
// is the rate of its path or the wait for the units under way has not been told
// apart.  NT: the weight passes by once (a single token tile) and need not stay
// in the caches.
template <int RT, int MT, int D, bool NT>
__global__ __launch_bounds__(512) void product_rows(PArgs a)
{
    constexpr int kWaves = 8, kV = RT * MT;
    constexpr int kUnit = 128 * MT;             // 16-byte vectors of a wave's x in LDS
    __shared__ u32x4 shared[kWaves * kUnit > 256 * kV ? kWaves * kUnit : 256 * kV];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4;
    const unsigned id = logical_id();
    const int mt = (int)(id % (unsigned)a.m_tiles), block = (int)(id / (unsigned)a.m_tiles);
    const int n0 = block * 16 * RT, m0 = mt * 16 * MT;
    const int row_tiles = min(RT, (a.N - n0 + 15) / 16), rows = min(16 * MT, a.M - m0);
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (long long)block * RT * a.pitch * 64,
                                                (unsigned)(row_tiles * a.pitch) * 1024u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + m0 * a.ldx, (unsigned)((rows - 1) * a.ldx) + (unsigned)a.K);
    const int units = a.pitch / 2;
    unsigned w_off[RT], x_off[2 * MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        w_off[r] = (unsigned)(r * a.pitch) * 1024u + 16u * lane;
#pragma unroll
    for (int t = 0; t < 2 * MT; ++t) {
        const int row = 8 * t + (lane >> 3);
        x_off[t] = row < rows ? (unsigned)(row * a.ldx) + 16u * (lane & 7) : kSkip;
    }
    i32x4 acc[RT][MT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            acc[r][t] = i32x4{0, 0, 0, 0};
    u32x4 wf[D][2][RT], xf[D][2 * MT];
    // past K: w is zero up to the end of its last unit, so that x may be anything there (the next row)
    const auto load = [&](int d, int u) {
        const unsigned wo = u < units ? (unsigned)u * 2048u : kSkip, xo = u < units ? (unsigned)u * (2 * kStep) : kSkip;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wf[d][k][r] = __builtin_amdgcn_raw_buffer_load_b128(wr, w_off[r] + wo + 1024u * k, 0, NT ? 2 : 0);
#pragma unroll
        for (int t = 0; t < 2 * MT; ++t)
            xf[d][t] = __builtin_amdgcn_raw_buffer_load_b128(xr, x_off[t] + xo, 0, 0);
    };
    // 16-byte chunk c of row r lies at c ^ (r % 8): written a row at a time and
    // read a column at a time without bank conflicts
    u32x4 *put = shared + wave * kUnit + (lane & ~7) + ((lane & 7) ^ (lane >> 3));
    const u32x4 *take = shared + wave * kUnit + 8 * (lane & 15);
#pragma unroll
    for (int d = 0; d < D; ++d)
        load(d, wave + kWaves * d);
    for (int u = wave; u < units; u += kWaves * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int t = 0; t < 2 * MT; ++t)
                put[64 * t] = xf[d][t];
            __builtin_amdgcn_wave_barrier();
            u32x4 x[2][MT];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    x[k][t] = take[128 * t + ((4 * k + g) ^ (lane & 7))];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[r][t] = mma64(wf[d][k][r], x[k][t], acc[r][t]);
            load(d, u + kWaves * (d + D));
        }
    }
    // waves 4..7 to LDS, 0..3 add theirs, all add the four
    i32x4(*part)[kV][64] = reinterpret_cast<i32x4(*)[kV][64]>(shared);
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
        const i32x4 sum = (part[0][v][lane] + part[1][v][lane]) + (part[2][v][lane] + part[3][v][lane]);
        const int m = m0 + 16 * (v % MT) + (lane & 15), n = n0 + 16 * (v / MT) + 4 * g;
        if (m < a.M && n < a.N)
            store4(a, m, n, sum, a.x_scale[m], channel_scales(a, n));
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

template <int T0>
struct TilesLayout {
    static constexpr int kXCopies = (T0 + 1) / 2;       // a wave's copies of x a stage
    static constexpr int kVecs = (32 + 8 * kXCopies) * 64;
    static constexpr int kStages = T0 == 1 ? 4 : T0 <= 4 ? 3 : 2;
    static constexpr int kBytes = kStages * kVecs * 16;
};

// Many tokens: 256 weight rows by 32 T0 tokens a workgroup of eight waves, each
// a quarter of the rows by half of the tokens, 4 x T0 products a K step.  Both
// operands are copied to LDS, two K steps a stage and up to three stages ahead
// -- w lies in MFMA order, x goes by lines, its 16-byte chunks in an order
// without bank conflicts -- and read into registers one step ahead of the
// products.  Bound by the matrix units and LDS side by side: 28 products of 16
// cycles against 11 reads of 1 KiB a wave and step (T0 = 7).  Reads ahead, and
// spread over the products, made 4000 x 6288 x 7168 193 -> 165 to 169 us (2130 TOP/s;
// the library's product alone, without scales, 178 us); a third stage at T0 = 3
// made 800 x 6288 x 7168 65 -> 51 us.
template <int T0>
__global__ __launch_bounds__(512, 2) void product_tiles(PArgs a)
{
    using L = TilesLayout<T0>;
    constexpr int kStages = L::kStages, kCopies = 4 + L::kXCopies;
    extern __shared__ u32x4 ring[];             // [kStages]: w [2 steps][16][64], x [8 kXCopies times 8 rows][64]
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
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (long long)nt * 16 * a.pitch * 64,
                                                (unsigned)(row_tiles * a.pitch) * 1024u);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + m0 * a.ldx, (unsigned)((rows - 1) * a.ldx) + (unsigned)a.K);
    // this wave's copies of a stage: row tiles 2 wave, 2 wave + 1 of w at both
    // steps, and every eighth 8 rows of x, 16-byte chunk c of row r at c ^ (r % 8)
    unsigned w_off[2], x_off[L::kXCopies];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w_off[j] = (unsigned)((2 * wave + j) * a.pitch) * 1024u + 16u * lane;
#pragma unroll
    for (int j = 0; j < L::kXCopies; ++j) {
        const int row = 8 * (wave + 8 * j) + (lane >> 3);
        x_off[j] = row < rows ? (unsigned)(row * a.ldx) + 16u * ((lane & 7) ^ (lane >> 3)) : kSkip;
    }
    const int stages = a.pitch / 2;
    // the same count of copies for every stage, past the last one too: the waits below count them
    const auto copy = [&](int st, int buf) __attribute__((always_inline)) {
        u32x4 *base = ring + buf * L::kVecs;
        const unsigned wo = st < stages ? (unsigned)st * 2048u : kSkip;
        const unsigned xo = st < stages ? (unsigned)st * (2 * kStep) : kSkip;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            copy_to_lds(wr, base + ((j & 1) * 16 + 2 * wave + (j >> 1)) * 64, w_off[j >> 1] + wo + (j & 1) * 1024u);
#pragma unroll
        for (int j = 0; j < L::kXCopies; ++j)
            copy_to_lds(xr, base + (32 + wave + 8 * j) * 64, x_off[j] + xo);
    };
    i32x4 acc[4][T0];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < T0; ++t)
            acc[i][t] = i32x4{0, 0, 0, 0};
    u32x4 wf[2][4], xf[2][T0];
    // operands of step k of a stage, in registers one step ahead of their products
    const auto read = [&](int buf, int k) __attribute__((always_inline)) {
        const u32x4 *base = ring + buf * L::kVecs;
        const u32x4 *at = base + k * 16 * 64 + lane;
        const u32x4 *xat = base + (32 + 2 * T0 * half) * 64 + 8 * (lane & 15) + ((4 * k + g) ^ (lane & 7));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            wf[k][i] = at[(4 * quarter + i) * 64];
#pragma unroll
        for (int t = 0; t < T0; ++t)
            xf[k][t] = xat[2 * t * 64];
    };
    const auto products = [&](int k) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < T0; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i][t] = mma64(wf[k][i], xf[k][t], acc[i][t]);
        // a read after every second product: all at the start, the waves of a SIMD wait for LDS together
#pragma unroll
        for (int r = 0; r < 4 + T0; ++r) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);      // products
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 4 * T0, 0);
    };
#pragma unroll
    for (int st = 0; st < kStages; ++st)
        copy(st, st);
    landed<(kStages - 1) * kCopies, 15>();
    read(0, 0);
    for (int st = 0, buf = 0; st < stages; ++st) {
        const int next = buf + 1 < kStages ? buf + 1 : 0;
        read(buf, 1);
        products(0);
        __builtin_amdgcn_sched_barrier(0);
        // this wave's copies of the next stage have landed, and it has read all of this one
        landed<(kStages - 2) * kCopies, 0>();
        copy(st + kStages, buf);
        read(next, 0);                          // after the last stage: what lies in LDS, and is not used
        products(1);
        __builtin_amdgcn_sched_barrier(0);
        buf = next;
    }
    __builtin_amdgcn_s_waitcnt(wait_for(0, 15));        // no copy outlives its workgroup's LDS
    f32x4 ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ws[i] = channel_scales(a, n0 + 64 * quarter + 16 * i + 4 * g);
#pragma unroll
    for (int t = 0; t < T0; ++t) {
        const int m = m0 + 16 * (T0 * half + t) + (lane & 15);
        if (m >= a.M)
            continue;
        const float xs = a.x_scale[m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 64 * quarter + 16 * i + 4 * g;
            if (n < a.N)
                store4(a, m, n, acc[i][t], xs, ws[i]);
        }
    }
}


// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

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

skinny_status hip_bad(hipError_t e, const char *what)
{
    return bad(e == hipErrorOutOfMemory ? SKINNY_ERR_NOMEM : SKINNY_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool is_type(int t) { return t == SKINNY_TYPE_BF16 || t == SKINNY_TYPE_F32 || t == SKINNY_TYPE_F16; }
int type_bytes(int t) { return t == SKINNY_TYPE_F32 ? 4 : 2; }

// One workgroup a row, in several launches where their threads pass 2^32 - 1, the most that one may have.
hipError_t launch_rows(const void *fn, QArgs a, int M, int type_bytes, unsigned threads, hipStream_t stream)
{
    void *params[] = {&a};
    const int most = (int)(0xFFFFFFFFu / threads);
    for (int left = M; left > 0; left -= most) {
        const int rows = left < most ? left : most;
        const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)rows), dim3(threads), params, 0, stream);
        if (e != hipSuccess)
            return e;
        a.x = static_cast<const char *>(a.x) + rows * a.ldx * type_bytes;
        a.q += rows * a.ldq;
        a.scale += rows;
    }
    return hipSuccess;
}

template <int TYPE>
hipError_t launch_quantize(const QArgs &a, int M, hipStream_t stream)
{
    constexpr int kVec = Elem<TYPE>::kVec, kBytes = sizeof(typename Elem<TYPE>::raw);
    const bool vec = a.K % kVec == 0 && (uintptr_t)a.x % 16 == 0 && a.ldx % kVec == 0 &&
                     (uintptr_t)a.q % kVec == 0 && a.ldq % kVec == 0;
    if (!vec)
        return launch_rows(reinterpret_cast<const void *>(quantize_element<TYPE>), a, M, kBytes, 256, stream);
    const int vecs = a.K / kVec;
    // four vectors a thread, 64 to 1024 threads
    int threads = 64;
    while (threads < 1024 && threads * 4 < vecs)
        threads *= 2;
    const int per = (vecs + threads - 1) / threads;
    const void *fn = per <= 1   ? reinterpret_cast<const void *>(quantize_vector<TYPE, 1>)
                     : per <= 2 ? reinterpret_cast<const void *>(quantize_vector<TYPE, 2>)
                     : per <= 4 ? reinterpret_cast<const void *>(quantize_vector<TYPE, 4>)
                     : per <= 5 ? reinterpret_cast<const void *>(quantize_vector<TYPE, 5>)
                                : reinterpret_cast<const void *>(quantize_vector<TYPE, 0>);
    return launch_rows(fn, a, M, kBytes, (unsigned)threads, stream);
}

// Two units ahead where there are few registers to fill (one row tile, one
// token tile) and where the long tile's products hide them (4 x 4); one
// elsewhere, which measured faster (3584 x 7168, 48 tokens: 11.8 against 12.9 us).
template <int RT, int MT, bool NT>
const void *rows_fn()
{
    return reinterpret_cast<const void *>(product_rows<RT, MT, RT == MT && RT != 2 ? 2 : 1, NT>);
}

template <int RT, bool NT>
const void *rows_kernel_of(int mt)
{
    return mt == 1 ? rows_fn<RT, 1, NT>() : mt == 2 ? rows_fn<RT, 2, NT>() : mt == 3 ? rows_fn<RT, 3, NT>()
                                                                           : rows_fn<RT, 4, NT>();
}

template <bool NT>
const void *rows_kernel(int rt, int mt)
{
    return rt == 1 ? rows_kernel_of<1, NT>(mt) : rt == 2 ? rows_kernel_of<2, NT>(mt) : rows_kernel_of<4, NT>(mt);
}

template <int T0>
const void *tiles_fn()
{
    return reinterpret_cast<const void *>(product_tiles<T0>);
}

const void *tiles_kernel(int t0)
{
    return t0 == 1 ? tiles_fn<1>() : t0 == 2 ? tiles_fn<2>() : t0 == 3 ? tiles_fn<3>() : t0 == 4 ? tiles_fn<4>()
         : t0 == 5 ? tiles_fn<5>() : t0 == 6 ? tiles_fn<6>() : t0 == 7 ? tiles_fn<7>() : tiles_fn<8>();
}

int tiles_lds(int t0)
{
    return t0 == 1 ? TilesLayout<1>::kBytes : t0 == 2 ? TilesLayout<2>::kBytes : t0 == 3 ? TilesLayout<3>::kBytes
         : t0 == 4 ? TilesLayout<4>::kBytes : t0 == 5 ? TilesLayout<5>::kBytes : t0 == 6 ? TilesLayout<6>::kBytes
         : t0 == 7 ? TilesLayout<7>::kBytes : TilesLayout<8>::kBytes;
}

// A tile shape and the time of its rounds over 256 CUs, in us over K = 7168.
// Other K change both kernels' alike, but for starts and ends: over 512 to 6288
// rows and 72 to 3200 tokens the kernel taken was within a geometric mean of 3.0,
// 1.8, 1.1 and 0.7 % of the better one at K = 512, 1536, 7168 and 18432 (at
// worst 1.2 to 1.7 times it, 3200 tokens of 512 rows).
struct Tiling {
    int r, t;                   // 16 r rows by 16 t tokens, or 256 rows by 32 t tokens
    float us;
};

// product_rows: a round is as long as the bytes a workgroup loads, 2.25 us
// (r + t).  Of equal ones the most tokens, which read the weight least often
// (3584 x 7168, 128 tokens: 2 x 4 14.8, 4 x 2 15.7, 4 x 4 and 2 x 2 17 us or more).
Tiling rows_tiling(int M, int N)
{
    Tiling best{0, 0, 0.0f};
    for (int t = min(4, (M + 15) / 16); t >= 1; --t)
        for (int r = 1; r <= 4; r *= 2) {
            const long long count = (long long)((N + 16 * r - 1) / (16 * r)) * ((M + 16 * t - 1) / (16 * t));
            const float us = (float)((count + 255) / 256) * 2.25f * (float)(r + t);
            if (!best.r || us < best.us)
                best = Tiling{r, t, us};
        }
    return best;
}

// product_tiles: a round measured at 6288 rows and 200 to 4000 tokens; three
// stages fit LDS up to t = 4, two above.
Tiling tiles_tiling(int M, int N)
{
    static const float round_us[9] = {0.0f, 36.0f, 41.0f, 47.0f, 51.0f, 73.0f, 76.0f, 83.0f, 89.0f};
    Tiling best{0, 0, 0.0f};
    for (int t = 8; t >= 1; --t) {
        const long long count = ((long long)N + 255) / 256 * ((M + 32 * t - 1) / (32 * t));
        const float us = (float)((count + 255) / 256) * round_us[t];
        if (!best.r || us < best.us)
            best = Tiling{16, t, us};
    }
    return best;
}

// Up to 64 tokens the rows kernel, which reads the weight once for every token
// tile (one to four).  Above, the shorter of both: 400 tokens of 6288 x 7168 54 against 42 us, of 3584 x 7168 26
// against 36 us, 800 of 1500 x 7168 25 against 29 us.
hipError_t launch_product(PArgs a, hipStream_t stream)
{
    constexpr unsigned kThreads = 512;
    constexpr int kSplit = 256;                 // rows and tokens of the largest tile: both halves begin on one
    void *params[] = {&a};
    const Tiling rows = rows_tiling(a.M, a.N);
    const Tiling tiles = a.M > 64 ? tiles_tiling(a.M, a.N) : rows;
    const bool many = tiles.us < rows.us;
    const int n_rows = many ? 256 : 16 * rows.r, tokens = many ? 32 * tiles.t : 16 * rows.t;
    const long long n_tiles = ((long long)a.N + n_rows - 1) / n_rows, m_tiles = ((long long)a.M + tokens - 1) / tokens;
    if (n_tiles * m_tiles > 0xFFFFFFFFu / kThreads) {
        // more threads than a launch may have: the two halves of the longer side, one after the other
        const int bytes = type_bytes(a.type);
        PArgs second = a;
        if (a.M >= a.N) {
            const int first = a.M / 2 / kSplit * kSplit;
            second.M = a.M - first;
            second.x += first * a.ldx;
            second.x_scale += first;
            second.out = static_cast<char *>(a.out) + first * a.ldo * bytes;
            if (a.res)
                second.res = static_cast<const char *>(a.res) + first * a.ldr * bytes;
            a.M = first;
        } else {
            const int first = a.N / 2 / kSplit * kSplit;
            second.N = a.N - first;
            second.w += (long long)(first / 16) * a.pitch * 64;
            second.w_scale += first;
            second.out = static_cast<char *>(a.out) + (long long)first * bytes;
            if (a.res)
                second.res = static_cast<const char *>(a.res) + (long long)first * bytes;
            a.N = first;
        }
        const hipError_t e = launch_product(a, stream);
        return e == hipSuccess ? launch_product(second, stream) : e;
    }
    a.n_tiles = (int)n_tiles;
    a.m_tiles = (int)m_tiles;
    const void *fn = many                ? tiles_kernel(tiles.t)
                     : a.m_tiles == 1 ? rows_kernel<true>(rows.r, rows.t)
                                      : rows_kernel<false>(rows.r, rows.t);
    return hipLaunchKernel(fn, dim3((unsigned)(n_tiles * m_tiles)), dim3(kThreads), params,
                           many ? (size_t)tiles_lds(tiles.t) : 0, stream);
}

// Dynamic LDS past 64 KiB has to be asked for, on every device that the kernels run on.
void raise_limits()
{
    for (int t0 = 1; t0 <= 8; ++t0)
        (void)hipFuncSetAttribute(tiles_kernel(t0),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, tiles_lds(t0));
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

skinny_status skinny_quantize_rows(const void *x, skinny_type type, int M, int K, long long ldx, void *q,
                                   long long ldq, float *scale, void *stream)
{
    if (!is_type((int)type))
        return bad(SKINNY_ERR_INVALID_ARG, "type %d is none of BF16, F32 and F16", (int)type);
    if (M < 0 || K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d and K=%d: M >= 0 and K >= 1 are needed", M, K);
    if (M == 0)
        return SKINNY_OK;
    if (!x || !q || !scale)
        return bad(SKINNY_ERR_INVALID_ARG, "x, q or scale is NULL");
    if (ldx < K || ldq < K)
        return bad(SKINNY_ERR_SHAPE, "ldx=%lld and ldq=%lld must be at least K=%d", ldx, ldq, K);
    if ((uintptr_t)x % type_bytes((int)type) || (uintptr_t)scale % 4)
        return bad(SKINNY_ERR_ALIGN, "x and scale must be aligned to their elements");
    const QArgs a{x, static_cast<signed char *>(q), scale, ldx, ldq, K};
    const hipStream_t s = (hipStream_t)stream;
    const hipError_t e = type == SKINNY_TYPE_F32   ? launch_quantize<SKINNY_TYPE_F32>(a, M, s)
                         : type == SKINNY_TYPE_F16 ? launch_quantize<SKINNY_TYPE_F16>(a, M, s)
                                                   : launch_quantize<SKINNY_TYPE_BF16>(a, M, s);
    return e == hipSuccess ? SKINNY_OK : hip_bad(e, "quantize launch");
}

skinny_status skinny_int8_prepare(const void *Wq, int N, int K, long long ldw, const float *w_scale,
                                  skinny_type out_type, void *stream, skinny_int8_plan **plan)
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
    if (K % 16 || K >= 131072)
        return bad(SKINNY_ERR_SHAPE, "K=%d must be a multiple of 16 below 131072", K);
    if (ldw < K)
        return bad(SKINNY_ERR_SHAPE, "ldw=%lld is less than K=%d", ldw, K);
    if ((uintptr_t)w_scale % 4)
        return bad(SKINNY_ERR_ALIGN, "w_scale must be 4-byte aligned");
    const int steps = (K + kStep - 1) / kStep, pitch = (steps + 1) / 2 * 2;
    const long long tiles = ((long long)N + 15) / 16, count = tiles * pitch * 64;
    if (count >= 1LL << 36)
        return bad(SKINNY_ERR_SHAPE, "N=%d by K=%d is too large", N, K);
    skinny_int8_plan *p = new (std::nothrow) skinny_int8_plan{N, K, pitch, out_type, 0, nullptr, nullptr};
    if (!p)
        return bad(SKINNY_ERR_NOMEM, "host allocation failed");
    int cus = 0;
    const skinny_status st = current_gfx950(&p->device, &cus);
    if (st != SKINNY_OK) {
        delete p;
        return st;
    }
    raise_limits();
    hipError_t e = hipMalloc(&p->w, (size_t)count * 16);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&p->w_scale), (size_t)N * sizeof(float));
    const hipStream_t s = (hipStream_t)stream;
    if (e == hipSuccess)
        e = hipMemcpyAsync(p->w_scale, w_scale, (size_t)N * sizeof(float), hipMemcpyDeviceToDevice, s);
    const signed char *src = static_cast<const signed char *>(Wq);
    u32x4 *dst = static_cast<u32x4 *>(p->w);
    constexpr long long kMost = 1LL << 31;      // vectors a launch: it may not have 2^32 threads
    for (long long first = 0; e == hipSuccess && first < count; first += kMost) {
        int n = N, k = K, ks = pitch;
        long long ld = ldw, c = count, f = first, left = count - first < kMost ? count - first : kMost;
        void *params[] = {&src, &ld, &n, &k, &ks, &dst, &f, &c};
        e = hipLaunchKernel(reinterpret_cast<const void *>(lay_out), dim3((unsigned)((left + 255) / 256)), dim3(256),
                            params, 0, s);
    }
    if (e == hipSuccess)
        e = hipStreamSynchronize(s);
    if (e != hipSuccess) {
        (void)hipFree(p->w);
        (void)hipFree(p->w_scale);
        delete p;
        return hip_bad(e, "int8 prepare");
    }
    *plan = p;
    return SKINNY_OK;
}

skinny_status skinny_int8_run(const skinny_int8_plan *p, const void *xq, long long ldx, const float *x_scale,
                              const void *residual, long long ldr, void *out, long long ldo, int M, void *stream)
{
    if (!p)
        return bad(SKINNY_ERR_INVALID_ARG, "plan is NULL");
    if (M < 0)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d is negative", M);
    if (M > kMaxRows)
        return bad(SKINNY_ERR_SHAPE, "M=%d: at most %d", M, kMaxRows);
    if (M == 0)
        return SKINNY_OK;
    if (!xq || !x_scale || !out)
        return bad(SKINNY_ERR_INVALID_ARG, "xq, x_scale or out is NULL");
    if (ldx < p->K || ldx % 16 || ldx >= kMaxPitch || ldo < p->N || (residual && ldr < p->N))
        return bad(SKINNY_ERR_SHAPE, "ldx=%lld must be a multiple of 16, at least K=%d and below 2^22, ldo=%lld and "
                   "ldr=%lld at least N=%d", ldx, p->K, ldo, ldr, p->N);
    const int eb = type_bytes((int)p->out);
    if ((uintptr_t)xq % 16 || (uintptr_t)x_scale % 4 || (uintptr_t)out % eb || (uintptr_t)residual % eb)
        return bad(SKINNY_ERR_ALIGN, "xq must be 16-byte aligned, x_scale, out and residual to their elements");
    PArgs a{};
    a.w = static_cast<const u32x4 *>(p->w);
    a.x = static_cast<const signed char *>(xq);
    a.x_scale = x_scale;
    a.w_scale = p->w_scale;
    a.res = residual;
    a.out = out;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldo = ldo;
    a.M = M;
    a.N = p->N;
    a.K = p->K;
    a.pitch = p->pitch;
    a.type = p->out;
    a.vec = (uintptr_t)out % (4 * eb) == 0 && ldo % 4 == 0 && (uintptr_t)residual % (4 * eb) == 0 && ldr % 4 == 0;
    const hipError_t e = launch_product(a, (hipStream_t)stream);
    return e == hipSuccess ? SKINNY_OK : hip_bad(e, "int8 product launch");
}

void skinny_int8_destroy(skinny_int8_plan *p)
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
