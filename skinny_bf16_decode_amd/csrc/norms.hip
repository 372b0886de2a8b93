// HIP kernels and entry points of what stands between two blocks of a decode
// layer, for gfx950 (CDNA4):
//
//   n = x r weight,  r = 1 / sqrt(mean x^2 + eps)
//   h = beta residual + alpha gate z,  z = norm(y) or y,  and the norm of h
//
// A norm is written in 16 or 32 bits, as 8-bit integers with a scale for each
// row, or as blocks of 4 or 8 bits, straight from fp32.  Squares are summed in
// 64 bits: whatever the order of the sum, r is then the same fp32 number (but
// for sums within 1e-15 of a border), and so is every rounding that follows.  A
// last place of r would carry a 4-bit value to the next one.
#include <hip/hip_runtime.h>

#include "norm_shape.h"
#include "operators.h"
#include "rows.h"
#include "skinny_internal.h"

// Products and sums round one by one, in the formulas' order.
#pragma clang fp contract(off)

namespace skinny {
namespace {

// What is written of a norm.
struct NormOut {
    const void *weight;
    void *out;                  // or NULL
    unsigned char *q;
    void *scale;                // float [M], or bytes [M][lds]
    long long ldo, ldq, lds;
    double eps, inverse_K;
    int weight_type, out_type, q_kind;
};

struct NArgs {
    const void *x;
    long long ldx;
    NormOut n;
    int type, M, K;
    int lanes;                  // threads of a row: a power of two, 16 to 1024
};

struct JArgs {
    const void *residual, *y, *weight, *gate;
    void *out;
    long long ldr, ldy, ldg, ldo;
    NormOut n;                  // n.weight NULL: no norm of the result
    double eps, inverse_K;
    float alpha, beta;
    int residual_type, y_type, weight_type, gate_type, sigmoid;
    int M, K;
    int lanes;
};

// This thread's row: `lanes` threads of the workgroup have one.
struct Place {
    int row, t, waves, first_wave;
    bool in;
};

__device__ __forceinline__ Place place_of(int lanes, int M)
{
    Place p;
    const int tid = (int)threadIdx.x, rows = (int)blockDim.x / lanes;
    const long long row = (long long)blockIdx.x * rows + tid / lanes;
    p.in = row < M;
    p.row = p.in ? (int)row : M - 1;            // rows past the last take part in the barriers and write nothing
    p.t = tid % lanes;
    p.waves = lanes / 64;
    p.first_wave = tid / lanes * p.waves;
    return p;
}

// v of the lane that a DPP control names.
template <int CTRL>
__device__ __forceinline__ unsigned lane_of(unsigned v)
{
    return (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double lane_of(double v)
{
    const unsigned long long u = __double_as_longlong(v);
    return __longlong_as_double((unsigned long long)lane_of<CTRL>((unsigned)(u >> 32)) << 32 | lane_of<CTRL>((unsigned)u));
}

// Both halves' v: of the lanes whose number's bit 4 (5) is 0, and is 1.
template <int BIT>
__device__ __forceinline__ void halves(unsigned v, unsigned &a, unsigned &b)
{
    typedef __attribute__((ext_vector_type(2))) unsigned int pair;
    const pair r = BIT == 4 ? __builtin_bit_cast(pair, __builtin_amdgcn_permlane16_swap(v, v, false, false))
                            : __builtin_bit_cast(pair, __builtin_amdgcn_permlane32_swap(v, v, false, false));
    a = r[0];
    b = r[1];
}
template <int BIT>
__device__ __forceinline__ void halves(double v, double &a, double &b)
{
    const unsigned long long u = __double_as_longlong(v);
    unsigned al, bl, ah, bh;
    halves<BIT>((unsigned)u, al, bl);
    halves<BIT>((unsigned)(u >> 32), ah, bh);
    a = __longlong_as_double((unsigned long long)ah << 32 | al);
    b = __longlong_as_double((unsigned long long)bh << 32 | bl);
}

__device__ __forceinline__ double both(double a, double b) { return a + b; }
__device__ __forceinline__ unsigned both(unsigned a, unsigned b) { return a > b ? a : b; }

// The sum (double) or maximum (unsigned) of a row's threads' v, in every one of
// them: within 16 lanes by quad permutes and mirrors, then by halves of 32 and
// 64, then over the row's waves through `shared`, which serves one call.
template <typename T>
__device__ __forceinline__ T over_row(T v, int lanes, const Place &p, T *shared)
{
    v = both(v, lane_of<0xB1>(v));              // lane ^ 1
    v = both(v, lane_of<0x4E>(v));              // lane ^ 2
    v = both(v, lane_of<0x141>(v));             // the other four of eight
    v = both(v, lane_of<0x140>(v));             // the other eight of 16
    if (lanes >= 32) {
        T a, b;
        halves<4>(v, a, b);
        v = both(a, b);
    }
    if (lanes >= 64) {
        T a, b;
        halves<5>(v, a, b);
        v = both(a, b);
    }
    if (lanes > 64) {
        if ((threadIdx.x & 63) == 0)
            shared[threadIdx.x >> 6] = v;
        __syncthreads();
        v = shared[p.first_wave];
        for (int w = 1; w < p.waves; ++w)
            v = both(v, shared[p.first_wave + w]);
    }
    return v;
}

__device__ __forceinline__ double squares(const float (&f)[8])
{
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double d = (double)f[e];
        s = fma(d, d, s);
    }
    return s;
}

// 1 / sqrt(sum / K + eps): the unit's reciprocal root (some 2^-26) and two steps
// of Newton's, which leave 64 bits' rounding errors.  Past the normal range of
// what they square, infinity and NaN among it, the unit's own result.
__device__ __forceinline__ float rms_factor(double sum, double inverse_K, double eps)
{
    const double v = fma(sum, inverse_K, eps);
    const double y0 = __builtin_amdgcn_rsq(v);
    const double h = 0.5 * v;
    const double y1 = fma(y0, fma(-h * y0, y0, 0.5), y0);
    const double y2 = fma(y1, fma(-h * y1, y1, 0.5), y1);
    return (float)(v < 0x1p1000 ? y2 : y0);
}

__device__ __forceinline__ const char *at_row(const void *p, long long row, long long ld, int type)
{
    return static_cast<const char *>(p) + row * ld * (type == SKINNY_TYPE_F32 ? 4 : 2);
}

// Element e of turn i.
template <Mode MODE>
__device__ __forceinline__ unsigned index_of(int i, int e, int lanes, const Place &p)
{
    // below K + 8 * 1024
    return MODE == kStrided ? (8u * i + e) * (unsigned)lanes + p.t : 8u * (p.t + (unsigned)i * lanes) + e;
}

// This thread's eight elements of turn i, zero past the row.
template <Mode MODE>
__device__ __forceinline__ Octet own_octet(const void *row, int type, int i, int K, int lanes, const Place &p)
{
    Octet v;
    v.a = v.b = u32x4{0u, 0u, 0u, 0u};
    if constexpr (MODE == kStrided) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned k = index_of<MODE>(i, e, lanes, p);
            unsigned u = 0u;
            if (k < (unsigned)K)
                u = type == SKINNY_TYPE_F32 ? static_cast<const unsigned *>(row)[k]
                                            : static_cast<const unsigned short *>(row)[k];
            if (type != SKINNY_TYPE_F32)
                v.a[e / 2] |= u << (16 * (e & 1));
            else if (e < 4)
                v.a[e] = u;
            else
                v.b[e - 4] = u;
        }
    } else {
        const int o = p.t + i * lanes;
        if (o < octets_of(K))
            v = load_octet<MODE == kVectors>(row, type, o, K);
    }
    return v;
}

template <Mode MODE>
__device__ __forceinline__ void put_octet(void *row, int type, int i, int K, int lanes, const Place &p, const Octet &v)
{
    if constexpr (MODE == kStrided) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned k = index_of<MODE>(i, e, lanes, p);
            if (k >= (unsigned)K)
                continue;
            if (type == SKINNY_TYPE_F32)
                static_cast<unsigned *>(row)[k] = e < 4 ? v.a[e & 3] : v.b[e & 3];
            else
                static_cast<unsigned short *>(row)[k] = (unsigned short)(v.a[e / 2] >> (16 * (e & 1)));
        }
    } else {
        const int o = p.t + i * lanes;
        if (o < octets_of(K))
            store_octet<MODE == kVectors>(row, type, o, K, v);
    }
}

// What is written of a thread's eight elements f of turn i of a norm.
template <Mode MODE>
__device__ __forceinline__ void write_octet(const NormOut &n, int i, int K, int lanes, const Place &p,
                                            const RowScale &scale8, float (&f)[8])
{
    if (n.q_kind == SKINNY_ROWS_MX4 || n.q_kind == SKINNY_ROWS_MX8) {
        if constexpr (MODE != kStrided) {       // whole blocks are asked for
            const int o = p.t + i * lanes;
            const bool here = p.in && o < K / 8;
            unsigned byte;
            unsigned char *q = n.q + p.row * n.ldq;
            if (n.q_kind == SKINNY_ROWS_MX4) {
                const u32x2 codes = block_codes<4>(f, byte);
                if (here)
                    store_codes<MODE == kVectors, 4>(q, o, codes);
            } else {
                const u32x2 codes = block_codes<8>(f, byte);
                if (here)
                    store_codes<MODE == kVectors, 8>(q, o, codes);
            }
            if (here && (o & 3) == 0)
                static_cast<unsigned char *>(n.scale)[p.row * n.lds + (o >> 2)] = (unsigned char)byte;
        }
    } else if (n.q_kind == SKINNY_ROWS_INT8 && p.in) {
        unsigned char *q = n.q + p.row * n.ldq;
        if constexpr (MODE == kVectors) {
            const int o = p.t + i * lanes;
            u32x2 codes;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                codes[e / 4] = (unsigned)(to_int8(f[e], scale8) & 0xFF) | (unsigned)(to_int8(f[e + 1], scale8) & 0xFF) << 8 |
                               (unsigned)(to_int8(f[e + 2], scale8) & 0xFF) << 16 |
                               (unsigned)to_int8(f[e + 3], scale8) << 24;
            if (o < K / 8)
                store_codes<true, 8>(q, o, codes);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned k = index_of<MODE>(i, e, lanes, p);
                if (k < (unsigned)K)
                    q[k] = (unsigned char)to_int8(f[e], scale8);
            }
        }
    }
    if (n.out && p.in) {
        const Octet y = pack_octet(n.out_type, f);
        put_octet<MODE>(const_cast<char *>(at_row(n.out, p.row, n.ldo, n.out_type)), n.out_type, i, K, lanes, p, y);
    }
}

// The norm of a row whose octets get(i, f) gives, i = 0, 1, ... for the octets
// t + i lanes of this thread; f is zero past the row.  OCTETS: how many at most,
// 0: any.  `first` is the weight's octet 0; the others are loaded one ahead.
template <Mode MODE, int OCTETS, typename Get>
__device__ __forceinline__ void write_norm(const NormOut &n, double sum, int K, int lanes, const Place &p,
                                           unsigned *tops, const Octet &first, Get get)
{
    const int octets = octets_of(K), turns = OCTETS ? OCTETS : (octets + lanes - 1) / lanes;
    const float r = rms_factor(sum, n.inverse_K, n.eps);
    const auto value = [&](int i, const Octet &raw, float (&f)[8]) {
        get(i, f);
        float w[8];
        unpack_octet(raw, n.weight_type, w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = f[e] * r * w[e];
    };
    RowScale scale8;
    scale8.lift = scale8.inverse = 0.0f;
    scale8.fine = false;
    if (n.q_kind == SKINNY_ROWS_INT8) {
        unsigned top = 0;
        Octet w = first;
#pragma unroll OCTETS ? OCTETS : 1
        for (int i = 0; i < turns; ++i) {
            const Octet next = i + 1 < turns ? own_octet<MODE>(n.weight, n.weight_type, i + 1, K, lanes, p) : w;
            float f[8];
            value(i, w, f);
            // past the row f is zero, but where r is NaN, and all of the row with it (eps keeps r below 2^60)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned m = mag(f[e]);
                top = m > top ? m : top;
            }
            w = next;
            __builtin_amdgcn_sched_barrier(0);
        }
        float scale;
        scale8 = row_scale(over_row(top, lanes, p, tops), scale);
        if (p.in && p.t == 0)
            static_cast<float *>(n.scale)[p.row] = scale;
    }
    Octet w = first;
#pragma unroll OCTETS ? OCTETS : 1
    for (int i = 0; i < turns; ++i) {
        const Octet next = i + 1 < turns ? own_octet<MODE>(n.weight, n.weight_type, i + 1, K, lanes, p) : w;
        float f[8];
        value(i, w, f);
        write_octet<MODE>(n, i, K, lanes, p, scale8, f);
        w = next;
        // one after the other, so that the registers of one serve the next
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A row's octets stay in registers between the sum and the norm (OCTETS = 0:
// the row is longer than that, and read again).  A few rows are a launch, a load, a
// reduction and a store, one after the other: 1 x 7168 3.2 us, 64 rows 3.4.
template <int OCTETS, Mode MODE, int type>
__global__ __launch_bounds__(1024) void norm_kernel(NArgs a)
{
    __shared__ double sums[16];
    __shared__ unsigned tops[16];
    const Place p = place_of(a.lanes, a.M);
    const char *x = at_row(a.x, p.row, a.ldx, type);
    const int octets = octets_of(a.K), turns = OCTETS ? OCTETS : (octets + a.lanes - 1) / a.lanes;
    const auto load = [&](int i) { return own_octet<MODE>(x, type, i, a.K, a.lanes, p); };
    Octet keep[OCTETS ? OCTETS : 1];
    double sum = 0.0;
    if constexpr (OCTETS > 0) {
#pragma unroll
        for (int i = 0; i < OCTETS; ++i)
            keep[i] = load(i);
    }
#pragma unroll OCTETS ? OCTETS : 1
    for (int i = 0; i < turns; ++i) {
        float f[8];
        unpack_octet(OCTETS ? keep[OCTETS ? i : 0] : load(i), type, f);
        sum += squares(f);
    }
    const Octet first = own_octet<MODE>(a.n.weight, a.n.weight_type, 0, a.K, a.lanes, p);
    sum = over_row(sum, a.lanes, p, sums);
    write_norm<MODE, OCTETS>(a.n, sum, a.K, a.lanes, p, tops, first, [&](int i, float (&f)[8]) {
        unpack_octet(OCTETS ? keep[OCTETS ? i : 0] : load(i), type, f);
    });
}

// Two norms, one after the other: 8 x 7168 5.2 us; 4000 x 7168 with a gate for each
// token and its sigmoid 65.5 us, 4.4 TB/s.
template <int OCTETS, Mode MODE, int y_type, int residual_type>
__global__ __launch_bounds__(1024) void join_kernel(JArgs a)
{
    __shared__ double sums[32];
    __shared__ unsigned tops[16];
    const Place p = place_of(a.lanes, a.M);
    const char *y = at_row(a.y, p.row, a.ldy, y_type);
    const char *res = at_row(a.residual, p.row, a.ldr, residual_type);
    const char *gate = a.gate ? at_row(a.gate, p.row, a.ldg, a.gate_type) : nullptr;
    char *out = const_cast<char *>(at_row(a.out, p.row, a.ldo, residual_type));
    const int octets = octets_of(a.K), turns = OCTETS ? OCTETS : (octets + a.lanes - 1) / a.lanes;
    const auto load = [&](const void *row, int type, int i) { return own_octet<MODE>(row, type, i, a.K, a.lanes, p); };
    Octet ys[OCTETS ? OCTETS : 1], hs[OCTETS ? OCTETS : 1];
    if constexpr (OCTETS > 0) {
#pragma unroll
        for (int i = 0; i < OCTETS; ++i) {
            ys[i] = load(y, y_type, i);
            hs[i] = load(res, residual_type, i);
        }
    }
    // of the weights and the gate, the first octet now and the others one ahead
    Octet w = Octet{}, g = Octet{}, first = Octet{};
    if (a.weight)
        w = load(a.weight, a.weight_type, 0);
    if (gate)
        g = load(gate, a.gate_type, 0);
    if (a.n.weight)
        first = load(a.n.weight, a.n.weight_type, 0);
    float r = 1.0f;
    if (a.weight) {
        double sum = 0.0;
#pragma unroll OCTETS ? OCTETS : 1
        for (int i = 0; i < turns; ++i) {
            float f[8];
            unpack_octet(OCTETS ? ys[OCTETS ? i : 0] : load(y, y_type, i), y_type, f);
            sum += squares(f);
        }
        r = rms_factor(over_row(sum, a.lanes, p, sums), a.inverse_K, a.eps);
    }
    double sum = 0.0;
#pragma unroll OCTETS ? OCTETS : 1
    for (int i = 0; i < turns; ++i) {
        Octet next_w = w, next_g = g;
        if (i + 1 < turns) {
            if (a.weight)
                next_w = load(a.weight, a.weight_type, i + 1);
            if (gate)
                next_g = load(gate, a.gate_type, i + 1);
        }
        float z[8], h[8], c[8];
        unpack_octet(OCTETS ? ys[OCTETS ? i : 0] : load(y, y_type, i), y_type, z);
        unpack_octet(OCTETS ? hs[OCTETS ? i : 0] : load(res, residual_type, i), residual_type, h);
        if (a.weight) {
            unpack_octet(w, a.weight_type, c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = z[e] * r * c[e];
        }
        if (gate) {
            unpack_octet(g, a.gate_type, c);
            if (a.sigmoid)
                sigmoid(c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] *= c[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[e] = index_of<MODE>(i, e, a.lanes, p) < (unsigned)a.K ? h[e] * a.beta + z[e] * a.alpha : 0.0f;
        // as it is held from here on
        const Octet v = pack_octet(residual_type, h);
        if (OCTETS)
            hs[OCTETS ? i : 0] = v;
        if (p.in)
            put_octet<MODE>(out, residual_type, i, a.K, a.lanes, p, v);
        sum += squares(h);
        w = next_w;
        g = next_g;
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!a.n.weight)
        return;
    sum = over_row(sum, a.lanes, p, sums + 16);
    // without registers: what this thread has written
    write_norm<MODE, OCTETS>(a.n, sum, a.K, a.lanes, p, tops, first, [&](int i, float (&f)[8]) {
        unpack_octet(OCTETS ? hs[OCTETS ? i : 0] : load(out, residual_type, i), residual_type, f);
    });
}

// ---------------------------------------------------------------------------
// Many rows: workgroups go from row to row
// ---------------------------------------------------------------------------
//
// A thread has the same C octets of every row, so that their weights (and a
// channel's gate) stay in its registers: read again for each row, from L2, they
// cost a fifth of the time (4003 x 7168 to BF16: 29.3 against 23.5 us without).  R
// rows go together, the next R are loaded before the reduction of these.  Bound by
// bytes: 4003 x 7168 in BF16 with fp32 weights, to BF16 and 8-bit blocks, 33.8 us, 4.3
// TB/s; 8192 x 2048 in FP16 13.1 us, 5.1 TB/s; 4000 x 7168 joined in BF16 49.9 us, 4.6 TB/s.

// lanes of the lower half: x of both halves, of the upper half: y of both (BIT 4: within each 32 lanes)
template <int BIT>
__device__ __forceinline__ void swap_halves(unsigned &x, unsigned &y)
{
    typedef __attribute__((ext_vector_type(2))) unsigned int pair;
    const pair r = BIT == 4 ? __builtin_bit_cast(pair, __builtin_amdgcn_permlane16_swap(x, y, false, false))
                            : __builtin_bit_cast(pair, __builtin_amdgcn_permlane32_swap(x, y, false, false));
    x = r[0];
    y = r[1];
}
template <int BIT>
__device__ __forceinline__ unsigned joined(unsigned x, unsigned y)
{
    swap_halves<BIT>(x, y);
    return both(x, y);
}
template <int BIT>
__device__ __forceinline__ double joined(double x, double y)
{
    const unsigned long long u = __double_as_longlong(x), v = __double_as_longlong(y);
    unsigned xl = (unsigned)u, yl = (unsigned)v, xh = (unsigned)(u >> 32), yh = (unsigned)(v >> 32);
    swap_halves<BIT>(xl, yl);
    swap_halves<BIT>(xh, yh);
    return both(__longlong_as_double((unsigned long long)xh << 32 | xl),
                __longlong_as_double((unsigned long long)yh << 32 | yl));
}

// The lane that has row j's result of over_rows.
template <int R>
__device__ __forceinline__ constexpr int lane_with(int j)
{
    return R == 4 ? 32 * (j & 1) + 16 * (j >> 1) : 32 * j;
}

// The sums (double) or maxima (unsigned) over the workgroup of R rows' v: in
// lanes lane_with<R>(j) .. + 15 those of row j.  Rows share the steps: two of them
// take half of the lanes each.  `shared` [4][16] serves every second call.
template <int R, typename T>
__device__ __forceinline__ T over_rows(const T (&v)[R], int waves, T (*shared)[16])
{
    T x;
    if constexpr (R == 4)
        x = joined<4>(joined<5>(v[0], v[1]), joined<5>(v[2], v[3]));
    else if constexpr (R == 2)
        x = joined<5>(v[0], v[1]);
    else
        x = joined<5>(v[0], v[0]);
    if constexpr (R < 4)
        x = joined<4>(x, x);
    const auto within16 = [](T y) {
        y = both(y, lane_of<0xB1>(y));
        y = both(y, lane_of<0x4E>(y));
        y = both(y, lane_of<0x141>(y));
        return both(y, lane_of<0x140>(y));
    };
    x = within16(x);
    if (waves > 1) {
        const int lane = threadIdx.x & 63;
        if ((lane & 15) == 0)
            shared[lane >> 4][threadIdx.x >> 6] = x;
        __syncthreads();
        x = within16((lane & 15) < waves ? shared[lane >> 4][lane & 15] : T(0));
    }
    return x;
}

__device__ __forceinline__ float from_lane(float v, int lane)
{
    return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// Octet i of this thread's in a row, zero past its end or without a row.
template <int TYPE>
__device__ __forceinline__ Octet octet_of(const void *base, long long row, long long ld, int type, bool in, int o)
{
    Octet v;
    v.a = v.b = u32x4{0u, 0u, 0u, 0u};
    if (in)
        v = load_octet<true>(at_row(base, row, ld, type), type, o, 0);
    return v;
}

// The norms of R rows from `first` on, of which f gives octet i of row j.
template <int C, int R, typename Get>
__device__ __forceinline__ void write_norms(const NormOut &n, const double (&squares_of)[R], const float (&w)[C][8],
                                            int K, long long first, int M, int waves, double (*sums)[16],
                                            unsigned (*tops)[16], Get get)
{
    const float rl = rms_factor(over_rows<R>(squares_of, waves, sums), n.inverse_K, n.eps);
    float r[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
        r[j] = from_lane(rl, lane_with<R>(j));
    RowScale scale8[R];
    if (n.q_kind == SKINNY_ROWS_INT8) {
        unsigned top[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            top[j] = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float f[8];
                get(j, i, f);
                // as in write_norm, past the row zero
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned m = mag(f[e] * r[j] * w[i][e]);
                    top[j] = m > top[j] ? m : top[j];
                }
            }
        }
        const unsigned all = over_rows<R>(top, waves, tops);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float scale;
            scale8[j] = row_scale((unsigned)__builtin_amdgcn_readlane((int)all, lane_with<R>(j)), scale);
            if (threadIdx.x == 0 && first + j < M)
                static_cast<float *>(n.scale)[first + j] = scale;
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float f[8];
            get(j, i, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = f[e] * r[j] * w[i][e];
            Place p;
            p.row = (int)(first + j);
            p.t = (int)threadIdx.x;
            p.in = first + j < M;
            write_octet<kVectors>(n, i, K, (int)blockDim.x, p, scale8[j], f);
            // one after the other, so that the registers of one serve the next
            __builtin_amdgcn_sched_barrier(0);
        }
}

template <int C, int R, int type>
__global__ __launch_bounds__(1024) void norm_stream(NArgs a)
{
    __shared__ double sums[2][4][16];
    __shared__ unsigned tops[2][4][16];
    const int octets = a.K / 8, waves = (int)blockDim.x / 64;
    float w[C][8];
    const auto load = [&](Octet (&x)[R][C], long long first) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int o = (int)threadIdx.x + i * (int)blockDim.x;
                x[j][i] = octet_of<type>(a.x, first + j, a.ldx, type, o < octets && first + j < a.M, o);
            }
    };
    long long first = (long long)blockIdx.x * R;
    const long long stride = (long long)gridDim.x * R;
    Octet x[R][C], next[R][C];
    load(x, first);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int o = (int)threadIdx.x + i * (int)blockDim.x;
        unpack_octet(octet_of<type>(a.n.weight, 0, 0, a.n.weight_type, o < octets, o), a.n.weight_type, w[i]);
    }
    for (int turn = 0; first < a.M; first += stride, turn ^= 1) {
        load(next, first + stride);
        double sum[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            sum[j] = 0.0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float f[8];
                unpack_octet(x[j][i], type, f);
                sum[j] += squares(f);
            }
        }
        write_norms<C, R>(a.n, sum, w, a.K, first, a.M, waves, sums[turn], tops[turn],
                          [&](int j, int i, float (&f)[8]) { unpack_octet(x[j][i], type, f); });
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < C; ++i)
                x[j][i] = next[j][i];
    }
}

template <int C, int R, int y_type, int residual_type>
__global__ __launch_bounds__(1024) void join_stream(JArgs a)
{
    __shared__ double sums[4][4][16];
    __shared__ unsigned tops[2][4][16];
    const int octets = a.K / 8, waves = (int)blockDim.x / 64;
    long long first = (long long)blockIdx.x * R;
    const long long stride = (long long)gridDim.x * R;
    Octet ys[R][C], hs[R][C], next_y[R][C], next_h[R][C];
    const auto load = [&](Octet (&y)[R][C], Octet (&h)[R][C], long long from) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int o = (int)threadIdx.x + i * (int)blockDim.x;
                const bool in = o < octets && from + j < a.M;
                y[j][i] = octet_of<y_type>(a.y, from + j, a.ldy, y_type, in, o);
                h[j][i] = octet_of<y_type>(a.residual, from + j, a.ldr, residual_type, in, o);
            }
    };
    load(ys, hs, first);
    float w[C][8], c[C][8], nw[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int o = (int)threadIdx.x + i * (int)blockDim.x;
        const bool in = o < octets;
        unpack_octet(octet_of<y_type>(a.weight, 0, 0, a.weight_type, in && a.weight, o), a.weight_type, w[i]);
        unpack_octet(octet_of<y_type>(a.n.weight, 0, 0, a.n.weight_type, in && a.n.weight, o), a.n.weight_type, nw[i]);
        unpack_octet(octet_of<y_type>(a.gate, 0, 0, a.gate_type, in && a.gate, o), a.gate_type, c[i]);
        if (a.sigmoid)
            sigmoid(c[i]);
    }
    for (int turn = 0; first < a.M; first += stride, turn ^= 1) {
        load(next_y, next_h, first + stride);
        float r[R];
        double sum[R];
        if (a.weight) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                sum[j] = 0.0;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    float f[8];
                    unpack_octet(ys[j][i], y_type, f);
                    sum[j] += squares(f);
                }
            }
            const float rl = rms_factor(over_rows<R>(sum, waves, sums[turn]), a.inverse_K, a.eps);
#pragma unroll
            for (int j = 0; j < R; ++j)
                r[j] = from_lane(rl, lane_with<R>(j));
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            sum[j] = 0.0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int o = (int)threadIdx.x + i * (int)blockDim.x;
                float z[8], h[8];
                unpack_octet(ys[j][i], y_type, z);
                unpack_octet(hs[j][i], residual_type, h);
                if (a.weight) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = z[e] * r[j] * w[i][e];
                }
                if (a.gate) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] *= c[i][e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[e] = h[e] * a.beta + z[e] * a.alpha;
                // as it is held from here on
                const Octet v = pack_octet(residual_type, h);
                hs[j][i] = v;
                const bool here = o < octets && first + j < a.M;
                if (here) {
                    store_octet<true>(const_cast<char *>(at_row(a.out, first + j, a.ldo, residual_type)), residual_type,
                                      o, 0, v);
                    sum[j] += squares(h);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (a.n.weight)
            write_norms<C, R>(a.n, sum, nw, a.K, first, a.M, waves, sums[2 + turn], tops[turn],
                              [&](int j, int i, float (&f)[8]) { unpack_octet(hs[j][i], residual_type, f); });
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                ys[j][i] = next_y[j][i];
                hs[j][i] = next_h[j][i];
            }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Whether octets of rows at p lie at 16-byte aligned places.
bool whole_octets(const void *p, long long ld, int type)
{
    return (uintptr_t)p % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

// The norm's kernel for many rows: one row at a time, or four of 16-bit values
// in up to 1024 octets.
template <int X>
const void *norm_stream_fn(int c, int rows)
{
    if constexpr (X != SKINNY_TYPE_F32)
        if (rows == 4)
            return reinterpret_cast<const void *>(norm_stream<1, 4, X>);
    return c == 1   ? reinterpret_cast<const void *>(norm_stream<1, 1, X>)
           : c == 2 ? reinterpret_cast<const void *>(norm_stream<2, 1, X>)
                    : reinterpret_cast<const void *>(norm_stream<3, 1, X>);
}

template <int Y, int R>
const void *join_stream_fn()
{
    return reinterpret_cast<const void *>(join_stream<1, join_rows_of(Y, R), Y, R>);
}

template <int X>
const void *norm_fn(int octets, Mode mode)
{
    if (mode == kElements)
        return octets == 1 ? reinterpret_cast<const void *>(norm_kernel<1, kElements, X>)
                           : reinterpret_cast<const void *>(norm_kernel<0, kElements, X>);
    if (mode == kStrided)
        return octets == 1   ? reinterpret_cast<const void *>(norm_kernel<1, kStrided, X>)
               : octets == 2 ? reinterpret_cast<const void *>(norm_kernel<2, kStrided, X>)
                             : reinterpret_cast<const void *>(norm_kernel<0, kStrided, X>);
    return octets == 1   ? reinterpret_cast<const void *>(norm_kernel<1, kVectors, X>)
           : octets == 2 ? reinterpret_cast<const void *>(norm_kernel<2, kVectors, X>)
           : octets == 4 ? reinterpret_cast<const void *>(norm_kernel<4, kVectors, X>)
                         : reinterpret_cast<const void *>(norm_kernel<0, kVectors, X>);
}

template <int Y, int R>
const void *join_fn(int octets, Mode mode)
{
    if (mode == kElements)
        return octets == 1 ? reinterpret_cast<const void *>(join_kernel<1, kElements, Y, R>)
                           : reinterpret_cast<const void *>(join_kernel<0, kElements, Y, R>);
    if (mode == kStrided)
        return octets == 1   ? reinterpret_cast<const void *>(join_kernel<1, kStrided, Y, R>)
               : octets == 2 ? reinterpret_cast<const void *>(join_kernel<2, kStrided, Y, R>)
                             : reinterpret_cast<const void *>(join_kernel<0, kStrided, Y, R>);
    return octets == 1   ? reinterpret_cast<const void *>(join_kernel<1, kVectors, Y, R>)
           : octets == 2 ? reinterpret_cast<const void *>(join_kernel<2, kVectors, Y, R>)
           : octets == 4 ? reinterpret_cast<const void *>(join_kernel<4, kVectors, Y, R>)
                         : reinterpret_cast<const void *>(join_kernel<0, kVectors, Y, R>);
}

const void *pick_norm_kernel(int octets, Mode mode, int type)
{
    return type == SKINNY_TYPE_F32   ? norm_fn<SKINNY_TYPE_F32>(octets, mode)
           : type == SKINNY_TYPE_F16 ? norm_fn<SKINNY_TYPE_F16>(octets, mode)
                                     : norm_fn<SKINNY_TYPE_BF16>(octets, mode);
}

template <int Y>
const void *pick_join_of(int octets, Mode mode, int residual_type)
{
    return residual_type == SKINNY_TYPE_F32   ? join_fn<Y, SKINNY_TYPE_F32>(octets, mode)
           : residual_type == SKINNY_TYPE_F16 ? join_fn<Y, SKINNY_TYPE_F16>(octets, mode)
                                              : join_fn<Y, SKINNY_TYPE_BF16>(octets, mode);
}

const void *pick_join_kernel(int octets, Mode mode, int y_type, int residual_type)
{
    return y_type == SKINNY_TYPE_F32   ? pick_join_of<SKINNY_TYPE_F32>(octets, mode, residual_type)
           : y_type == SKINNY_TYPE_F16 ? pick_join_of<SKINNY_TYPE_F16>(octets, mode, residual_type)
                                       : pick_join_of<SKINNY_TYPE_BF16>(octets, mode, residual_type);
}

template <int Y>
const void *join_stream_type(int residual_type)
{
    return residual_type == SKINNY_TYPE_F32   ? join_stream_fn<Y, SKINNY_TYPE_F32>()
           : residual_type == SKINNY_TYPE_F16 ? join_stream_fn<Y, SKINNY_TYPE_F16>()
                                              : join_stream_fn<Y, SKINNY_TYPE_BF16>();
}

const void *pick_join_stream(int y_type, int residual_type)
{
    return y_type == SKINNY_TYPE_F32   ? join_stream_type<SKINNY_TYPE_F32>(residual_type)
           : y_type == SKINNY_TYPE_F16 ? join_stream_type<SKINNY_TYPE_F16>(residual_type)
                                       : join_stream_type<SKINNY_TYPE_BF16>(residual_type);
}

// What both entries ask of a norm's weight and places; K and M are checked.
skinny_status check_norm(const NormOut &n, int K)
{
    if (!is_type(n.weight_type))
        return bad(SKINNY_ERR_INVALID_ARG, "weight type %d is none of BF16, F32 and F16", n.weight_type);
    if (!(n.eps >= 0x1p-120 && n.eps <= 0x1p120))
        return bad(SKINNY_ERR_INVALID_ARG, "eps=%g must be from 2^-120 to 2^120", n.eps);
    if (n.out && !is_type(n.out_type))
        return bad(SKINNY_ERR_INVALID_ARG, "output type %d is none of BF16, F32 and F16", n.out_type);
    if (n.out && n.ldo < K)
        return bad(SKINNY_ERR_SHAPE, "a norm's pitch %lld must be at least K=%d", n.ldo, K);
    if (n.q_kind < SKINNY_ROWS_NONE || n.q_kind > SKINNY_ROWS_MX8)
        return bad(SKINNY_ERR_INVALID_ARG, "q_kind=%d is none of the kinds of rows", n.q_kind);
    if (!n.out && n.q_kind == SKINNY_ROWS_NONE)
        return bad(SKINNY_ERR_INVALID_ARG, "nothing to write: out is NULL and q_kind is SKINNY_ROWS_NONE");
    if (n.q_kind != SKINNY_ROWS_NONE && (!n.q || !n.scale))
        return bad(SKINNY_ERR_INVALID_ARG, "q or scale is NULL");
    const bool mx = n.q_kind == SKINNY_ROWS_MX4 || n.q_kind == SKINNY_ROWS_MX8;
    if (mx && K % kBlock)
        return bad(SKINNY_ERR_SHAPE, "K=%d must be a multiple of 32, whole blocks", K);
    const long long row_bytes = n.q_kind == SKINNY_ROWS_MX4 ? K / 2 : K;
    if (n.q_kind != SKINNY_ROWS_NONE && n.ldq < row_bytes)
        return bad(SKINNY_ERR_SHAPE, "ldq=%lld must be at least %lld bytes", n.ldq, row_bytes);
    if (mx && n.lds < K / kBlock)
        return bad(SKINNY_ERR_SHAPE, "lds=%lld must be at least %d", n.lds, K / kBlock);
    if ((n.out && (uintptr_t)n.out % type_bytes(n.out_type)) || (uintptr_t)n.weight % type_bytes(n.weight_type) ||
        (n.q_kind == SKINNY_ROWS_INT8 && (uintptr_t)n.scale % 4))
        return bad(SKINNY_ERR_ALIGN, "weights, outputs and fp32 scales must be aligned to their elements");
    return SKINNY_OK;
}

bool norm_octets(const NormOut &n)
{
    const int bytes = n.q_kind == SKINNY_ROWS_MX4 ? 4 : 8;
    return whole_octets(n.weight, 0, n.weight_type) && (!n.out || whole_octets(n.out, n.ldo, n.out_type)) &&
           (n.q_kind == SKINNY_ROWS_NONE || ((uintptr_t)n.q % bytes == 0 && n.ldq % bytes == 0));
}

// The norm's places `rows` rows on.
void advance(NormOut &n, int rows)
{
    if (n.out)
        n.out = static_cast<char *>(n.out) + rows * n.ldo * type_bytes(n.out_type);
    if (n.q_kind != SKINNY_ROWS_NONE) {
        n.q += rows * n.ldq;
        n.scale = static_cast<char *>(n.scale) + (n.q_kind == SKINNY_ROWS_INT8 ? 4LL * rows : rows * n.lds);
    }
}

NormOut norm_out(const void *weight, int weight_type, void *out, int out_type, long long ldo, int q_kind, void *q,
                 long long ldq, void *scale, long long lds, double eps, int K)
{
    NormOut n{};
    n.weight = weight;
    n.weight_type = weight_type;
    n.out = out;
    n.out_type = out_type;
    n.ldo = ldo;
    n.q_kind = q_kind;
    n.q = static_cast<unsigned char *>(q);
    n.ldq = ldq;
    n.scale = scale;
    n.lds = lds;
    n.eps = eps;
    n.inverse_K = 1.0 / K;
    return n;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" {

skinny_status skinny_norm_rows(const skinny_norm_args *p, void *stream)
{
    if (!p)
        return bad(SKINNY_ERR_INVALID_ARG, "args is NULL");
    if (!is_type(p->x_type))
        return bad(SKINNY_ERR_INVALID_ARG, "x type %d is none of BF16, F32 and F16", p->x_type);
    if (p->M < 0 || p->K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d and K=%d: M >= 0 and K >= 1 are needed", p->M, p->K);
    if (p->M == 0)
        return SKINNY_OK;
    if (!p->x || !p->weight)
        return bad(SKINNY_ERR_INVALID_ARG, "x or weight is NULL");
    if (p->ldx < p->K)
        return bad(SKINNY_ERR_SHAPE, "ldx=%lld must be at least K=%d", p->ldx, p->K);
    if ((uintptr_t)p->x % type_bytes(p->x_type))
        return bad(SKINNY_ERR_ALIGN, "x must be aligned to its elements");
    NArgs a{};
    a.n = norm_out(p->weight, p->weight_type, p->out, p->out_type, p->ldo, p->q_kind, p->q, p->ldq, p->scale, p->lds,
                   p->eps, p->K);
    const skinny_status st = check_norm(a.n, p->K);
    if (st != SKINNY_OK)
        return st;
    const bool vec = p->K % 8 == 0 && whole_octets(p->x, p->ldx, p->x_type) && norm_octets(a.n);
    a.x = p->x;
    a.ldx = p->ldx;
    a.type = p->x_type;
    a.K = p->K;
    const RowStream stream_shape = norm_stream_of(p->M, p->K, a.type, vec);
    if (stream_shape.c) {
        a.M = p->M;
        const void *many = a.type == SKINNY_TYPE_F32   ? norm_stream_fn<SKINNY_TYPE_F32>(stream_shape.c, stream_shape.rows)
                           : a.type == SKINNY_TYPE_F16 ? norm_stream_fn<SKINNY_TYPE_F16>(stream_shape.c, stream_shape.rows)
                                                       : norm_stream_fn<SKINNY_TYPE_BF16>(stream_shape.c, stream_shape.rows);
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(many, dim3((unsigned)stream_shape.groups),
                                             dim3((unsigned)stream_shape.threads), params, 0, (hipStream_t)stream);
        return e == hipSuccess ? SKINNY_OK : hip_bad(e, "norm launch");
    }
    const Mode mode = mode_of(vec, a.n.q_kind);
    const RowShape s = row_shape_of(p->M, p->K, mode);
    a.lanes = s.lanes;
    const void *fn = pick_norm_kernel(s.octets, mode, a.type);
    const int most = rows_of_launch(s), per_group = s.threads / s.lanes;
    for (int left = p->M; left > 0; left -= most) {
        a.M = left < most ? left : most;
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)((a.M + per_group - 1) / per_group)),
                                             dim3((unsigned)s.threads), params, 0, (hipStream_t)stream);
        if (e != hipSuccess)
            return hip_bad(e, "norm launch");
        a.x = static_cast<const char *>(a.x) + a.M * a.ldx * type_bytes(a.type);
        advance(a.n, a.M);
    }
    return SKINNY_OK;
}

skinny_status skinny_join_rows(const skinny_join_args *p, void *stream)
{
    if (!p)
        return bad(SKINNY_ERR_INVALID_ARG, "args is NULL");
    if (!is_type(p->residual_type) || !is_type(p->y_type) || (p->gate && !is_type(p->gate_type)) ||
        (p->weight && !is_type(p->weight_type)))
        return bad(SKINNY_ERR_INVALID_ARG, "a type of residual (%d), y (%d), gate (%d) and weight (%d) is none of BF16, "
                   "F32 and F16", p->residual_type, p->y_type, p->gate_type, p->weight_type);
    if (p->M < 0 || p->K < 1)
        return bad(SKINNY_ERR_INVALID_ARG, "M=%d and K=%d: M >= 0 and K >= 1 are needed", p->M, p->K);
    if (p->M == 0)
        return SKINNY_OK;
    if (!p->residual || !p->y || !p->out)
        return bad(SKINNY_ERR_INVALID_ARG, "residual, y or out is NULL");
    if (p->ldr < p->K || p->ldy < p->K || p->ldo < p->K || (p->gate && p->ldg != 0 && p->ldg < p->K))
        return bad(SKINNY_ERR_SHAPE, "ldr=%lld, ldy=%lld, ldo=%lld and ldg=%lld (or 0) must be at least K=%d", p->ldr,
                   p->ldy, p->ldo, p->ldg, p->K);
    if ((uintptr_t)p->residual % type_bytes(p->residual_type) || (uintptr_t)p->out % type_bytes(p->residual_type) ||
        (uintptr_t)p->y % type_bytes(p->y_type) || (p->gate && (uintptr_t)p->gate % type_bytes(p->gate_type)) ||
        (p->weight && (uintptr_t)p->weight % type_bytes(p->weight_type)))
        return bad(SKINNY_ERR_ALIGN, "residual, y, out, gate and weight must be aligned to their elements");
    if (!(p->eps >= 0x1p-120 && p->eps <= 0x1p120))
        return bad(SKINNY_ERR_INVALID_ARG, "eps=%g must be from 2^-120 to 2^120", p->eps);
    JArgs a{};
    const bool next = p->next_weight != nullptr;
    if (next) {
        a.n = norm_out(p->next_weight, p->next_weight_type, p->next_out, p->next_type, p->ldn, p->q_kind, p->q, p->ldq,
                       p->scale, p->lds, p->eps, p->K);
        const skinny_status st = check_norm(a.n, p->K);
        if (st != SKINNY_OK)
            return st;
    } else if (p->next_out || p->q_kind != SKINNY_ROWS_NONE) {
        return bad(SKINNY_ERR_INVALID_ARG, "a place for the next norm without its weight");
    }
    const bool vec = p->K % 8 == 0 && whole_octets(p->residual, p->ldr, p->residual_type) &&
                     whole_octets(p->y, p->ldy, p->y_type) && whole_octets(p->out, p->ldo, p->residual_type) &&
                     (!p->gate || whole_octets(p->gate, p->ldg, p->gate_type)) &&
                     (!p->weight || whole_octets(p->weight, 0, p->weight_type)) && (!next || norm_octets(a.n));
    a.residual = p->residual;
    a.y = p->y;
    a.weight = p->weight;
    a.gate = p->gate;
    a.out = p->out;
    a.ldr = p->ldr;
    a.ldy = p->ldy;
    a.ldg = p->ldg;
    a.ldo = p->ldo;
    a.eps = p->eps;
    a.inverse_K = 1.0 / p->K;
    a.alpha = p->alpha;
    a.beta = p->beta;
    a.residual_type = p->residual_type;
    a.y_type = p->y_type;
    a.weight_type = p->weight_type;
    a.gate_type = p->gate_type;
    a.sigmoid = p->sigmoid != 0;
    a.K = p->K;
    const RowStream stream_shape = join_stream_of(p->M, p->K, p->y_type, p->residual_type, vec, p->gate && p->ldg != 0);
    if (stream_shape.c) {
        a.M = p->M;
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(pick_join_stream(a.y_type, a.residual_type),
                                             dim3((unsigned)stream_shape.groups), dim3((unsigned)stream_shape.threads),
                                             params, 0, (hipStream_t)stream);
        return e == hipSuccess ? SKINNY_OK : hip_bad(e, "join launch");
    }
    const Mode mode = mode_of(vec, a.n.q_kind);
    const RowShape s = row_shape_of(p->M, p->K, mode);
    a.lanes = s.lanes;
    const void *fn = pick_join_kernel(s.octets, mode, a.y_type, a.residual_type);
    const int most = rows_of_launch(s), per_group = s.threads / s.lanes;
    for (int left = p->M; left > 0; left -= most) {
        a.M = left < most ? left : most;
        void *params[] = {&a};
        const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)((a.M + per_group - 1) / per_group)),
                                             dim3((unsigned)s.threads), params, 0, (hipStream_t)stream);
        if (e != hipSuccess)
            return hip_bad(e, "join launch");
        a.residual = static_cast<const char *>(a.residual) + a.M * a.ldr * type_bytes(a.residual_type);
        a.y = static_cast<const char *>(a.y) + a.M * a.ldy * type_bytes(a.y_type);
        a.out = static_cast<char *>(a.out) + a.M * a.ldo * type_bytes(a.residual_type);
        if (a.gate)
            a.gate = static_cast<const char *>(a.gate) + a.M * a.ldg * type_bytes(a.gate_type);
        if (next)
            advance(a.n, a.M);
    }
    return SKINNY_OK;
}

}  // extern "C"
