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
    double eps;
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
    double eps;
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

// The sum of a row's threads' v, in every one of them.
__device__ __forceinline__ double row_sum(double v, int lanes, const Place &p, double *shared)
{
    const int within = lanes < 64 ? lanes : 64;
    for (int s = 1; s < within; s *= 2)
        v += __shfl_xor(v, s, 64);
    if (lanes > 64) {
        const int wave = (int)threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            shared[wave] = v;
        __syncthreads();
        v = 0.0;
        for (int w = 0; w < p.waves; ++w)
            v += shared[p.first_wave + w];
    }
    return v;
}

__device__ __forceinline__ unsigned row_max(unsigned v, int lanes, const Place &p, double *shared)
{
    const int within = lanes < 64 ? lanes : 64;
    for (int s = 1; s < within; s *= 2) {
        const unsigned o = (unsigned)__shfl_xor((int)v, s, 64);
        v = o > v ? o : v;
    }
    if (lanes > 64) {
        unsigned *tops = reinterpret_cast<unsigned *>(shared);
        const int wave = (int)threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            tops[wave] = v;
        __syncthreads();
        for (int w = 0; w < p.waves; ++w) {
            const unsigned o = tops[p.first_wave + w];
            v = o > v ? o : v;
        }
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

__device__ __forceinline__ float rms_factor(double sum, int K, double eps)
{
    return (float)(1.0 / sqrt(sum / (double)K + eps));
}

__device__ __forceinline__ const char *at_row(const void *p, long long row, long long ld, int type)
{
    return static_cast<const char *>(p) + row * ld * (type == SKINNY_TYPE_F32 ? 4 : 2);
}

// The norm of a row whose octets get(i, f) gives, i = 0, 1, ... for the octets
// t + i lanes of this thread; f is zero past the row.  OCTETS: how many at most, 0: any.
template <bool VEC, int OCTETS, typename Get>
__device__ __forceinline__ void write_norm(const NormOut &n, double sum, int K, int lanes, const Place &p,
                                           double *shared, Get get)
{
    const int octets = (K + 7) / 8, turns = OCTETS ? OCTETS : (octets + lanes - 1) / lanes;
    const float r = rms_factor(sum, K, n.eps);
    const auto value = [&](int i, float (&f)[8]) {
        const int o = p.t + i * lanes;
        get(i, f);
        float w[8];
        Octet raw;
        raw.a = raw.b = u32x4{0u, 0u, 0u, 0u};
        if (o < octets)
            raw = load_octet<VEC>(n.weight, n.weight_type, o, K);
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
#pragma unroll
        for (int i = 0; i < turns; ++i) {
            float f[8];
            value(i, f);
            // past the row the weight is zero, and r may be infinite or NaN
            const int left = K - 8 * (p.t + i * lanes);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned m = e < left ? mag(f[e]) : 0u;
                top = m > top ? m : top;
            }
        }
        float scale;
        scale8 = row_scale(row_max(top, lanes, p, shared), scale);
        if (p.in && p.t == 0)
            static_cast<float *>(n.scale)[p.row] = scale;
    }
#pragma unroll
    for (int i = 0; i < turns; ++i) {
        const int o = p.t + i * lanes;
        float f[8];
        value(i, f);
        const bool here = p.in && o < octets;
        if (n.q_kind == SKINNY_ROWS_MX4 || n.q_kind == SKINNY_ROWS_MX8) {
            unsigned byte;
            unsigned char *q = n.q + p.row * n.ldq;
            if (n.q_kind == SKINNY_ROWS_MX4) {
                const u32x2 codes = block_codes<4>(f, byte);
                if (here)
                    store_codes<VEC, 4>(q, o, codes);
            } else {
                const u32x2 codes = block_codes<8>(f, byte);
                if (here)
                    store_codes<VEC, 8>(q, o, codes);
            }
            if (here && (o & 3) == 0)
                static_cast<unsigned char *>(n.scale)[p.row * n.lds + (o >> 2)] = (unsigned char)byte;
        } else if (n.q_kind == SKINNY_ROWS_INT8 && here) {
            unsigned char *q = n.q + p.row * n.ldq;
            u32x2 codes;
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                codes[e / 4] = (unsigned)(to_int8(f[e], scale8) & 0xFF) | (unsigned)(to_int8(f[e + 1], scale8) & 0xFF) << 8 |
                               (unsigned)(to_int8(f[e + 2], scale8) & 0xFF) << 16 | (unsigned)to_int8(f[e + 3], scale8) << 24;
            if constexpr (VEC) {
                store_codes<true, 8>(q, o, codes);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned w = codes[e / 4];
                    if (8LL * o + e < K)
                        q[8LL * o + e] = (unsigned char)(w >> (8 * (e & 3)));
                }
            }
        }
        if (n.out && here) {
            const Octet y = pack_octet(n.out_type, f);
            store_octet<VEC>(const_cast<char *>(at_row(n.out, p.row, n.ldo, n.out_type)), n.out_type, o, K, y);
        }
    }
}

// A row's octets stay in registers between the sum and the norm (OCTETS = 0:
// the row is longer than that, and read again).
template <int OCTETS, bool VEC>
__global__ __launch_bounds__(1024) void norm_kernel(NArgs a)
{
    __shared__ double shared[16];
    const Place p = place_of(a.lanes, a.M);
    const char *x = at_row(a.x, p.row, a.ldx, a.type);
    const int octets = (a.K + 7) / 8, turns = OCTETS ? OCTETS : (octets + a.lanes - 1) / a.lanes;
    const auto load = [&](int i) {
        const int o = p.t + i * a.lanes;
        Octet v;
        v.a = v.b = u32x4{0u, 0u, 0u, 0u};
        if (o < octets)
            v = load_octet<VEC>(x, a.type, o, a.K);
        return v;
    };
    Octet keep[OCTETS ? OCTETS : 1];
    double sum = 0.0;
    if constexpr (OCTETS > 0) {
#pragma unroll
        for (int i = 0; i < OCTETS; ++i)
            keep[i] = load(i);
    }
#pragma unroll
    for (int i = 0; i < turns; ++i) {
        float f[8];
        unpack_octet(OCTETS ? keep[OCTETS ? i : 0] : load(i), a.type, f);
        sum += squares(f);
    }
    sum = row_sum(sum, a.lanes, p, shared);
    write_norm<VEC, OCTETS>(a.n, sum, a.K, a.lanes, p, shared, [&](int i, float (&f)[8]) {
        unpack_octet(OCTETS ? keep[OCTETS ? i : 0] : load(i), a.type, f);
    });
}

template <int OCTETS, bool VEC>
__global__ __launch_bounds__(1024) void join_kernel(JArgs a)
{
    __shared__ double shared[16];
    const Place p = place_of(a.lanes, a.M);
    const char *y = at_row(a.y, p.row, a.ldy, a.y_type);
    const char *res = at_row(a.residual, p.row, a.ldr, a.residual_type);
    const char *gate = a.gate ? at_row(a.gate, p.row, a.ldg, a.gate_type) : nullptr;
    char *out = const_cast<char *>(at_row(a.out, p.row, a.ldo, a.residual_type));
    const int octets = (a.K + 7) / 8, turns = OCTETS ? OCTETS : (octets + a.lanes - 1) / a.lanes;
    const auto load = [&](const void *row, int type, int i) {
        const int o = p.t + i * a.lanes;
        Octet v;
        v.a = v.b = u32x4{0u, 0u, 0u, 0u};
        if (o < octets)
            v = load_octet<VEC>(row, type, o, a.K);
        return v;
    };
    Octet ys[OCTETS ? OCTETS : 1], hs[OCTETS ? OCTETS : 1];
    if constexpr (OCTETS > 0) {
#pragma unroll
        for (int i = 0; i < OCTETS; ++i) {
            ys[i] = load(y, a.y_type, i);
            hs[i] = load(res, a.residual_type, i);
        }
    }
    float r = 1.0f;
    if (a.weight) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < turns; ++i) {
            float f[8];
            unpack_octet(OCTETS ? ys[OCTETS ? i : 0] : load(y, a.y_type, i), a.y_type, f);
            sum += squares(f);
        }
        r = rms_factor(row_sum(sum, a.lanes, p, shared), a.K, a.eps);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < turns; ++i) {
        const int o = p.t + i * a.lanes;
        float z[8], h[8];
        unpack_octet(OCTETS ? ys[OCTETS ? i : 0] : load(y, a.y_type, i), a.y_type, z);
        unpack_octet(OCTETS ? hs[OCTETS ? i : 0] : load(res, a.residual_type, i), a.residual_type, h);
        if (a.weight) {
            float w[8];
            unpack_octet(load(a.weight, a.weight_type, i), a.weight_type, w);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = z[e] * r * w[e];
        }
        if (gate) {
            float g[8];
            unpack_octet(load(gate, a.gate_type, i), a.gate_type, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] *= a.sigmoid ? 1.0f / (1.0f + expf(-g[e])) : g[e];
        }
        const int left = a.K - 8 * o;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[e] = e < left ? h[e] * a.beta + z[e] * a.alpha : 0.0f;
        // as it is held from here on
        const Octet v = pack_octet(a.residual_type, h);
        if (OCTETS)
            hs[OCTETS ? i : 0] = v;
        if (p.in && o < octets)
            store_octet<VEC>(out, a.residual_type, o, a.K, v);
        sum += squares(h);
    }
    if (!a.n.weight)
        return;
    sum = row_sum(sum, a.lanes, p, shared);
    // without registers: what this thread has written
    write_norm<VEC, OCTETS>(a.n, sum, a.K, a.lanes, p, shared, [&](int i, float (&f)[8]) {
        unpack_octet(OCTETS ? hs[OCTETS ? i : 0] : load(out, a.residual_type, i), a.residual_type, f);
    });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Whether octets of rows at p lie at 16-byte aligned places.
bool whole_octets(const void *p, long long ld, int type)
{
    return (uintptr_t)p % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

// Octets a thread keeps and threads a row.
struct Shape {
    int octets, lanes, threads;
};

Shape shape_of(int M, int K)
{
    const int octets = (K + 7) / 8;
    // few rows: one octet a thread; many: up to four, so that a workgroup has more loads under way
    const int each = M <= 512 ? 1 : 4;
    int lanes = 16;
    while (lanes < 1024 && lanes * each < octets)
        lanes *= 2;
    const int per = (octets + lanes - 1) / lanes;
    return Shape{per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 0, lanes, lanes < 256 ? 256 : lanes};
}

#define SKINNY_PICK(kernel)                                                                          \
    const void *pick_##kernel(int octets, bool vec)                                                  \
    {                                                                                                \
        if (vec)                                                                                     \
            return octets == 1   ? reinterpret_cast<const void *>(kernel<1, true>)                   \
                   : octets == 2 ? reinterpret_cast<const void *>(kernel<2, true>)                   \
                   : octets == 4 ? reinterpret_cast<const void *>(kernel<4, true>)                   \
                                 : reinterpret_cast<const void *>(kernel<0, true>);                  \
        return octets == 1 ? reinterpret_cast<const void *>(kernel<1, false>)                        \
                           : reinterpret_cast<const void *>(kernel<0, false>);                       \
    }
SKINNY_PICK(norm_kernel)
SKINNY_PICK(join_kernel)
#undef SKINNY_PICK

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
                 long long ldq, void *scale, long long lds, double eps)
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
    return n;
}

// Rows of a launch of fewer than 2^32 threads.
int rows_of_launch(const Shape &s) { return (int)(0xFFFFFFFFu / (unsigned)s.threads - 1u) * (s.threads / s.lanes); }

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
                   p->eps);
    const skinny_status st = check_norm(a.n, p->K);
    if (st != SKINNY_OK)
        return st;
    const Shape s = shape_of(p->M, p->K);
    const bool vec = p->K % 8 == 0 && whole_octets(p->x, p->ldx, p->x_type) && norm_octets(a.n);
    a.x = p->x;
    a.ldx = p->ldx;
    a.type = p->x_type;
    a.K = p->K;
    a.lanes = s.lanes;
    const void *fn = pick_norm_kernel(s.octets, vec);
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
                       p->scale, p->lds, p->eps);
        const skinny_status st = check_norm(a.n, p->K);
        if (st != SKINNY_OK)
            return st;
    } else if (p->next_out || p->q_kind != SKINNY_ROWS_NONE) {
        return bad(SKINNY_ERR_INVALID_ARG, "a place for the next norm without its weight");
    }
    const Shape s = shape_of(p->M, p->K);
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
    a.alpha = p->alpha;
    a.beta = p->beta;
    a.residual_type = p->residual_type;
    a.y_type = p->y_type;
    a.weight_type = p->weight_type;
    a.gate_type = p->gate_type;
    a.sigmoid = p->sigmoid != 0;
    a.K = p->K;
    a.lanes = s.lanes;
    const void *fn = pick_join_kernel(s.octets, vec);
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
