// How norms.hip deals rows to threads, from their sizes alone: code without
// HIP, so that it is tested without it too.
#pragma once

#include "../../include/skinny.h"

namespace skinny {

// How a row's elements go to its threads, eight a turn: neighbours in whole
// 16-byte vectors; neighbours one by one (blocks at unaligned places); or lanes
// side by side, so that a load of single elements takes whole lines (4000 x 4097
// in FP16: 35 to 36 against 57 us).
enum Mode { kVectors, kElements, kStrided };

inline Mode mode_of(bool vec, int q_kind)
{
    return vec ? kVectors : q_kind == SKINNY_ROWS_MX4 || q_kind == SKINNY_ROWS_MX8 ? kElements : kStrided;
}

// Octets of a row of K >= 1 elements, the last one part full.  K + 7 may pass 2^31; counted
// unsigned for that, joins of 4000 x 7168 took 65.9 us in place of 65.4.
constexpr int octets_of(int K) { return (K - 1) / 8 + 1; }

// Octets a thread keeps (0: any number, read again) and threads a row.
struct RowShape {
    int octets, lanes, threads;
};

inline RowShape row_shape_of(int M, int K, Mode mode)
{
    const int octets = octets_of(K);
    // few rows: one octet a thread; many: up to four, so that a workgroup has more
    // loads under way (single elements have eight times the loads anyway)
    const int each = M <= 512 || mode != kVectors ? 1 : 4;
    int lanes = 16;
    while (lanes < 1024 && lanes * each < octets)
        lanes *= 2;
    const int per = (octets + lanes - 1) / lanes;
    const int most = mode == kVectors ? 4 : mode == kStrided ? 2 : 1;
    const int kept = per <= 1 ? 1 : per <= 2 ? 2 : 4;
    return RowShape{per <= most ? kept : 0, lanes, lanes < 256 ? 256 : lanes};
}

// Rows of a launch of fewer than 2^32 threads.
inline int rows_of_launch(const RowShape &s)
{
    return (int)(0xFFFFFFFFu / (unsigned)s.threads - 1u) * (s.threads / s.lanes);
}

// One of fp32 rows; two of others (4000 x 7168 in BF16 50.0 against 54.5 us).
constexpr int join_rows_of(int y_type, int residual_type)
{
    return y_type == SKINNY_TYPE_F32 || residual_type == SKINNY_TYPE_F32 ? 1 : 2;
}

// Octets a thread, threads a row, rows at a time and workgroups of the kernels for
// many rows; c = 0: not for these.
struct RowStream {
    int c, threads, rows, groups;
};

// `most` octets a thread at most, `waves` of a CU.
inline RowStream row_stream_of(int M, int K, bool vec, int most, int rows, int waves)
{
    const int octets = K / 8, c = (octets + 1023) / 1024;
    // shorter rows go several to a wave
    if (!vec || octets <= 32 || c > most)
        return RowStream{0, 0, 0, 0};
    const int threads = ((octets + c - 1) / c + 63) / 64 * 64;
    const int places = 256 * (64 * waves / threads), batches = (int)(((long long)M + rows - 1) / rows);
    return RowStream{c, threads, rows, batches < places ? batches : places};
}

// From 256 rows on; four at a time where they fill the chip's turns to within a
// twentieth (4003 x 7168 with fp32 weights: 34.5 against 36.3 us one at a time on
// twice the workgroups; 2500: 23.6 against 21.5; row by row 37.7 and 21.6).
inline RowStream norm_stream_of(int M, int K, int type, bool vec)
{
    if (M < 256)
        return RowStream{0, 0, 0, 0};
    if (K > 8192)
        return row_stream_of(M, K, vec, 3, 1, 16);
    const RowStream four = row_stream_of(M, K, vec, 1, 4, 16);
    if (four.c && type != SKINNY_TYPE_F32) {
        const long long turn = 4LL * 256 * (1024 / four.threads), whole = (M + turn - 1) / turn * turn;
        if (M >= 3 * turn && 20 * whole <= 21LL * M)
            return four;
    }
    return row_stream_of(M, K, vec, 1, 1, 32);
}

// From 1024 rows on (600 x 7168: 14.9 us against 12.7 row by row, 1500: 20.3
// against 22.0), but not with a gate for each token, which fills the registers
// (4000 x 7168: 70 against 66 us).
inline RowStream join_stream_of(int M, int K, int y_type, int residual_type, bool vec, bool token_gate)
{
    if (M < 1024 || token_gate)
        return RowStream{0, 0, 0, 0};
    return row_stream_of(M, K, vec, 1, join_rows_of(y_type, residual_type), 16);
}

}  // namespace skinny
