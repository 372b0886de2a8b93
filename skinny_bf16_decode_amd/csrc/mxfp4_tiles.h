// Which kernel and tile a 4-bit product takes, from its sizes alone: host code
// without HIP, so that it is tested without it too.
#pragma once

namespace skinny {

// The largest tiles whose registers fit: 32 * 8 4-bit tokens, 32 * 6 8-bit ones,
// 32 * 4 with powers of any alignment.  32 * 1 is never the shortest: 64 rows by 32 tokens of
// product_rows take at most four of its rounds and less time.
constexpr int kFewest = 2, kTiles = 8, kTiles8 = 6, kAnyTiles = 4;

constexpr int most_tiles(int bits, bool words) { return !words ? kAnyTiles : bits == 4 ? kTiles : kTiles8; }

// A tile shape and the time of its rounds over 256 CUs, in us over K = 7168.
struct Tiling {
    int r, t;                   // 16 r rows by 16 t tokens, or 256 rows by 32 t tokens
    float us;
};

// product_tiles and product_tiles8: a round on the scale of rows_tiling, 8-bit
// tokens' a fifth below what it takes alone.  Over 512 to 6288 rows, 65 to 2000 tokens
// and K = 1536 to 18432 the kernel taken was within a geometric mean of 0.1 % (4
// bits) and 0.8 % (8 bits) of the fastest, at worst 2 and 10 %.
inline Tiling tiles_tiling(int M, int N, int bits, bool words)
{
    static const float us4[kTiles + 1] = {0.0f, 0.0f, 23.5f, 27.0f, 30.4f, 35.5f, 39.3f, 43.5f, 47.6f};
    static const float us8[kTiles8 + 1] = {0.0f, 0.0f, 50.0f, 57.0f, 65.0f, 81.0f, 91.0f};
    Tiling best{0, 0, 0.0f};
    for (int t = most_tiles(bits, words); t >= kFewest; --t) {
        const long long count = ((long long)N + 255) / 256 * ((M + 32 * t - 1) / (32 * t));
        const float us = (float)((count + 255) / 256) * (bits == 4 ? us4 : us8)[t];
        if (!best.r || us < best.us)
            best = Tiling{16, t, us};
    }
    return best;
}

// product_rows: what each further workgroup of a CU adds, measured at K = 7168
// over 1024 to 14336 rows and 1 to 128 tokens (both grow with K alike).  16 x 32
// tiles and those of 48 and 64 tokens were never the fastest (64 x 6288 x 7168:
// 64 rows by 32 tokens 8.8 us, by 64 14.8).  32 rows by 32 8-bit tokens take as many rounds
// as 64 by 16 and are a little ahead: 37 x 3584 x 7168 9.0 against 9.2 us.
inline Tiling rows_tiling(int M, int N, int bits)
{
    static const struct {
        int r, t;
        float us4, us8;
    } kShapes[] = {{1, 1, 1.65f, 2.45f}, {2, 1, 2.05f, 3.2f}, {4, 1, 3.4f, 5.35f}, {2, 2, 3.2f, 5.2f}, {4, 2, 4.6f, 9.7f}};
    Tiling best{0, 0, 0.0f};
    for (const auto &k : kShapes) {
        if (k.t == 2 && M <= 16)
            continue;
        const long long count = ((long long)N + 16 * k.r - 1) / (16 * k.r) * ((M + 16 * k.t - 1) / (16 * k.t));
        const float us = (float)((count + 255) / 256) * (bits == 4 ? k.us4 : k.us8);
        if (!best.r || us < best.us)
            best = Tiling{k.r, k.t, us};
    }
    return best;
}

// The kernel of a product: product_rows of r row tiles by t token tiles, x_rows
// rows of x a load, `once` where the weight passes by once, or (many) a tile kernel.
struct Product {
    bool many;
    int r, t, x_rows;
    bool once;
    long long n_tiles, m_tiles;
};

// Up to 64 tokens product_rows, above the shorter of both: 400 tokens of 6288 x 7168
// 27.7 against 23.6 us in 4 bits, of 1536 x 7168 12.1 against 21.2.
inline Product product_of(int M, int N, int bits, bool words)
{
    const Tiling rows = rows_tiling(M, N, bits);
    const Tiling tiles = M > 64 ? tiles_tiling(M, N, bits, words) : rows;
    const bool many = tiles.us < rows.us;
    const int n_rows = many ? 256 : 16 * rows.r, tokens = many ? 32 * tiles.t : 16 * rows.t;
    Product p;
    p.many = many;
    p.r = many ? tiles.r : rows.r;
    p.t = many ? tiles.t : rows.t;
    p.n_tiles = ((long long)N + n_rows - 1) / n_rows;
    p.m_tiles = ((long long)M + tokens - 1) / tokens;
    p.once = !many && p.m_tiles == 1;
    p.x_rows = many ? 0 : M <= 4 ? 4 : M <= 8 ? 8 : 16;
    return p;
}

}  // namespace skinny
