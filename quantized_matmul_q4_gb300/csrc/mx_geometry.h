// Launch geometry of the MX products: plain host C++ (no CUDA types), so that
// the CPU tests compile this same header and check it.
#pragma once

namespace q4mm {

#if defined(__CUDACC__)
#define Q4MM_HD __host__ __device__
#else
#define Q4MM_HD
#endif

// A split tile's 128 rows are shared out in fours: rank s of S adds up the
// rows from first_row(s) to first_row(s + 1).
constexpr int kMxMaxSplit = 8;  // a portable cluster
Q4MM_HD constexpr int mx_first_row(int s, int S) { return 4 * (32 * s / S); }

// CTAs that share a tile's K: as many as fill the SMs with two CTAs each, at
// most 8 and two stages of K to each.
inline int mx_split(int row_tiles, int tok_tiles, int stages, int num_sms) {
    const long long tiles = (long long)row_tiles * tok_tiles;
    int S = 1;
    while (S < kMxMaxSplit && tiles * (S + 1) <= 2LL * num_sms && 2 * (S + 1) <= stages) ++S;
    return S;
}

// Tiles of the CTA-pair kernel: 256 weight rows by tile_tok tokens, a multiple
// of 32 up to 256 that splits the tokens evenly.  x_tiles: 128-row scale
// tiles that the tokens of any tile touch, counted from the tile that holds
// its first token.
struct MxPairTiles {
    int tile_tok, tok_tiles, row_tiles, x_tiles;
};
inline MxPairTiles mx_pair_tiles(int T, int N) {
    MxPairTiles g;
    g.tok_tiles = (int)(((long long)T + 255) / 256);
    const int each = (int)(((long long)T + g.tok_tiles - 1) / g.tok_tiles);
    g.tile_tok = (each + 31) / 32 * 32;
    g.row_tiles = (int)(((long long)N + 255) / 256);
    // The first token's offset in its scale tile is a multiple of
    // gcd(tile_tok, 128).
    int step = 128;
    while (g.tile_tok % step) step /= 2;
    const int offset = g.tok_tiles > 1 ? 128 - step : 0;
    g.x_tiles = (offset + g.tile_tok + 127) / 128;
    return g;
}

// Pairs or single CTAs with K split?
inline bool mx_use_pairs(int T, int N, int num_sms) {
    const MxPairTiles g = mx_pair_tiles(T, N);
    return T > 128 && 2LL * g.row_tiles * g.tok_tiles >= num_sms / 2;
}

}  // namespace q4mm
