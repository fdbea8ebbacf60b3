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

// Estimates, in microseconds of a call, of the two forms of the product; the
// form and the split with the lower estimate run.  `stages` are ring stages
// of K (256 values with 4-bit x, 128 with 8-bit).  The constants are fitted
// to 1144 measurements of 286 products on GB300 (chains of calls in a CUDA
// graph, 17 to 2048 tokens, K and N of 256 to 16384, with 1, 2 and 4 times
// the fewest tiles of tokens), where the choice costs 0.4% on the mean against
// always the fastest, 8% at most; some of them, single CTAs with K split / CTA
// pairs:
//   T    K        N       x     measured       estimated
//   17   256   -> 4096    4     2.5 /  3.5      2.3 /  3.4
//   64   4096  -> 4096    8     6.6 /  8.1      7.0 /  8.1
//   64   2560  -> 6912    4     6.2 /  4.8      6.1 /  5.1
//   128  1024  -> 4096    8     6.4 /  4.5      6.4 /  4.8
//   128  4096  -> 4096    4     7.2 /  6.0      7.4 /  6.2
//   128  4096  -> 11008   8    12.7 /  9.7     12.6 /  9.3
//   200  4096  -> 4096    8    10.7 /  9.0     11.5 /  8.9
//   256  1024  -> 1024    8     6.2 /  4.5      6.4 /  4.6
//   256  8192  -> 8192    4    15.9 / 11.7     15.3 / 10.1
//   420  11008 -> 4096    8    24.1 / 19.5     24.5 / 18.4
//   512  4096  -> 11008   8    32.4 / 21.7     34.6 / 21.2
//   1024 11008 -> 4096    8    37.2 / 29.5     37.1 / 29.4

// Single CTAs, tiles of 128 rows x up to 128 tokens, S of them sharing a
// tile's K: rounds of two CTAs per SM through their stages, then the stores
// of y or, before them, the sum of the partial sums over the cluster.  (One
// token, 4096 -> 22016, 8 bits: 11.9 us unsplit, 14.8 in two rounds of S = 3.)
inline double mx_split_us(int row_tiles, int tok_tiles, int tokens, int stages, int S, int x_bits, int num_sms) {
    const long long ctas = (long long)row_tiles * tok_tiles * S, slots = 2LL * num_sms;
    const double tok = tokens < 128 ? tokens / 128.0 : 1.0;
    const double stage = x_bits == 8 ? 0.35 + 0.02 * tok : 0.40 + 0.02 * tok;
    // CTAs that have an SM to themselves fetch sums twice as fast; clusters of
    // more than four are packed two to an SM well before the SMs run out.
    const bool alone = ctas <= (S > 4 ? num_sms / 2 : num_sms);
    const double end = S == 1 ? 3.94 * tok : 1.17 + (alone ? 3.19 : 6.07) * tok;
    const double rounds = (double)((ctas + slots - 1) / slots);
    return 1.33 + rounds * (((stages + S - 1) / S) * stage + end) + (rounds - 1.0) * 1.7;
}

// The split with the lowest estimate: at most 8 CTAs, two stages to each.
inline int mx_split(int row_tiles, int tok_tiles, int tokens, int stages, int x_bits, int num_sms) {
    int best = 1;
    double us = mx_split_us(row_tiles, tok_tiles, tokens, stages, 1, x_bits, num_sms);
    for (int S = 2; S <= kMxMaxSplit && 2 * S <= stages; ++S) {
        // Above 16 tokens shares of 16 to 28 rows are summed slowly: 128 tokens
        // through 4096 x 4096 in 8 bits take 8.3, 12.1 and 10.9 us with S = 4, 6, 8.
        if (tokens > 16 && S > 4 && S < 8) continue;
        const double t = mx_split_us(row_tiles, tok_tiles, tokens, stages, S, x_bits, num_sms);
        if (t < us) us = t, best = S;
    }
    return best;
}

// Tiles of the CTA-pair kernel: 256 weight rows by tile_tok tokens, a multiple
// of 32 up to 256 that splits the tokens evenly.  x_tiles: 128-row scale
// tiles that the tokens of any tile touch, counted from the tile that holds
// its first token.
struct MxPairTiles {
    int tile_tok, tok_tiles, row_tiles, x_tiles;
};

// Tiles of up to this many tokens take two of the ring stages that `stages`
// counts as one.
constexpr int kMxPairTwoBlocks = 128;

// CTA pairs, one per two SMs.
inline double mx_pair_us(const MxPairTiles &g, int stages, int x_bits, int num_sms) {
    const long long tiles = (long long)g.row_tiles * g.tok_tiles, pairs = num_sms > 1 ? num_sms / 2 : 1;
    const double n = g.tile_tok / 256.0, waves = (double)((tiles + pairs - 1) / pairs);
    const double in_stages =
        g.tile_tok <= kMxPairTwoBlocks ? ((stages + 1) / 2) * (x_bits == 8 ? 0.292 + 0.068 * n : 0.304 + 0.096 * n)
                                       : stages * (x_bits == 8 ? 0.248 + 0.032 * n : 0.278 + 0.014 * n);
    return 2.66 + 1.73 * n + 0.014 * (double)(tiles < pairs ? tiles : pairs) + waves * in_stages + (waves - 1.0) * 0.48;
}

// As few tiles of tokens as there can be, or twice or four times as many
// where the estimate is lower: smaller tiles end sooner while there are pairs
// to spare.
inline MxPairTiles mx_pair_tiles(int T, int N, int stages, int x_bits, int num_sms) {
    MxPairTiles best{};
    double us = 0.0;
    for (int more = 1; more <= 4; more *= 2) {
        MxPairTiles g;
        const long long parts = ((long long)T + 255) / 256 * more;
        g.tile_tok = (int)(((T + parts - 1) / parts + 31) / 32 * 32);
        g.tok_tiles = (int)(((long long)T + g.tile_tok - 1) / g.tile_tok);
        g.row_tiles = (int)(((long long)N + 255) / 256);
        // The first token's offset in its scale tile is a multiple of
        // gcd(tile_tok, 128).
        int step = 128;
        while (g.tile_tok % step) step /= 2;
        const int offset = g.tok_tiles > 1 ? 128 - step : 0;
        g.x_tiles = (offset + g.tile_tok + 127) / 128;
        const double t = mx_pair_us(g, stages, x_bits, num_sms);
        if (more == 1 || t < us) us = t, best = g;
    }
    return best;
}

// Which form runs: CTA pairs never for the smallest calls, whose one tile of
// 16 tokens they cannot beat.
inline bool mx_use_pairs(int T, int N, int stages, int x_bits, int num_sms) {
    if (T <= 16) return false;
    const int row_tiles = (int)(((long long)N + 127) / 128), tok_tiles = (int)(((long long)T + 127) / 128);
    if (tok_tiles > 65535) return true;  // the other form's grid has them in y
    const int S = mx_split(row_tiles, tok_tiles, T, stages, x_bits, num_sms);
    return mx_pair_us(mx_pair_tiles(T, N, stages, x_bits, num_sms), stages, x_bits, num_sms) <
           mx_split_us(row_tiles, tok_tiles, T, stages, S, x_bits, num_sms);
}

}  // namespace q4mm
