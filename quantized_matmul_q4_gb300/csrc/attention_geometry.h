// How attention is split over the GPU: host code, compiled by the kernels'
// launchers and by the tests.
#pragma once

namespace q4mm {

constexpr int kFewWarps = 8;      // warps of a CTA for few rows
constexpr int kFewGroup = 16;     // tokens a warp takes at once
constexpr int kFewMaxSplit = 8;   // CTAs of a cluster that share a row tile's keys

// Row tiles of 8 that a CTA takes: two where a sequence and kv head have more than 8 rows on average.
inline int few_row_tiles(long long tokens, int group, int seqs) { return tokens * group > 8LL * seqs ? 2 : 1; }

// Tiles of 8 · nr rows, at most (see row_tile).
inline long long few_tiles(long long tokens, int group, int nr, int seqs) { return tokens * group / (8 * nr) + seqs; }

// Keys of a sequence, at most: what its table has room for (their number is the device's to know).
inline int few_keys(int width, int page) {
    const long long keys = (long long)width * page;
    return keys < 0x7FFFFFFF ? (int)keys : 0x7FFFFFFF;
}

// How a tile's keys are shared: `parts` clusters of `cluster` CTAs.
struct FewSplit {
    int cluster, parts;
};

// Enough to give the SMs two CTAs each, while each warp has a group: up to a
// cluster, and with two groups a warp several of them, joined by a second kernel.
// One row over 1000 tokens, 32 heads: 8.1 us with a group a warp, 10.0 with two.
// Over 131072, one key head: 29.7 us in 37 clusters of 8 (in 75 of 4 37.0, the join is longer; of
// clusters of 16 only 14 are resident at once).
inline FewSplit few_split(long long tiles, int kv_heads, int keys, int num_sms) {
    const long long ctas = tiles * kv_heads, groups = ((long long)keys + kFewGroup - 1) / kFewGroup;
    const long long fill = 2LL * num_sms / (ctas > 0 ? ctas : 1);
    const long long each = groups / kFewWarps < fill ? groups / kFewWarps : fill;
    int s = 1;
    while (s < kFewMaxSplit && 2 * s <= each) s *= 2;
    const long long both = groups / (2 * kFewWarps) < fill ? groups / (2 * kFewWarps) : fill;
    const int parts = (int)(both / s);
    return FewSplit{s, s == kFewMaxSplit && parts > 1 ? parts : 1};
}

constexpr int kManyKeys = 128;   // keys of a tile on tcgen05
constexpr int kManyMaxSplit = 8;  // CTAs that share a row tile's keys there

// Rows of a sequence and kv head, on average, from which tiles of 128 on the
// tensor cores are faster.
inline bool many_rows(long long tokens, int group, int seqs) { return tokens * group > 32LL * (seqs > 0 ? seqs : 1); }

// CTAs of a cluster over the keys: while one CTA per SM is not passed, and
// each has two tiles of keys.
inline int many_split(long long rows, int tile_rows, int seqs, int kv_heads, int keys, int num_sms) {
    const long long whole = rows / tile_rows, tiles = whole > seqs ? whole : seqs;
    const int key_tiles = (keys + kManyKeys - 1) / kManyKeys;
    int s = 1;
    while (s < kManyMaxSplit && tiles * kv_heads * s * 2 <= num_sms && key_tiles >= 4 * s) s *= 2;
    return s;
}

}  // namespace q4mm
