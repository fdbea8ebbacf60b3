// How attention is split over the GPU: host code, compiled by the kernels'
// launchers and by the tests.
#pragma once

namespace q4mm {

constexpr int kFewWarps = 8;      // warps of a CTA for few rows
constexpr int kFewGroup = 16;     // tokens a warp takes at once
#ifndef PROBE_MAX
#define PROBE_MAX 8
#define PROBE_PART 4
#define PROBE_LEAST 2
#endif
constexpr int kFewMaxSplit = PROBE_MAX;  // CTAs of a cluster that share a row tile's keys
constexpr int kFewPartSplit = PROBE_PART;  // and of each, where there are several clusters

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

// Enough to give the SMs two CTAs each, unless a warp would have less than
// kFewLeast groups; beyond a cluster's 16, parts joined by a second kernel.
constexpr int kFewLeast = PROBE_LEAST;
inline FewSplit few_split(long long tiles, int kv_heads, int keys, int num_sms) {
    const long long ctas = tiles * kv_heads, groups = ((long long)keys + kFewGroup - 1) / kFewGroup;
    long long want = 2LL * num_sms / (ctas > 0 ? ctas : 1);
    const long long most = groups / (kFewLeast * kFewWarps);
    if (want > most) want = most;
    const int most_cta = want > kFewMaxSplit ? kFewPartSplit : kFewMaxSplit;
    int s = 1;
    while (s < most_cta && 2 * s <= want) s *= 2;
    const int parts = want > kFewMaxSplit ? (int)(want / s) : 1;
    return FewSplit{s, parts > 1 ? parts : 1};
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
