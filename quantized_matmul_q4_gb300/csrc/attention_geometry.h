// How attention is split over the GPU: host code, compiled by the kernels'
// launchers and by the tests.
#pragma once

namespace q4mm {

constexpr int kFewWarps = 8;      // warps of a CTA for few rows
constexpr int kFewGroup = 16;     // tokens a warp takes at once
constexpr int kFewMaxSplit = 16;  // CTAs that share a row tile's keys (a cluster)

// CTAs of a cluster over the keys of one row tile: a power of two that gives
// the SMs two CTAs each, unless a warp would have less than two groups.
inline int few_split(long long tiles, int kv_heads, int keys, int num_sms) {
    const long long ctas = tiles * kv_heads;
    const int groups = (keys + kFewGroup - 1) / kFewGroup;
    int s = 1;
    while (s < kFewMaxSplit && ctas * s < 2LL * num_sms && groups >= 4 * s * kFewWarps) s *= 2;
    return s;
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
