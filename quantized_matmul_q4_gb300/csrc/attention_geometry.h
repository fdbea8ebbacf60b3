// How attention is split over the GPU: host code, compiled by the kernels'
// launchers and by the tests.
#pragma once

namespace q4mm {

constexpr int kMaxSplit = 8;  // CTAs of a cluster that share a row tile's keys (of 16 only 14 are resident)

// Clusters of s CTAs that are resident at once with one CTA an SM, and with
// two, on 152 SMs: the GPU's processing clusters have 16 to 20 SMs, so that larger
// clusters leave some over, most of all those of 7, which are not used.
constexpr int kResident[2][kMaxSplit + 1] = {{0, 152, 76, 46, 36, 28, 23, 15, 15}, {0, 304, 152, 97, 74, 58, 46, 38, 36}};
inline long long resident(int cluster, bool two, int num_sms) {
    const long long n = (long long)kResident[two][cluster] * num_sms / 152;
    return n > 0 ? n : 1;
}

// Row tiles where the rows are spread evenly over the sequences that can have any.
inline long long even_tiles(long long tokens, int group, int tile_rows, int seqs) {
    const long long some = tokens < seqs ? tokens : seqs, each = (long long)tile_rows * some;
    return some * ((tokens * group + each - 1) / each);
}

constexpr int kFewWarps = 8;      // warps of a CTA for few rows
constexpr int kFewGroup = 16;     // tokens a warp takes at once

// Tiles of 8 · nr rows, at most (see row_tile).
inline long long few_tiles(long long tokens, int group, int nr, int seqs) { return tokens * group / (8 * nr) + seqs; }

// Keys of a sequence, at most, on the host (their number is the device's to
// know) and on the device: what its table has room for, and a tile's keys and a few
// groups more than which can still be numbered in 32 bits.
constexpr int kMaxKeys = 0x7FFFFF00;
constexpr int table_keys(int width, int page) {
    const long long keys = (long long)width * page;
    return keys < kMaxKeys ? (int)keys : kMaxKeys;
}

constexpr int kPartedTiles = 64;  // tiles of 8 rows and key heads, at most, that are shared by several clusters

// How few rows are split: tiles of 8 · rows_8 rows, the keys of each shared by
// `parts` clusters of `cluster` CTAs, whose sums a second kernel joins.
struct FewSplit {
    int rows_8, cluster, parts;
};

// Microseconds of a split. A CTA is paid for by the rounds of 8 groups that
// its warps take: 4 and 1.04 a round alone on its SM, 4.9 and 1.34 for two there, where
// the registers leave room for two (8 rows, 16-bit), and 5 and 1.08 with 16
// rows; fp32 takes 4.3 and 1.2, 5.4 and 1.48.  A cluster costs 1.5, the second
// kernel 2.4 and 0.3 a part.  These were fitted to 9000 measurements, of 1 to
// 64 sequences, 60 to 40000 keys, 8 to 24 rows: the split of least cost takes
// 1.1% longer than the best of those measured on average, 16% at most (one that
// fills the SMs' places twice with clusters of 1, 2, 4 or 8 14% and 129%).  8 sequences
// with 8 heads over 8000 keys, whole, in clusters of 2, 4 and 8: 71.6, 49.5, 30.6, 38.1 us;
// 20 with 5 over 1000, 7 rows, by tiles of 8 and of 16: whole 17.4 and 15.9, in
// clusters of 2 13.7 and 21.8.
inline double few_cost(long long tiles, int kv_heads, long long groups, const FewSplit &f, bool f32, int num_sms) {
    const long long clusters = tiles * kv_heads * f.parts, shares = (long long)kFewWarps * f.cluster * f.parts;
    const double rounds = (double)((groups + shares - 1) / shares);
    const double more = (f.cluster > 1 ? 1.5 : 0) + (f.parts > 1 ? 2.4 + 0.3 * f.parts : 0);
    const long long one = resident(f.cluster, false, num_sms);
    if (f.rows_8 == 1 && !f32) {
        const long long two = resident(f.cluster, true, num_sms), rest = clusters % two;
        const double alone = 4 + 1.04 * rounds, pair = 4.9 + 1.34 * rounds;
        return more + (double)(clusters / two) * pair + (rest == 0 ? 0 : rest <= one ? alone : pair);
    }
    const double each = !f32 ? 5 + 1.08 * rounds : f.rows_8 == 1 ? 4.3 + 1.2 * rounds : 5.4 + 1.48 * rounds;
    return more + (double)((clusters + one - 1) / one) * each;
}

// Steps of 16 keys that a sum in the tensor cores has at most (0: any number).  Each
// drops what falls below the sum's last bit, 1.7e-8 of it on average, so that 4096 leave 7e-5, a
// third of half a step of fp16; bf16 has eight times that.  (fp32 sums are taken out
// every few steps.)
constexpr int kChainF16 = 4096, kChainBf16 = 8 * kChainF16;
inline bool few_chain_passes(int keys, const FewSplit &f, int chain) {
    const long long groups = ((long long)keys + kFewGroup - 1) / kFewGroup;
    return chain && groups > (long long)chain * kFewWarps * f.cluster * f.parts;
}

// The split of least cost, as if the rows were spread evenly over the sequences and all of the table were keys, of those
// whose sums have no more steps than `chain`; least stays below 0 where there is none.
inline FewSplit few_split(long long tokens, int group, int seqs, int kv_heads, int keys, bool f32, int num_sms,
                          double &least, int chain = 0) {
    const long long groups = ((long long)keys + kFewGroup - 1) / kFewGroup;
    FewSplit best = {1, 1, 1};
    least = -1;
    const auto consider = [&](long long tiles, const FewSplit &f) {
        if (few_chain_passes(keys, f, chain)) return;
        const double c = few_cost(tiles, kv_heads, groups, f, f32, num_sms);
        if (least < 0 || c < least) best = f, least = c;
    };
    for (int nr = 1; nr <= (tokens * group > 8LL * seqs ? 2 : 1); ++nr) {
        const long long tiles = even_tiles(tokens, group, 8 * nr, seqs);
        for (int s = 1; s <= kMaxSplit; ++s)
            if (s != 7) consider(tiles, {nr, s, 1});
        // As many parts as are resident, alone on an SM or by twos; a workspace has room for all tiles there may be.
        for (int two = 0; two < 2 && few_tiles(tokens, group, 1, seqs) * kv_heads < kPartedTiles; ++two) {
            const long long parts = resident(kMaxSplit, two, num_sms) / (tiles * kv_heads);
            if (parts > 1 && parts * kMaxSplit * kFewWarps <= groups) consider(tiles, {nr, kMaxSplit, (int)parts});
        }
    }
    return best;
}

constexpr int kManyKeys = 128;  // keys of a tile on tcgen05

// CTAs of a cluster that share a tile's keys there, by the same kind of cost:
// 8 us and 2.2 a tile of keys and pair of row tiles, 5.4 and 3.0 for fp32's
// tile, 2.6 for a cluster.  Fitted to 2600 measurements (1 and 4 sequences, 34 to 3000
// rows, 400 to 30000 keys); it takes 1.1% longer than their best on average.
inline int many_split(long long tokens, int group, int tile_rows, int seqs, int kv_heads, int keys, bool f32, int num_sms,
                      double &least, int chain = 0) {
    const long long clusters = even_tiles(tokens, group, tile_rows, seqs) * kv_heads;
    const int tiles = (int)(((long long)keys + kManyKeys - 1) / kManyKeys);
    int best = 1;
    least = -1;
    for (int s = 1; s <= kMaxSplit; ++s) {
        if (s == 7) continue;
        const long long n = resident(s, false, num_sms);
        const double waves = clusters <= 3 * n ? (double)((clusters + n - 1) / n) : (double)clusters / n + 0.5;
        const int each = (tiles + s - 1) / s;
        if (chain && each > chain / (kManyKeys / 16)) continue;
        const double c = 3 + waves * ((f32 ? 5.4 + 3.0 * each : 8 + 2.2 * each) + (s > 1 ? 2.6 : 0));
        if (least < 0 || c < least) best = s, least = c;
    }
    return best;
}

// How a call is made: by tiles of 128 rows on the tensor cores (`many`, with
// clusters of `split`) or by the kernel for few rows, whichever costs less.
// (Of 375 calls measured both ways it takes 0.2% longer than the faster on average, 57%
// at most.  By rows alone, more than 32 a sequence and head, it took up to twice as
// long: one sequence with 2 heads, 400 rows each, over 500, 2600 and 8100 keys takes
// 17.0, 22.7 and 35.7 us on tcgen05, 8.5, 18.2 and 41.3 as few rows; 4 sequences with 8
// heads over 2500 keys with 32 rows 23.2 and 19.0, with 120 24.7 and 54.0.)
struct AttentionPlan {
    bool many;
    int split;
    FewSplit few;
    bool few_as_f32, many_as_f32;  // 16-bit rows by the form for fp32, whose sums may have any length
};

inline AttentionPlan attention_plan(long long tokens, int group, int seqs, int kv_heads, int keys, bool f32,
                                    int num_sms, int chain = 0) {
    double few = 0, many = 0;
    AttentionPlan p;
    p.few = few_split(tokens, group, seqs, kv_heads, keys, f32, num_sms, few, chain);
    p.few_as_f32 = few < 0;
    if (p.few_as_f32) p.few = few_split(tokens, group, seqs, kv_heads, keys, true, num_sms, few);
    p.split = many_split(tokens, group, f32 ? 128 : 256, seqs, kv_heads, keys, f32, num_sms, many, chain);
    p.many_as_f32 = many < 0;
    if (p.many_as_f32) p.split = many_split(tokens, group, 128, seqs, kv_heads, keys, true, num_sms, many);
    p.many = many < few;
    return p;
}

}  // namespace q4mm
