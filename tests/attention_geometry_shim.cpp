// C entry points over the attention kernels' geometry header for the CPU tests.
#include "attention_geometry.h"

extern "C" {
void att_geo_few(long long tokens, int group, int seqs, int kv_heads, int width, int page, int num_sms, int *out) {
    const int nr = q4mm::few_row_tiles(tokens, group, seqs);
    const long long tiles = q4mm::few_tiles(tokens, group, nr, seqs);
    const q4mm::FewSplit f = q4mm::few_split(tiles, kv_heads, q4mm::few_keys(width, page), num_sms);
    out[0] = nr, out[1] = (int)tiles, out[2] = f.cluster, out[3] = f.parts;
}
int att_geo_many(long long tokens, int group, int seqs) { return q4mm::many_rows(tokens, group, seqs); }
int att_geo_many_split(long long rows, int tile_rows, int seqs, int kv_heads, int keys, int num_sms) {
    return q4mm::many_split(rows, tile_rows, seqs, kv_heads, keys, num_sms);
}
}
