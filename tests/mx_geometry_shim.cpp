// C entry points over the MX products' geometry header for the CPU tests.
#include "mx_geometry.h"

extern "C" {
int mx_geo_split(int row_tiles, int tok_tiles, int tokens, int stages, int x_bits, int num_sms) {
    return q4mm::mx_split(row_tiles, tok_tiles, tokens, stages, x_bits, num_sms);
}
int mx_geo_use_pairs(int T, int N, int stages, int x_bits, int num_sms) {
    return q4mm::mx_use_pairs(T, N, stages, x_bits, num_sms);
}
int mx_geo_first_row(int s, int S) { return q4mm::mx_first_row(s, S); }
void mx_geo_pairs(int T, int N, int stages, int x_bits, int num_sms, int *out) {
    const q4mm::MxPairTiles g = q4mm::mx_pair_tiles(T, N, stages, x_bits, num_sms);
    out[0] = g.tile_tok, out[1] = g.tok_tiles, out[2] = g.row_tiles, out[3] = g.x_tiles;
}
}
