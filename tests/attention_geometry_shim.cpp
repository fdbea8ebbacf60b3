// C entry points over the attention kernels' geometry header for the CPU tests.
#include "attention_geometry.h"

extern "C" {
void att_geo(long long tokens, int group, int seqs, int kv_heads, int width, int page, int f32, int num_sms, int *out) {
    const q4mm::AttentionPlan p = q4mm::attention_plan(tokens, group, seqs, kv_heads, q4mm::table_keys(width, page), f32, num_sms);
    out[0] = p.few.rows_8, out[1] = (int)q4mm::few_tiles(tokens, group, p.few.rows_8, seqs), out[2] = p.few.cluster, out[3] = p.few.parts;
    out[4] = p.many, out[5] = p.split;
}
}
