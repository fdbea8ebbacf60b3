// C entry points over the attention kernels' limits for the CPU tests.
#include "attention_geometry.h"

extern "C" {
int att_table_keys(int width, int page) { return q4mm::table_keys(width, page); }
// A plan whose tensor-core sums are bounded by `chain` steps (0: not).
void att_chain(long long tokens, int group, int seqs, int kv_heads, int width, int page, int chain, int num_sms, int *out) {
    const q4mm::AttentionPlan p = q4mm::attention_plan(tokens, group, seqs, kv_heads, q4mm::table_keys(width, page), false, num_sms, chain);
    out[0] = p.many, out[1] = p.split, out[2] = p.many_as_f32;
    out[3] = p.few.rows_8, out[4] = p.few.cluster, out[5] = p.few.parts, out[6] = p.few_as_f32;
}
int att_chain_of(int bf16) { return bf16 ? q4mm::kChainBf16 : q4mm::kChainF16; }
int att_tile_keys(void) { return q4mm::kManyKeys > 8 * q4mm::kFewGroup ? q4mm::kManyKeys : 8 * q4mm::kFewGroup; }
}
