// C entry points over the attention kernels' limits for the CPU tests.
#include "attention_geometry.h"

extern "C" {
int att_table_keys(int width, int page) { return q4mm::table_keys(width, page); }
int att_tile_keys(void) { return q4mm::kManyKeys > 8 * q4mm::kFewGroup ? q4mm::kManyKeys : 8 * q4mm::kFewGroup; }
}
