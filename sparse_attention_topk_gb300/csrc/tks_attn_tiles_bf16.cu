// The tiles kernel over a bfloat16 cache (a translation unit of its own, so that the two compile
// side by side).
#define TKS_TILES_BF16 1
#include "tks_attn_tiles.cu"
