// attn_tiles4_64.cu -- the attention kernel over a 4-bit cache at head_dim 64.
#define PA_ATTN_TILES4 64
#include "attn_fwd.cu"
