// attn_tiles4_32.cu -- the attention kernel over a 4-bit cache at head_dim 32.
#define PA_ATTN_TILES4 32
#include "attn_fwd.cu"
