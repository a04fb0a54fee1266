// attn_tiles4_128.cu -- the attention kernel over a 4-bit cache at head_dim 128.
#define PA_ATTN_TILES4 128
#include "attn_fwd.cu"
