// attn_two_128.cu -- the variant of the attention kernel with cached keys in two terms at
// head_dim 128.
#define PA_ATTN_TWO 128
#include "attn_fwd.cu"
