// attn_two_64.cu -- the variant of the attention kernel with cached keys in two terms at
// head_dim 64.
#define PA_ATTN_TWO 64
#include "attn_fwd.cu"
