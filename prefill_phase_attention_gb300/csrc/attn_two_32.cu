// attn_two_32.cu -- the variant of the attention kernel with cached keys in two terms at
// head_dim 32.
#define PA_ATTN_TWO 32
#include "attn_fwd.cu"
