// attn_long_64.cu -- the long-context variant of the attention kernel (sink
// tokens, a shared prefix, split units) at head_dim 64.
#define PA_ATTN_LONG 64
#include "attn_fwd.cu"
