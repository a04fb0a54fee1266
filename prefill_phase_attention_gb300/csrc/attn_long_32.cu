// attn_long_32.cu -- the long-context variant of the attention kernel (sink
// tokens, a shared prefix, split units) at head_dim 32.
#define PA_ATTN_LONG 32
#include "attn_fwd.cu"
