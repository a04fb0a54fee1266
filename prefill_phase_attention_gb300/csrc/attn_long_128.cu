// attn_long_128.cu -- the long-context variant of the attention kernel (sink
// tokens, a shared prefix, split units) at head_dim 128.
#define PA_ATTN_LONG 128
#include "attn_fwd.cu"
