// attn_rows4_128.cu -- the row kernel over the 4-bit cache at head_dim 128.
#include "attn_rows4.cuh"

namespace pa {

cudaError_t launch_attn_rows4_128(const Rows4Params& p, int grid, cudaStream_t st) {
    switch (p.cache.groups) {
        case 1: return rows4::launch<128, 1>(p, grid, st);
        case 2: return rows4::launch<128, 2>(p, grid, st);
        default: return rows4::launch<128, 4>(p, grid, st);
    }
}

}  // namespace pa
