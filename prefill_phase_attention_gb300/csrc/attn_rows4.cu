// attn_rows4.cu -- the row kernel over the 4-bit cache at head_dim 32 and 64, and its launch.
#include "attn_rows4.cuh"

namespace pa {

cudaError_t launch_attn_rows4(const Rows4Params& p, int head_dim, int grid, cudaStream_t st) {
    if (head_dim == 32) return rows4::launch<32, 1>(p, grid, st);
    if (head_dim == 64) return p.cache.groups == 1 ? rows4::launch<64, 1>(p, grid, st) : rows4::launch<64, 2>(p, grid, st);
    return launch_attn_rows4_128(p, grid, st);
}

}  // namespace pa
