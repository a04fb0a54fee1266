// attn_rows4.cu -- the row kernel over the 4-bit cache at head_dim 32 and 64, and its launch.
#include "attn_rows4.cuh"

namespace pa {

template <>
cudaError_t launch_attn_rows4_d<64>(const Rows4Params& p, int row_tiles, int grid, cudaStream_t st) {
    if (p.cache.groups == 1) return row_tiles == 1 ? rows4::launch<64, 1, 1>(p, grid, st) : rows4::launch<64, 1, 2>(p, grid, st);
    return row_tiles == 1 ? rows4::launch<64, 2, 1>(p, grid, st) : rows4::launch<64, 2, 2>(p, grid, st);
}

cudaError_t launch_attn_rows4(const Rows4Params& p, int head_dim, int row_tiles, int grid, cudaStream_t st) {
    switch (head_dim) {
        case 32: return row_tiles == 1 ? rows4::launch<32, 1, 1>(p, grid, st) : rows4::launch<32, 1, 2>(p, grid, st);
        case 64: return launch_attn_rows4_d<64>(p, row_tiles, grid, st);
        default: return launch_attn_rows4_d<128>(p, row_tiles, grid, st);
    }
}

}  // namespace pa
