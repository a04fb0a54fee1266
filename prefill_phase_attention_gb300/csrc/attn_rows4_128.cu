// attn_rows4_128.cu -- the row kernel over the 4-bit cache at head_dim 128.
#include "attn_rows4.cuh"

namespace pa {

template <>
cudaError_t launch_attn_rows4_d<128>(const Rows4Params& p, int row_tiles, int grid, cudaStream_t st) {
    switch (p.cache.groups) {
        case 1: return row_tiles == 1 ? rows4::launch<128, 1, 1>(p, grid, st) : rows4::launch<128, 1, 2>(p, grid, st);
        case 2: return row_tiles == 1 ? rows4::launch<128, 2, 1>(p, grid, st) : rows4::launch<128, 2, 2>(p, grid, st);
        default: return row_tiles == 1 ? rows4::launch<128, 4, 1>(p, grid, st) : rows4::launch<128, 4, 2>(p, grid, st);
    }
}

}  // namespace pa
