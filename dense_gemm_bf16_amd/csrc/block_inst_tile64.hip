// Kernel instantiations of the staged tiles of 64 rows.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_tile<64, 128, 2, 2, 2, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
template hipError_t launch_block_tile<64, 64, 2, 2, 1, 4>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
template hipError_t launch_block_tile<64, 64, 2, 2, 2, 4>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
}  // namespace gemm
