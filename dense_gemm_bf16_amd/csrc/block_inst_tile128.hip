// Kernel instantiations of the 128 x 128 staged tiles.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_tile<128, 128, 2, 2, 1, 2>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
template hipError_t launch_block_tile<128, 128, 2, 2, 2, 2>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
}  // namespace gemm
