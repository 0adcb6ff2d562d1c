// Kernel instantiations of the 256 x 128 staged tile.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_tile<256, 128, 4, 2, 1, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
}  // namespace gemm
