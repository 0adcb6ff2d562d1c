// Kernel instantiations of the 256 x 256 staged tile.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_tile<256, 256, 2, 4, 1, 2>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
}  // namespace gemm
