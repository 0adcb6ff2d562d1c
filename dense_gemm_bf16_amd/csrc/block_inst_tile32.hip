// Kernel instantiations of the staged tiles of 32 rows.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_tile<32, 128, 1, 4, 1, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
template hipError_t launch_block_tile<32, 64, 2, 2, 4, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
template hipError_t launch_block_tile<32, 32, 2, 2, 4, 4>(const BlockArgs&, int, hipStream_t,
                                                              int, int);
}  // namespace gemm
