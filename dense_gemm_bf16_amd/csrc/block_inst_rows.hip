// Kernel instantiations of the register-streamed shapes for few rows.
#include "block_launch.hpp"
namespace gemm {
template hipError_t launch_block_row<1, 1, 4, 4>(const BlockArgs&, int, hipStream_t, int, int);
template hipError_t launch_block_row<2, 2, 4, 2>(const BlockArgs&, int, hipStream_t, int, int);
template hipError_t launch_block_row<4, 2, 4, 2>(const BlockArgs&, int, hipStream_t, int, int);
}  // namespace gemm
