// Kernel instantiation of the register-streamed shape for few rows.
#include "block_launch.hpp"

namespace gemm {
template hipError_t launch_block_row<1, 1, 8, 4>(const BlockArgs&, int, hipStream_t, int, int);
}  // namespace gemm
