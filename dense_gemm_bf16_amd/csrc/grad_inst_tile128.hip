// Instantiations of the 128 x 128 tile for the gradients' products.
#include "grad_launch.hpp"

namespace gemm {
template hipError_t launch_grad_tile<128, 128, 2, 2, 2>(const BlockArgs&, int, hipStream_t, int, int, int);
}  // namespace gemm
