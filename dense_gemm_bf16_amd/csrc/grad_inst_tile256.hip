// Instantiations of the 256 x 256 tile for the gradients' products.
#include "grad_launch.hpp"

namespace gemm {
template hipError_t launch_grad_pair<256, 256, 2, 4, 2>(const GradPair&, hipStream_t, int, int, int);
}  // namespace gemm
