// Instantiations of the 128 x 128 tile for the gradients' products.
#include "grad_launch.hpp"

namespace gemm {
template hipError_t launch_grad_pair<128, 128, 2, 2, 2>(const GradPair&, hipStream_t, int, int, int);
}  // namespace gemm
