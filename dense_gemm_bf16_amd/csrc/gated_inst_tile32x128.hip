// Instantiations of the 32 x 128 tile for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_tile<32, 128, 1, 4, 1, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int, bool, bool);
}  // namespace gemm
