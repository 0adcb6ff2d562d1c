// Instantiations of the 256 x 128 tile for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_tile<256, 128, 4, 2, 1, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int, bool, bool);
}  // namespace gemm
