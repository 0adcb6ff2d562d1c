// Instantiations of the 256 x 192 tile for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_tile<256, 192, 2, 4, 1, 2>(const BlockArgs&, int, hipStream_t,
                                                              int, int, bool, bool);
}  // namespace gemm
