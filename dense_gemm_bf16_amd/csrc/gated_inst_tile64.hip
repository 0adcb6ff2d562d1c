// Instantiations of the 64 x 64 tile for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_tile<64, 64, 2, 2, 1, 4>(const BlockArgs&, int, hipStream_t,
                                                              int, int, bool, bool);
}  // namespace gemm
