// Instantiations of the 32 x 64 tile with 4 wave groups along K for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_tile<32, 64, 2, 2, 4, 3>(const BlockArgs&, int, hipStream_t,
                                                              int, int, bool, bool);
}  // namespace gemm
