// Instantiations of the register-streamed shape for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
template hipError_t launch_gated_row<1, 1, 8, 4>(const BlockArgs&, int, hipStream_t, int, int,
                                                 bool, bool);
}  // namespace gemm
