// Instantiations of the register-streamed shapes for integer and gated products.
#include "gated_launch.hpp"

namespace gemm {
#define INSTANTIATE(NAME, A, B, C, D, E)                                                            \
  template hipError_t launch_gated_row<A, B, C, D, E>(const BlockArgs&, int, hipStream_t, int, int, \
                                                   bool, bool);
GATED_ROWS(INSTANTIATE)
#undef INSTANTIATE
}  // namespace gemm
