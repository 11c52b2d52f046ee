// hidden weight^T with its epilogue in bfloat16: the tiles that linear_shape chooses from.
#include "linear_tile.hpp"

namespace arcs {

hipError_t launch_linear_forward_bf16(const LinearProduct& p, hipStream_t stream) {
  const bool known = launch_linear_tile<__bf16, kLinForward, 2, 4, 4, 2, 2>(p, stream) ||
                     launch_linear_tile<__bf16, kLinForward, 2, 2, 2, 2, 2>(p, stream) ||
                     launch_linear_tile<__bf16, kLinForward, 2, 2, 1, 1, 4>(p, stream) ||
                     launch_linear_tile<__bf16, kLinForward, 4, 1, 1, 1, 3>(p, stream);
  return known ? hipGetLastError() : hipErrorInvalidValue;
}

}  // namespace arcs
