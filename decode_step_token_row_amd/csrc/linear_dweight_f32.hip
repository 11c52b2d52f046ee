// dz^T hidden in float32: the tiles that linear_shape chooses from.
#include "linear_tile.hpp"

namespace arcs {

hipError_t launch_linear_dweight_f32(const LinearProduct& p, hipStream_t stream) {
  const bool known = launch_linear_tile<float, kLinDweight, 2, 2, 2, 1, 2>(p, stream) ||
                     launch_linear_tile<float, kLinDweight, 2, 2, 1, 1, 4>(p, stream);
  return known ? hipGetLastError() : hipErrorInvalidValue;
}

}  // namespace arcs
