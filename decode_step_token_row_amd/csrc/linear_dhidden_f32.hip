// dz weight in float32: the tiles that linear_shape chooses from.
#include "linear_tile.hpp"

namespace arcs {

hipError_t launch_linear_dhidden_f32(const LinearProduct& p, hipStream_t stream) {
  const bool known = launch_linear_tile<float, kLinDhidden, 2, 2, 2, 1, 2>(p, stream) ||
                     launch_linear_tile<float, kLinDhidden, 2, 2, 1, 1, 4>(p, stream) ||
                     launch_linear_tile<float, kLinDhidden, 4, 1, 1, 1, 3>(p, stream);
  return known ? hipGetLastError() : hipErrorInvalidValue;
}

}  // namespace arcs
