// What the tile kernels on the matrix instructions share: the order of tiles, and
// where a lane's 16 bytes of a load into LDS come from.
//
// A tile of an operand is 128 bytes of k.  Loads write LDS in lane order, so bank
// conflicts are avoided by permuting the lanes' global addresses:
//   rows along k:      a row's 128 bytes are 8 chunks, chunk c of row r at c ^ (r / 2 % 8);
//   rows along m or n: a row's 32-byte chunks, chunk q of row k at q ^ 2 (k % 4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace arcs {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 uniform4(u32x4 d) {
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = __builtin_amdgcn_readfirstlane(d[e]);
  return d;
}

// Tile `id` of mt x nt: bands of eight along m, in a band m first.
__device__ __forceinline__ void tile_place(int id, int mt, int nt, int64_t& m, int64_t& n) {
  const int band = id / (8 * nt), in = id - band * 8 * nt, high = mt - band * 8 < 8 ? mt - band * 8 : 8;
  m = band * 8 + in % high;
  n = in / high;
}
__device__ __forceinline__ int tile_index(int m, int n, int mt, int nt) {
  const int band = m / 8, high = mt - band * 8 < 8 ? mt - band * 8 : 8;
  return band * 8 * nt + n * high + m - band * 8;
}

// Where a lane's 16 bytes of load `inst` lie in its tile: row and element in the row.
template <typename T, int W>
__device__ __forceinline__ void outer_place(int inst, int lane, int& k, int& col) {
  constexpr int kLanes = W * (int)sizeof(T) / 16;
  k = inst * (64 / kLanes) + lane / kLanes;
  const int p = lane % kLanes;
  const int turn = W >= 128 ? (k & 3) << 1 : W == 64 ? ((k >> 1) & 1) << 1 : 0;
  col = sizeof(T) == 2 ? ((p >> 1) ^ turn) * 16 + (p & 1) * 8 : p * 4;
}
template <typename T>
__device__ __forceinline__ void inner_place(int inst, int lane, int& r, int& k) {
  r = inst * 8 + (lane >> 3);
  k = ((lane & 7) ^ ((r >> 1) & 7)) * (16 / (int)sizeof(T));
}

}  // namespace arcs
