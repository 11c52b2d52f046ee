// Host and device declarations of the linear layer's kernels.
//
//   z = hidden weight^T + bias,  out = residual + act(z)             [N, V]
//   dz = grad_out * act'(z),  dhidden = dz weight,  dweight = dz^T hidden,  dbias = sum_n dz
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "arcs.h"
#include "linear_shape.hpp"

namespace arcs {

struct LinearArgs {
  const void* hidden;    // [N, hidden_stride] of T
  int64_t hidden_stride;
  const void* weight;    // [V, weight_stride] of T
  int64_t weight_stride;
  int64_t N, V, D;
  int act;
  float cap, inv_cap;  // SOFTCAP: 1 / cap
  // forward
  const void* bias;      // [V] of T, or NULL
  const void* residual;  // [N, residual_stride] of T, or NULL
  int64_t residual_stride;
  void* out;             // [N, out_stride]
  int64_t out_stride;
  int out_bf16;
  void* out_pre;         // [N, V] of T, dense, or NULL
  // backward
  const void* pre;       // [N, V] of T, dense (NULL without an activation)
  const void* grad;      // [N, grad_stride]
  int64_t grad_stride;
  int grad_bf16;
  void* out_dhidden;     // [N, D] of T, dense, or NULL
  void* out_dweight;     // [V, D] of T, dense, or NULL
  void* out_dbias;       // [V] of T, or NULL
  char* workspace;
};

// The workspace's parts, in bytes from its start.
struct LinearPlan {
  size_t hidden, weight;  // rows off the 16-byte grid: copies on it, padded with zeros
  size_t dz;              // backward: [N][ldz] of T
  size_t dbias;           // backward: [chunks][V] float
  size_t slab;            // parts of shared tiles
  size_t total;
  int64_t ldd, ldz;       // of the copies and of dz, in elements
  int64_t chunk_rows;     // rows of a dbias chunk
};
LinearPlan linear_plan(int64_t N, int64_t V, int64_t D, int dtype, bool aligned, bool backward);

// Whether rows of T are on the 16-byte grid and a tile's rows within 32-bit offsets.
bool linear_rows_aligned(const void* p, int64_t stride, int64_t columns, int dtype);

hipError_t launch_linear(LinearArgs a, int dtype, bool aligned, hipStream_t stream);
hipError_t launch_linear_backward(LinearArgs a, int dtype, bool aligned, hipStream_t stream);

// One product on the tile kernels (linear_tile.hpp; one source for each mode and type).
struct LinearProduct {
  const void *a, *b;
  int64_t lda, ldb;  // elements between rows
  int64_t M, N, K;
  void* out;         // [N, ldo]
  int64_t ldo;
  int out_bf16;
  float* slab;
  LinearShape shape;
  // the epilogue (FORWARD)
  const void* bias;
  const void* residual;
  int64_t ldr;
  void* pre;
  int64_t ldp;
  int act;
  float cap, inv_cap;  // SOFTCAP: 1 / cap
};
hipError_t launch_linear_forward_bf16(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_forward_f32(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_dhidden_bf16(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_dhidden_f32(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_dweight_bf16(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_dweight_f32(const LinearProduct& p, hipStream_t stream);
hipError_t launch_linear_product(const LinearProduct& p, int mode, int dtype, hipStream_t stream);
// linear_kernel.hip: at most kLinearFewRows rows of the forward pass.
constexpr int64_t kLinearFewRows = 16;

}  // namespace arcs
