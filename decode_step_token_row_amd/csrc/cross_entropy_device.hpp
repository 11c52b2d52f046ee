// Device-side pieces the linear cross entropy's kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cross_entropy.hpp"
#include "device_common.hpp"

namespace arcs {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float finite_or_zero(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// The products, C[m, n] = sum_k A[m, k] B[n, k]:
//   STATS    m: vocabulary, n: listed rows, k: D    maximum and sum per slice
//   DS       the same                               dz / gmax of the piece
//   DHIDDEN  m: D, n: listed rows, k: the piece     adds to the split's slab
//   DWEIGHT  m: D, n: the piece, k: listed rows     rows of dweight
enum CeMode { kCeStats, kCeDs, kCeDhidden, kCeDweight };

struct CePiece {
  int64_t v0, len;  // the piece of the vocabulary
  int first;        // DHIDDEN: the slab holds nothing yet
  int gather;       // matrix kernels: hidden states are read through the row list
  int direct;       // STATS of few rows: no row list, every row is computed
};

// 0: the row counts, -1: it is masked, otherwise its status code.
__device__ __forceinline__ int ce_row_kind(const CeArgs& a, int64_t n, int32_t& target, float& T) {
  target = a.targets[n];
  T = a.temperature ? a.temperature[n] : 1.0f;
  if (target == a.ignore_index) return -1;
  if (target < 0 || (int64_t)target >= a.V) return ARCS_ROW_BAD_TARGET;
  if (!(T > 0.0f) || T == __builtin_inff()) return ARCS_ROW_BAD_TEMPERATURE;
  return 0;
}

// The record of a listed row in the backward pass.
__device__ __forceinline__ CeRow ce_row(const CeArgs& a, int64_t n, int32_t target, float T, float gmax) {
  CeRow r = {};
  r.row = (int32_t)n;
  r.target = target;
  r.a = kLog2e / T;
  r.c = (a.grad_loss[n] / T) / gmax;
  // lse comes rounded to float32, so every probability is off by up to 2^-24 |lse|; a
  // float32 product here would add as much again
  const double lse2 = (double)a.lse[n] * 1.4426950408889634074;
  r.lse2 = (float)lse2;
  r.rest = fabsf(r.lse2) < __builtin_inff() ? exp2f((float)((double)r.lse2 - lse2)) : 1.0f;
  return r;
}

// cross_entropy_kernel.hip
void launch_cross_entropy_prep(const CeArgs& a, bool backward, hipStream_t stream);
void launch_cross_entropy_combine(const CeArgs& a, bool direct, hipStream_t stream);
void launch_cross_entropy_dhidden(const CeArgs& a, bool bf16, hipStream_t stream);
// cross_entropy_mfma.hip
bool cross_entropy_matrix_path(const CeArgs& a, int dtype);
hipError_t launch_cross_entropy_matrix(const CeArgs& a, int dtype, bool backward, hipStream_t stream);

}  // namespace arcs
