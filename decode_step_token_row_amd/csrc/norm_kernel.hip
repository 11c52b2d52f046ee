// The global norm of many gradients, and clipping to it.
//
//   norm = sqrt(sum of x^2 over all tensors),  y = x * max_norm / norm where norm > max_norm
//
// The plan lists pieces of tensors, 32 bytes each, so that a workgroup knows its
// work from one load.  A first launch leaves each workgroup's sum of squares in the
// workspace, in double precision (no square of a float32 overflows there, and the order of
// the sums does not show in the norm's 24 bits); a second one adds the workgroups' sums up, every
// workgroup by itself and in the same order, and writes the scaled gradients.  It goes through
// the plan from its end, where the first launch has left what the cache still holds.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "linear_device.hpp"

namespace arcs {

constexpr int kNormThreads = 256;

template <typename T>
__device__ __forceinline__ double piece_squares(const T* p, int count) {
  constexpr int kEach = 16 / sizeof(T);
  const int whole = count / kEach;
  double s = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < whole; i += kNormThreads) {
    float v[kEach];
    load_some<T, kEach>(p + (int64_t)i * kEach, kEach, v);
#pragma unroll
    for (int e = 0; e < kEach; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
  }
  const int i = whole * kEach + threadIdx.x;
  if (i < count) {
    const double x = (double)widen(p[i]);
    s = __builtin_fma(x, x, s);
  }
  return s;
}

// The workgroup's sum of a double of every thread, in every thread.
__device__ __forceinline__ double group_sum(double s) {
  __shared__ double waves[kNormThreads / 64];
  s = dpp_wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kNormThreads / 64; ++w) s += waves[w];
  return s;
}

__global__ __launch_bounds__(kNormThreads) void norm_squares_kernel(NormArgs a) {
  double s = 0.0;
  for (int64_t i = blockIdx.x; i < a.pieces; i += gridDim.x) {
    const NormPiece p = a.plan[i];
    s += p.bf16 ? piece_squares((const __bf16*)p.from, p.count) : piece_squares((const float*)p.from, p.count);
  }
  s = group_sum(s);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const NormArgs& a) {
  double s = 0.0;
  for (int i = threadIdx.x; i < a.groups; i += kNormThreads) s += a.sums[i];
  return __builtin_sqrt(group_sum(s));
}

__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs a) {
  const double norm = norm_of(a);
  if (threadIdx.x == 0) *a.out_norm = (float)norm;
}

template <typename T, typename O>
__device__ __forceinline__ void piece_scale(const T* p, O* to, int count, double scale) {
  constexpr int kEach = 16 / sizeof(T);
  const int whole = count / kEach;
#pragma unroll 4
  for (int i = threadIdx.x; i < whole; i += kNormThreads) {
    float v[kEach];
    load_some<T, kEach>(p + (int64_t)i * kEach, kEach, v);
#pragma unroll
    for (int e = 0; e < kEach; ++e) v[e] = (float)((double)v[e] * scale);
    store_some<O, kEach>(to + (int64_t)i * kEach, kEach, v);
  }
  const int i = whole * kEach + threadIdx.x;
  if (i < count) to[i] = (O)(float)((double)widen(p[i]) * scale);
}

__global__ __launch_bounds__(kNormThreads) void clip_kernel(NormArgs a) {
  const double norm = norm_of(a);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.out_norm = (float)norm;
  const bool clipped = norm > a.max_norm && norm < __builtin_inf();
  const double scale = clipped ? a.max_norm / norm : 1.0;
  for (int64_t i = a.pieces - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const NormPiece p = a.plan[i];
    if (p.to == nullptr || (!clipped && p.from == p.to)) continue;
    if (p.bf16) {
      if (p.to_bf16) piece_scale((const __bf16*)p.from, (__bf16*)p.to, p.count, scale);
      else piece_scale((const __bf16*)p.from, (float*)p.to, p.count, scale);
    } else {
      if (p.to_bf16) piece_scale((const float*)p.from, (__bf16*)p.to, p.count, scale);
      else piece_scale((const float*)p.from, (float*)p.to, p.count, scale);
    }
  }
}

hipError_t launch_norm(NormArgs a, bool clip, hipStream_t stream) {
  a.groups = norm_groups(a.pieces);
  const int64_t blocks = a.groups;
  if (blocks > 0) hipLaunchKernelGGL(norm_squares_kernel, dim3((unsigned)blocks), dim3(kNormThreads), 0, stream, a);
  if (clip && blocks > 0) hipLaunchKernelGGL(clip_kernel, dim3((unsigned)blocks), dim3(kNormThreads), 0, stream, a);
  else hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kNormThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace arcs
