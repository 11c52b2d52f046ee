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
//
// Memory bounds it: 927 M bfloat16 gradients to float32 take 345 us (5.4 TB/s) and 1,220 us (5.6 GB
// read and written, 4.6 TB/s; a copy 4.8).  The gradients have to be read twice where they do not stay in
// the cache.  12 tensors of 1.3 M elements take 2.7 and 3.9 us, 1,500 of 5.7 M float32 5.9 and 9.0: two
// launches, and the plan, the data and the sums one after the other.  Accesses through generic pointers
// and sums read one by one cost 3 us more, a clipping kernel of 96 registers 2.  Stores that
// pass the cache by: norm 296 us, clipping 1,312.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "linear_device.hpp"

namespace arcs {

constexpr int kNormThreads = 256;

// A thread's part of a piece as it is in memory: up to four times 16 bytes, one workgroup's width
// apart, and one of the elements behind the last 16 bytes.
struct PieceData {
  u32x4 x[4];
  float rest;
};
template <typename T>
struct PieceShape {
  static constexpr int kEach = 16 / sizeof(T), kLoads = (int)(kNormPiece / kEach / kNormThreads);
  static_assert(kLoads >= 1 && kLoads <= 4 && kLoads * kEach * kNormThreads == kNormPiece, "a piece is whole loads");
};
// Pointers out of the plan are to global memory, which the compiler cannot see.
#define ARCS_GLOBAL __attribute__((address_space(1)))
template <typename T>
__device__ __forceinline__ void piece_load(const void* from, int count, PieceData& d) {
  using S = PieceShape<T>;
  const ARCS_GLOBAL T* p = (const ARCS_GLOBAL T*)from;
  const int whole = count / S::kEach;
#pragma unroll
  for (int j = 0; j < S::kLoads; ++j) {
    const int i = j * kNormThreads + threadIdx.x;
    if (i < whole) d.x[j] = ((const ARCS_GLOBAL Bytes16*)(p + i * S::kEach))->v;
  }
  const int i = whole * S::kEach + threadIdx.x;
  if (i < count) d.rest = widen((T)p[i]);
}
__device__ __forceinline__ void piece_load(const NormPiece& p, PieceData& d) {
  if (p.bf16) piece_load<__bf16>(p.from, p.count, d);
  else piece_load<float>(p.from, p.count, d);
}

template <typename T>
__device__ __forceinline__ void piece_widen(u32x4 x, float (&v)[PieceShape<T>::kEach]) {
  T t[PieceShape<T>::kEach];
  __builtin_memcpy(t, &x, 16);
#pragma unroll
  for (int e = 0; e < PieceShape<T>::kEach; ++e) v[e] = widen(t[e]);
}

template <typename T>
__device__ __forceinline__ double piece_squares(const PieceData& d, int count) {
  using S = PieceShape<T>;
  const int whole = count / S::kEach;
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < S::kLoads; ++j) {
    if (j * kNormThreads + (int)threadIdx.x >= whole) continue;
    float v[S::kEach];
    piece_widen<T>(d.x[j], v);
#pragma unroll
    for (int e = 0; e < S::kEach; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
  }
  if (whole * S::kEach + (int)threadIdx.x < count) s = __builtin_fma((double)d.rest, (double)d.rest, s);
  return s;
}

template <typename T, typename O>
__device__ __forceinline__ void piece_store(const PieceData& d, void* out, int count, double scale) {
  using S = PieceShape<T>;
  constexpr int kBytes = S::kEach * (int)sizeof(O);
  ARCS_GLOBAL O* to = (ARCS_GLOBAL O*)out;
  const int whole = count / S::kEach;
#pragma unroll
  for (int j = 0; j < S::kLoads; ++j) {
    const int i = j * kNormThreads + threadIdx.x;
    if (i >= whole) continue;
    float v[S::kEach];
    piece_widen<T>(d.x[j], v);
    O y[S::kEach];
#pragma unroll
    for (int e = 0; e < S::kEach; ++e) y[e] = (O)(float)((double)v[e] * scale);
    ARCS_GLOBAL O* at = to + i * S::kEach;
    if constexpr (kBytes == 8) {
      uint64_t b;
      __builtin_memcpy(&b, y, 8);
      ((ARCS_GLOBAL Bytes8*)at)->v = b;
    } else {
#pragma unroll
      for (int k = 0; k < kBytes / 16; ++k) {
        u32x4 b;
        __builtin_memcpy(&b, (char*)y + k * 16, 16);
        ((ARCS_GLOBAL Bytes16*)at)[k].v = b;
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // the 64-bit products of one load at a time, for registers
  }
  const int i = whole * S::kEach + threadIdx.x;
  if (i < count) to[i] = (O)(float)((double)d.rest * scale);
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

// The next piece is asked for before one is summed.
__global__ __launch_bounds__(kNormThreads) void norm_squares_kernel(NormArgs a) {
  double s = 0.0;
  auto squares = [&](const NormPiece& p, const PieceData& d) {
    s += p.bf16 ? piece_squares<__bf16>(d, p.count) : piece_squares<float>(d, p.count);
  };
  NormPiece p, q;
  PieceData d, e;
  int64_t i = blockIdx.x;
  auto ask = [&](NormPiece& p, PieceData& d) {
    i += gridDim.x;
    if (i >= a.pieces) return false;
    p = a.plan[i];
    piece_load(p, d);
    return true;
  };
  p = a.plan[i];
  piece_load(p, d);
  while (true) {
    bool more = ask(q, e);
    squares(p, d);
    if (!more) break;
    more = ask(p, d);
    squares(q, e);
    if (!more) break;
  }
  s = group_sum(s);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const NormArgs& a) {
  constexpr int kEach = kNormGroups / kNormThreads;
  double x[kEach], s = 0.0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = j * kNormThreads + threadIdx.x;
    x[j] = a.sums[i < a.groups ? i : 0];
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) s += j * kNormThreads + (int)threadIdx.x < a.groups ? x[j] : 0.0;
  return __builtin_sqrt(group_sum(s));
}

__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs a) {
  const double norm = norm_of(a);
  if (threadIdx.x == 0) *a.out_norm = (float)norm;
}

// A workgroup's first piece is asked for before the norm is added up.
__global__ __launch_bounds__(kNormThreads) void clip_kernel(NormArgs a) {
  int64_t i = a.pieces - 1 - blockIdx.x;
  NormPiece p = a.plan[i];
  PieceData d;
  piece_load(p, d);
  const double norm = norm_of(a);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.out_norm = (float)norm;
  const bool clipped = norm > a.max_norm && norm < __builtin_inf();
  const double scale = clipped ? a.max_norm / norm : 1.0;
  while (true) {
    if (p.to != nullptr && (clipped || p.from != p.to)) {
      if (p.bf16) {
        if (p.to_bf16) piece_store<__bf16, __bf16>(d, p.to, p.count, scale);
        else piece_store<__bf16, float>(d, p.to, p.count, scale);
      } else {
        if (p.to_bf16) piece_store<float, __bf16>(d, p.to, p.count, scale);
        else piece_store<float, float>(d, p.to, p.count, scale);
      }
    }
    i -= gridDim.x;
    if (i < 0) return;
    p = a.plan[i];
    if (p.to != nullptr && (clipped || p.from != p.to)) piece_load(p, d);
  }
}

// An empty plan has no sums, and the norm 0.
__global__ void norm_zero_kernel(float* out_norm) { *out_norm = 0.0f; }

hipError_t launch_norm(NormArgs a, bool clip, hipStream_t stream) {
  a.groups = norm_groups(a.pieces);
  const int64_t blocks = a.groups;
  if (blocks == 0) {
    hipLaunchKernelGGL(norm_zero_kernel, dim3(1), dim3(1), 0, stream, a.out_norm);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(norm_squares_kernel, dim3((unsigned)blocks), dim3(kNormThreads), 0, stream, a);
  if (clip) hipLaunchKernelGGL(clip_kernel, dim3((unsigned)blocks), dim3(kNormThreads), 0, stream, a);
  else hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kNormThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace arcs
