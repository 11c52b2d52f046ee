// Device-side pieces the linear layer's kernels share: activations, and rows that
// are not on the 16-byte grid.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.hpp"
#include "lds_load.hpp"
#include "mfma_tile.hpp"

namespace arcs {

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__bf16 x) { return (float)x; }

constexpr float kGeluA = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// act(z).  All in binary32; the activation is the same for a whole launch.  The normal
// distribution function and (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)) are taken in the forms that
// keep their digits where they are near 0.
__device__ __forceinline__ float act_value(float z, int act, float cap) {
  switch (act) {
    case ARCS_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case ARCS_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752440f);
    case ARCS_ACT_GELU_TANH: return z / (1.0f + expf(-2.0f * kGeluA * fmaf(kGeluB * z * z, z, z)));
    case ARCS_ACT_SILU: return z / (1.0f + expf(-z));
    case ARCS_ACT_SOFTCAP: return cap * tanhf(z / cap);
    default: return z;
  }
}

// act'(z).  1 - tanh^2 u is taken as 4 e / (1 + e)^2 with e = exp(-2 |u|), which keeps its
// digits where tanh u is near 1.
__device__ __forceinline__ float act_slope(float z, int act, float cap) {
  switch (act) {
    case ARCS_ACT_RELU: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case ARCS_ACT_GELU:
      return 0.5f * erfcf(z * -0.70710678118654752440f) + z * expf(-0.5f * z * z) * 0.39894228040143267794f;
    case ARCS_ACT_GELU_TANH: {
      const float zz = z * z, u = kGeluA * fmaf(kGeluB * zz, z, z);
      const float e = expf(-2.0f * fabsf(u)), d = 1.0f / (1.0f + e);
      const float half = u >= 0.0f ? d : e * d;  // (1 + tanh u) / 2
      // e is 0 where the rest may be infinite
      const float rest = e > 0.0f ? 2.0f * z * e * d * d * kGeluA * fmaf(3.0f * kGeluB, zz, 1.0f) : 0.0f;
      return z != z ? z : half + rest;
    }
    case ARCS_ACT_SILU: {
      const float e = expf(-fabsf(z)), d = 1.0f / (1.0f + e);
      const float s = z >= 0.0f ? d : e * d;
      // z s (1 - s), 0 in the limit
      return z != z ? z : s + (e > 0.0f ? z * e * d * d : 0.0f);
    }
    case ARCS_ACT_SOFTCAP: {
      const float e = expf(-2.0f * fabsf(z / cap)), d = 1.0f / (1.0f + e);
      return z != z ? z : 4.0f * e * d * d;
    }
    default: return 1.0f;
  }
}

// 16 bytes from an address that is aligned to its elements only (global memory takes
// such loads and stores whole).
struct __attribute__((packed, aligned(2))) Bytes16 {
  u32x4 v;
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint32_t x, y;
};
__device__ __forceinline__ u32x4 load16(const void* p) { return ((const Bytes16*)p)->v; }
__device__ __forceinline__ void store16(void* p, u32x4 v) { ((Bytes16*)p)->v = v; }

// `n` of E consecutive elements as float32 (zeros past n).
template <typename T, int E>
__device__ __forceinline__ void load_some(const T* p, int n, float (&v)[E]) {
  if (n >= E) {
    T t[E];
    if constexpr (E * sizeof(T) == 8) {
      const Bytes8 b = *(const Bytes8*)p;
      __builtin_memcpy(t, &b, 8);
    } else {
#pragma unroll
      for (int i = 0; i < (int)(E * sizeof(T) / 16); ++i) {
        const u32x4 b = load16((const char*)p + i * 16);
        __builtin_memcpy((char*)t + i * 16, &b, 16);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = widen(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = e < n ? widen(p[e]) : 0.0f;
  }
}
// Writes n of E consecutive elements.
template <typename T, int E>
__device__ __forceinline__ void store_some(T* p, int n, const float (&v)[E]) {
  T t[E];
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = (T)v[e];
  if (n >= E) {
    if constexpr (E * sizeof(T) == 8) {
      Bytes8 b;
      __builtin_memcpy(&b, t, 8);
      *(Bytes8*)p = b;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(E * sizeof(T) / 16); ++i) {
        u32x4 b;
        __builtin_memcpy(&b, (char*)t + i * 16, 16);
        store16((char*)p + i * 16, b);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < n) p[e] = t[e];
  }
}

}  // namespace arcs
