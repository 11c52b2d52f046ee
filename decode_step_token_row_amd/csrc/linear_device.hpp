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

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kGeluA = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// exp2 and the reciprocal of the vector unit are off by one unit in the last place.  (The
// library's expf and division made dz three times as long as its way through memory.)
// exp_fast's argument is rounded, which is |x| 2^-23 of the result: for what falls as fast.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2E); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// exp(-c (x + dx)) for x >= 0, `high` and `low` being c log2 e in two parts: what the argument's rounding
// leaves, which would be x 2^-24 of the result, is applied to it as a factor.  (4,096 x 4,096
// bfloat16, dz without it and without half powers 17.6 us with silu and 19.4 with gelu by tanh, 19.7 and
// 23.2 with both; the forward product of 4,096 columns of k 135 and 125, 139 and 128.)
__device__ __forceinline__ float exp2_minus(float t, float rest) {
  const float y = __builtin_amdgcn_exp2f(-t);
  return fmaf(y * -0.69314718055994530942f, rest, y);
}
__device__ __forceinline__ float exp_minus(float x, float high, float low) {
  const float t = x * high;
  return exp2_minus(t, fmaf(x, low, fmaf(x, high, -t)));
}
__device__ __forceinline__ float exp_minus(float x, float dx, float high, float low) {
  const float t = x * high;
  return exp2_minus(t, fmaf(dx, high, fmaf(x, low, fmaf(x, high, -t))));
}
// A constant's float32 value and what that leaves.
constexpr float high_part(double c) { return (float)c; }
constexpr float low_part(double c) { return (float)(c - (double)(float)c); }

// exp(-a / 2), 0 past 256.
__device__ __forceinline__ float half_power(float a) {
  constexpr double kC = 0.5 * 1.4426950408889634;
  return exp_minus(__builtin_fminf(a, 256.0f), high_part(kC), low_part(kC));
}
// exp(-u), u = sqrt(2 / pi) (a + 0.044715 a^3), 0 past 16; u in two parts, each step with what it leaves.
__device__ __forceinline__ float half_power_tanh(float a) {
  constexpr double kB = 0.044715, kC = 0.79788456080286535588 * 1.4426950408889634;
  a = __builtin_fminf(a, 16.0f);
  const float aa = a * a, aa_left = fmaf(a, a, -aa);
  const float s = fmaf(aa, high_part(kB), 1.0f);  // 1 - s is exact, s being at least 1
  const float s_left = fmaf(aa_left, high_part(kB), fmaf(aa, low_part(kB), fmaf(aa, high_part(kB), 1.0f - s)));
  const float u = a * s, u_left = fmaf(a, s_left, fmaf(a, s, -u));
  return exp_minus(u, u_left, high_part(kC), low_part(kC));
}

// The normal distribution function's smaller tail, Phi(-a) = H exp(-a^2 / 2), a = |z|, as H and
// h = exp(-a^2 / 4): H falls as slowly as 1 / a, and h is applied twice, so that z h H h keeps its digits
// as long as it is a normal number itself.  H = t P(t), t = 1 / (1 + 0.36 a), P of degree 8 fitted to
// the least largest relative error over a in 0 .. 40, which is 1.5 2^-24 (6.3 2^-24 with its own
// roundings; one degree less 16, one more 0.3 and 4.8).  a^2 / 4 is carried in two parts, as its
// rounding alone would be 2^-24 a^2 / 4 of h.  Past 32 all of it is 0.
__device__ __forceinline__ float normal_tail(float a, float& h) {
  constexpr double kC = 0.25 * 1.4426950408889634;
  a = __builtin_fminf(a, 32.0f);
  const float aa = a * a;
  h = exp_minus(aa, fmaf(a, a, -aa), high_part(kC), low_part(kC));
  const float t = rcp_fast(fmaf(0.36f, a, 1.0f));
  float s = fmaf(t, -0.030238168f, 0.13950802f);
  s = fmaf(t, s, -0.22359903f);
  s = fmaf(t, s, 0.10736878f);
  s = fmaf(t, s, -0.00038622523f);
  s = fmaf(t, s, 0.09603733f);
  s = fmaf(t, s, 0.12400976f);
  s = fmaf(t, s, 0.14368188f);
  s = fmaf(t, s, 0.14361766f);
  return s * t;
}

// c tanh u, u = z / c.  Up to |u| = 1/4 by the series of tanh u to u^9 (the next term is 8e-9 of it), as
// z + z (tanh u / u - 1), so that z whose u is too small for a number of its own stay what they are; above that
// c (1 - e) / (1 + e) with e = exp(-2 |u|).
__device__ __forceinline__ float softcap(float z, float c, float inv_c) {
  const float u = z * inv_c, w = u * u;
  float s = fmaf(w, 62.0f / 2835.0f, -17.0f / 315.0f);
  s = fmaf(w, s, 2.0f / 15.0f);
  s = fmaf(w, s, -1.0f / 3.0f);
  s = fmaf(w * s, z, z);
  const float e = exp_fast(-2.0f * fabsf(u));
  const float far = c * __builtin_copysignf((1.0f - e) * rcp_fast(1.0f + e), u);
  return fabsf(u) < 0.25f ? s : far;
}

// z / (1 + exp(-x)), where h = exp(-|x| / 2) and x has the sign of z.  Below 0 that is z h^2 / (1 + h^2),
// which keeps its digits as long as it is a normal number itself.
__device__ __forceinline__ float gated(float z, float h) {
  return (z >= 0.0f ? z : z * h * h) * rcp_fast(fmaf(h, h, 1.0f));
}

// act(z) in binary32, within 20 2^-24 of itself.  (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)).
template <int ACT>
__device__ __forceinline__ float act_value(float z, float cap, float inv_cap) {
  switch (ACT) {
    case ARCS_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case ARCS_ACT_GELU: {
      float h;
      const float tail = normal_tail(fabsf(z), h);
      return z < 0.0f ? z * h * tail * h : z * (1.0f - tail * h * h);
    }
    case ARCS_ACT_GELU_TANH: return gated(z, half_power_tanh(fabsf(z)));
    case ARCS_ACT_SILU: return gated(z, half_power(fabsf(z)));
    case ARCS_ACT_SOFTCAP: return softcap(z, cap, inv_cap);
    default: return z;
  }
}

// act'(z).  1 - tanh^2 u is taken as 4 e / (1 + e)^2 with e = exp(-2 |u|), which keeps its
// digits where tanh u is near 1.
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float inv_cap) {
  switch (ACT) {
    case ARCS_ACT_RELU: return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    case ARCS_ACT_GELU: {
      // Phi(z) + z phi(z), 0 or 1 in the limits
      const float a = __builtin_fminf(fabsf(z), 32.0f);
      float h;
      const float tail = normal_tail(a, h), e = h * h, rest = a * 0.39894228040143267794f;
      return z != z ? z : z < 0.0f ? e * (tail - rest) : fmaf(e, rest - tail, 1.0f);
    }
    case ARCS_ACT_GELU_TANH: {
      // half + rest, half = (1 + tanh u) / 2
      const float a = __builtin_fminf(fabsf(z), 16.0f), h = half_power_tanh(a);
      const float e = h * h, d = rcp_fast(1.0f + e), ed = e * d;
      const float rest = 2.0f * kGeluA * a * ed * d * fmaf(3.0f * kGeluB, a * a, 1.0f);
      return z != z ? z : z >= 0.0f ? d + rest : ed - rest;
    }
    case ARCS_ACT_SILU: {
      // s + z s (1 - s), s = 1 / (1 + exp(-z))
      const float a = __builtin_fminf(fabsf(z), 256.0f), h = half_power(a);
      const float e = h * h, d = rcp_fast(1.0f + e), ed = e * d, rest = a * ed * d;
      return z != z ? z : z >= 0.0f ? d + rest : ed - rest;
    }
    case ARCS_ACT_SOFTCAP: {
      const float e = exp_fast(-2.0f * fabsf(z * inv_cap)), d = rcp_fast(1.0f + e);
      return z != z ? z : 4.0f * e * d * d;
    }
    default: return 1.0f;
  }
}

// The activation is the same for a whole launch: one branch for several elements, whose
// chains of operations then overlap.
template <int ACT, int E>
__device__ __forceinline__ void act_each(float (&v)[E], float cap, float inv_cap) {
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = act_value<ACT>(v[e], cap, inv_cap);
}
template <int E>
__device__ __forceinline__ void act_values(float (&v)[E], int act, float cap, float inv_cap) {
  switch (act) {
    case ARCS_ACT_RELU: return act_each<ARCS_ACT_RELU>(v, cap, inv_cap);
    case ARCS_ACT_GELU: return act_each<ARCS_ACT_GELU>(v, cap, inv_cap);
    case ARCS_ACT_GELU_TANH: return act_each<ARCS_ACT_GELU_TANH>(v, cap, inv_cap);
    case ARCS_ACT_SILU: return act_each<ARCS_ACT_SILU>(v, cap, inv_cap);
    case ARCS_ACT_SOFTCAP: return act_each<ARCS_ACT_SOFTCAP>(v, cap, inv_cap);
    default: return;
  }
}
// g times act'(z)
template <int ACT, int E>
__device__ __forceinline__ void slope_each(float (&g)[E], const float (&z)[E], float inv_cap) {
#pragma unroll
  for (int e = 0; e < E; ++e) g[e] *= act_slope<ACT>(z[e], inv_cap);
}
template <int E>
__device__ __forceinline__ void act_slopes(float (&g)[E], const float (&z)[E], int act, float inv_cap) {
  switch (act) {
    case ARCS_ACT_RELU: return slope_each<ARCS_ACT_RELU>(g, z, inv_cap);
    case ARCS_ACT_GELU: return slope_each<ARCS_ACT_GELU>(g, z, inv_cap);
    case ARCS_ACT_GELU_TANH: return slope_each<ARCS_ACT_GELU_TANH>(g, z, inv_cap);
    case ARCS_ACT_SILU: return slope_each<ARCS_ACT_SILU>(g, z, inv_cap);
    case ARCS_ACT_SOFTCAP: return slope_each<ARCS_ACT_SOFTCAP>(g, z, inv_cap);
    default: return;
  }
}

// 16 bytes from an address that is aligned to its elements only (global memory takes
// such loads and stores whole).
struct __attribute__((packed, aligned(2))) Bytes16 {
  u32x4 v;
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint64_t v;
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
// Eight consecutive elements as they are in memory, so that the loads can fly while other work is
// done; `n` of them exist (zeros past n).
template <typename T>
struct Raw8 {
  u32x4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(Raw8<T>& r, const T* p, int n) {
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = load16((const char*)p + i * 16);
  } else {
    T t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = e < n ? p[e] : (T)0.0f;
    __builtin_memcpy(&r, t, sizeof(r));
  }
}
template <typename T>
__device__ __forceinline__ void widen_raw(const Raw8<T>& r, float (&v)[8]) {
  T t[8];
  __builtin_memcpy(t, &r, sizeof(r));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = widen(t[e]);
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
