// Head logits from 4-bit weights with group scales.
//
//   logits[b, v] = sum_g scale[v, g] * sum_{d in g} (q[v, d] - zero[v, g]) hidden[b, d]
//
// q is two weights a byte, the lower d in the low nibble.  The products run
// on the bfloat16 matrix instruction with the batch as its rows and 16
// vocabulary rows as its columns.  A nibble becomes the bfloat16 16 + q by an
// AND and an OR on two weights at a time (0x4180 is 16.0 and a step of its
// mantissa's bit 3 is 1), which is exact, and the group's sum is put right
// with the sum of the hidden state over the group, from a product with ones:
//   sum (q - z) h = sum (16 + q) h - (16 + z) sum h.
// Scales are applied to the group's float32 sums, so no weight is rounded.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "arcs.h"
#include "device_common.hpp"
#include "launch.hpp"

namespace arcs {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kW4Chunk = 128;  // k of one step: 16 bytes of a weight row in each of four lanes

// Eight nibbles as bfloat16 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 w4_unpack(uint32_t w) {
  u32x4 d;
  d[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
  d[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
  d[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
  d[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8, d);
}

// Eight bfloat16 in the same order.
__device__ __forceinline__ bf16x8 w4_order(u32x4 x) {
  u32x4 d;
  d[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
  d[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
  d[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
  d[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
  return __builtin_bit_cast(bf16x8, d);
}

// w[i] of lane group j <-> w[j] of lane group i (groups of 16 lanes).
__device__ __forceinline__ void w4_transpose(u32x4& w) {
  auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}

// GROUP 128: a lane's 16 bytes are 32 consecutive k and one product takes 8 of
// each lane group's.  GROUP 32, 64: the 16 bytes are exchanged between the four
// lane groups first, so that a product's 32 k are consecutive and lie in one group.
template <int RT, int GROUP, bool ZERO, bool SF32, bool OF32>
__global__ __launch_bounds__(256) void w4_logits_kernel(W4Args a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, j = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * (RT * 16);
  if (v0 >= a.V) return;
  const int64_t b0 = (int64_t)blockIdx.y * 16;
  constexpr int kGroups = kW4Chunk / GROUP, kSteps = 4 / kGroups;
  constexpr bool kTurn = GROUP < 128;
  const int64_t b = b0 + r < a.B ? b0 + r : a.B - 1;
  const uint16_t* x = a.hidden + b * a.hidden_stride;
  const uint8_t* q[RT];
  int64_t sc[RT], zr[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t v = v0 + t * 16 + r < a.V ? v0 + t * 16 + r : a.V - 1;
    q[t] = a.qweight + v * a.qweight_stride;
    sc[t] = v * a.scale_stride;
    zr[t] = v * a.zero_stride;
  }
  const u32x4 one4 = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, one4);
  const u32x4 zero4 = {0, 0, 0, 0};
  const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 total[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) total[t] = none;

  for (int64_t k = 0; k < a.D; k += kW4Chunk) {
    u32x4 w[RT];
    const bool here = !kTurn || k + j * 32 < a.D;
#pragma unroll
    for (int t = 0; t < RT; ++t) w[t] = here ? *(const u32x4*)(q[t] + (k >> 1) + j * 16) : zero4;
    bf16x8 xs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = k + (kTurn ? i * 32 + j * 8 : j * 32 + i * 8);
      xs[i] = w4_order(!kTurn || k + i * 32 < a.D ? *(const u32x4*)(x + at) : zero4);
    }
    if (kTurn) {
#pragma unroll
      for (int t = 0; t < RT; ++t) w4_transpose(w[t]);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (kTurn && k + g * GROUP >= a.D) break;
      const int64_t at = k / GROUP + g;
      f32x4 sum = none;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[g * kSteps + i], ones, sum, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f32x4 acc = none;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[g * kSteps + i], w4_unpack(w[t][g * kSteps + i]), acc, 0, 0, 0);
        const float s = SF32 ? ((const float*)a.scales)[sc[t] + at] : bf16_to_f32(((const uint16_t*)a.scales)[sc[t] + at]);
        const float off = 16.0f + (ZERO ? (float)a.zeros[zr[t] + at] : 8.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) total[t][e] = fmaf(s, fmaf(-off, sum[e], acc[e]), total[t][e]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t v = v0 + t * 16 + r;
    if (v >= a.V) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t row = b0 + j * 4 + e;
      if (row >= a.B) continue;
      if (OF32) ((float*)a.logits)[row * a.row_stride + v] = total[t][e];
      else ((__bf16*)a.logits)[row * a.row_stride + v] = (__bf16)total[t][e];
    }
  }
}

template <int GROUP, bool ZERO, bool SF32>
static void launch_w4_typed(const W4Args& a, bool f32, hipStream_t stream) {
  constexpr int kRT = 2;
  const dim3 grid((unsigned)((a.V + 64 * kRT - 1) / (64 * kRT)), (unsigned)((a.B + 15) / 16)), block(256);
  if (f32) hipLaunchKernelGGL((w4_logits_kernel<kRT, GROUP, ZERO, SF32, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((w4_logits_kernel<kRT, GROUP, ZERO, SF32, false>), grid, block, 0, stream, a);
}

template <int GROUP>
static void launch_w4_group(const W4Args& a, bool sf32, bool f32, hipStream_t stream) {
  if (a.zeros) {
    if (sf32) launch_w4_typed<GROUP, true, true>(a, f32, stream);
    else launch_w4_typed<GROUP, true, false>(a, f32, stream);
  } else {
    if (sf32) launch_w4_typed<GROUP, false, true>(a, f32, stream);
    else launch_w4_typed<GROUP, false, false>(a, f32, stream);
  }
}

hipError_t launch_w4_logits(const W4Args& a, int scale_dtype, int logits_dtype, int group, hipStream_t stream) {
  const bool sf32 = scale_dtype == ARCS_DTYPE_F32, f32 = logits_dtype == ARCS_DTYPE_F32;
  if (group == 32) launch_w4_group<32>(a, sf32, f32, stream);
  else if (group == 64) launch_w4_group<64>(a, sf32, f32, stream);
  else launch_w4_group<128>(a, sf32, f32, stream);
  return hipGetLastError();
}

}  // namespace arcs
