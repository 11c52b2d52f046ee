// Logits before sampling: penalties for tokens in the history, biases, grammar masks.
//
//   z' = penalise(z, count of the token in the row's history)   (the sampler's arithmetic)
//   z' = z' + (the token's biases, summed in list order)
//   z' = -inf where the token's mask bit is 0
//
// A workgroup has kAdjustSlice tokens of a row.  It goes over the row's whole history
// and bias lists, keeps what falls into its slice in two LDS tables (counts, sums of biases),
// and every thread then looks its own tokens up.  Reading the logits and writing
// them bounds the call; tokens that a mask takes away are not read, and in place only groups
// of 16 bytes that change are read and written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "linear_device.hpp"
#include "sample_common.hpp"

namespace arcs {

constexpr int kAdjustThreads = 256, kAdjustSlice = 4096;

// Whether any of a mask row's V bits is set.
__device__ __forceinline__ bool any_allowed(const uint32_t* mask, int64_t V) {
  const int64_t words = (V + 31) / 32;
  uint32_t any = 0;
  for (int64_t i = threadIdx.x; i < words; i += kAdjustThreads) {
    const uint32_t last = i == words - 1 && V % 32 != 0 ? (1u << (V % 32)) - 1u : 0xFFFFFFFFu;
    any |= mask[i] & last;
  }
  return __syncthreads_or(any != 0) != 0;
}

template <typename T, typename O, bool LISTS>
__global__ __launch_bounds__(kAdjustThreads) void adjust_kernel(AdjustArgs a) {
  constexpr int G = 16 / sizeof(T), kGroups = kAdjustSlice / kAdjustThreads / G;  // a thread's groups of G tokens
  __shared__ __align__(16) uint32_t count[LISTS ? kAdjustSlice : 4];
  __shared__ __align__(16) float sum[LISTS ? kAdjustSlice : 4];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / a.per_row;
  const int slice = (int)(blockIdx.x % a.per_row);

  int status = ARCS_ROW_OK;
  const uint32_t* mask = nullptr;
  if (a.mask != nullptr) {
    const int64_t at = a.mask_rows != nullptr ? a.mask_rows[b] : b;
    if (at >= 0 && at < a.masks) mask = a.mask + at * a.mask_stride;
    else if (at != -1) status = ARCS_ROW_BAD_MASK;
  }
  PenCtx pc = {};
  bool penalised = false;
  if (a.params != nullptr) {
    const arcs_row_params P = a.params[b];
    if (!(__builtin_isfinite(P.presence) && __builtin_isfinite(P.frequency) && __builtin_isfinite(P.repetition)) ||
        P.repetition < 0.0f)
      status = ARCS_ROW_BAD_PENALTY;
    set_penalty_values(pc, P);
    penalised = pc.rep_on || P.presence != 0.0f || P.frequency != 0.0f;
  }
  if (slice == a.slices || (a.per_row == a.slices && slice == 0 && a.out_status != nullptr)) {
    if (status == ARCS_ROW_OK && mask != nullptr && !any_allowed(mask, a.V)) status = ARCS_ROW_NOTHING_ALLOWED;
    if (tid == 0) a.out_status[b] = status;
    if (slice == a.slices) return;
  }

  const int64_t lo = (int64_t)slice * kAdjustSlice;
  const int len = (int)(a.V - lo < kAdjustSlice ? a.V - lo : kAdjustSlice);
  const T* row = (const T*)a.logits + b * a.stride + lo;
  O* to = (O*)a.out + b * a.out_stride + lo;
  if (status == ARCS_ROW_BAD_MASK || status == ARCS_ROW_BAD_PENALTY) {
    for (int i = tid; i < len; i += kAdjustThreads) to[i] = (O)__builtin_nanf("");
    return;
  }

  // the groups' tokens that are left, and their logits
  uint32_t keep[kGroups];
  float z[kGroups][G];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int at = (g * kAdjustThreads + tid) * G;
    keep[g] = at < len ? (1u << G) - 1u : 0u;
    if (mask != nullptr && at < len) keep[g] &= ((const uint8_t*)(mask + lo / 32))[at / 8] >> (at % 8);
  }
  auto load = [&](int g) {
    const int at = (g * kAdjustThreads + tid) * G;
    if (keep[g] != 0) load_some<T, G>(row + at, len - at, z[g]);
  };
  if (!a.in_place) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) load(g);
  }

  uint32_t c[kGroups][G];
  float bias[kGroups][G];
  bool listed = false;
  if constexpr (LISTS) {
    int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    if (penalised && a.hist_ids != nullptr) {
      h0 = a.hist_offsets[b];
      h1 = a.hist_offsets[b + 1];
    }
    if (a.bias_ids != nullptr) {
      b0 = a.bias_offsets[b];
      b1 = a.bias_offsets[b + 1];
    }
    listed = h1 > h0 || b1 > b0;
    if (listed) {
      const u32x4 zero = {0u, 0u, 0u, 0u}, none = {0x80000000u, 0x80000000u, 0x80000000u, 0x80000000u};
      for (int i = tid; i < kAdjustSlice / 4; i += kAdjustThreads) {
        ((u32x4*)count)[i] = zero;
        ((u32x4*)sum)[i] = none;  // -0: adding it changes nothing
      }
      __syncthreads();
#pragma unroll 4
      for (int64_t i = h0 + tid; i < h1; i += kAdjustThreads) {
        const int64_t at = (int64_t)a.hist_ids[i] - lo;
        if (at >= 0 && at < len) atomicAdd(&count[at], 1u);
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int e = 0; e < G; ++e) c[g][e] = count[(g * kAdjustThreads + tid) * G + e];
      if (b1 > b0) {
        // The counts' table now says who is next where a token is listed several times:
        // the lowest entry adds its bias first, so that sums have the list's order.
        __syncthreads();
        for (int i = tid; i < kAdjustSlice / 4; i += kAdjustThreads) ((u32x4*)count)[i] = zero;
        for (int64_t i0 = b0; i0 < b1; i0 += kAdjustThreads) {
          const int64_t i = i0 + tid;
          const int64_t at = i < b1 ? (int64_t)a.bias_ids[i] - lo : -1;
          bool waits = at >= 0 && at < len;
          const float value = waits ? a.bias_values[i] : 0.0f;
          while (__syncthreads_or(waits)) {
            if (waits) atomicMax(&count[at], (uint32_t)(kAdjustThreads - tid));
            __syncthreads();
            const bool next = waits && count[at] == (uint32_t)(kAdjustThreads - tid);
            __syncthreads();
            if (next) {
              sum[at] += value;
              count[at] = 0u;
              waits = false;
            }
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int e = 0; e < G; ++e) bias[g][e] = sum[(g * kAdjustThreads + tid) * G + e];
    }
  }

#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int at = (g * kAdjustThreads + tid) * G, left = len - at;
    if (left <= 0) continue;
    if (a.in_place) {
      const uint32_t all = (1u << (left < G ? left : G)) - 1u;
      bool changes = (keep[g] & all) != all;
      if (listed) {
#pragma unroll
        for (int e = 0; e < G; ++e) changes |= c[g][e] != 0u || __float_as_uint(bias[g][e]) != 0x80000000u;
      }
      if (!changes) continue;
      load(g);
    }
#pragma unroll
    for (int e = 0; e < G; ++e) {
      float y = z[g][e];
      if (listed) {
        if (c[g][e] != 0u) y = penalize(y, c[g][e], pc);
        y = y + bias[g][e];
      }
      z[g][e] = (keep[g] >> e) & 1u ? y : -__builtin_inff();
    }
    store_some<O, G>(to + at, left, z[g]);
  }
}

namespace {

template <typename T, typename O>
void launch(const AdjustArgs& a, unsigned blocks, hipStream_t stream) {
  if (a.hist_ids != nullptr || a.bias_ids != nullptr)
    hipLaunchKernelGGL((adjust_kernel<T, O, true>), dim3(blocks), dim3(kAdjustThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((adjust_kernel<T, O, false>), dim3(blocks), dim3(kAdjustThreads), 0, stream, a);
}

}  // namespace

bool adjust_fits(int64_t B, int64_t V) {
  return B * ((V + kAdjustSlice - 1) / kAdjustSlice + 1) <= 2147483647;
}

hipError_t launch_adjust(AdjustArgs a, int dtype, int out_dtype, int64_t B, hipStream_t stream) {
  a.slices = (int)((a.V + kAdjustSlice - 1) / kAdjustSlice);
  // one workgroup more a row looks the mask through where the status is wanted
  a.per_row = a.slices + (a.out_status != nullptr && a.mask != nullptr ? 1 : 0);
  const unsigned blocks = (unsigned)(B * a.per_row);
  if (dtype == ARCS_DTYPE_BF16) {
    if (out_dtype == ARCS_DTYPE_BF16) launch<__bf16, __bf16>(a, blocks, stream);
    else launch<__bf16, float>(a, blocks, stream);
  } else {
    if (out_dtype == ARCS_DTYPE_BF16) launch<float, __bf16>(a, blocks, stream);
    else launch<float, float>(a, blocks, stream);
  }
  return hipGetLastError();
}

}  // namespace arcs
