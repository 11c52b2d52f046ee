// Logits before sampling: penalties for tokens in the history, biases, grammar masks.
//
//   z' = penalise(z, count of the token in the row's history)   (the sampler's arithmetic)
//   z' = z' + (the token's biases, summed in list order)
//   z' = -inf where the token's mask bit is 0
//
// A workgroup has kAdjustSlice tokens of a row.  It goes over the row's whole history and counts
// what falls into its slice in an LDS table, from which every thread takes the counts of its own
// tokens; then the table holds the sums of the slice's biases.  Reading the logits and
// writing them bounds the call; tokens that a mask takes away are not read, and in place only
// groups of 16 bytes that change are read and written.  The first ids of both lists are asked
// for before the logits, so that the lists' work is done while the logits come in.
//
// 256 rows x 129,280 bfloat16 with 1,024 history ids and 100 biases each, half of the rows
// masked: 33 us (119 MB, 3.6 TB/s); 59 with an LDS table for counts and one for biases and loads
// that waited for each other, 42 with one table, 37.5 with the first ids ahead of the logits, 33
// with the logits kept as they are in memory until the lists are done (52 registers, eight waves a
// SIMD).  What remains is the chain of a workgroup: offsets, ids and mask, logits, table and
// barriers, about 5 us, five and a half rounds of it.  37 rows x 50,001 float32 with 20,000 ids: 14 us,
// most of it the lists.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "linear_device.hpp"
#include "sample_common.hpp"

namespace arcs {

constexpr int kAdjustSlice = 4096;

// Whether any of a mask row's V bits is set.
template <int kThreads>
__device__ __forceinline__ bool any_allowed(const uint32_t* mask, int64_t V) {
  const int64_t words = (V + 31) / 32;
  uint32_t any = 0;
  for (int64_t i = threadIdx.x; i < words; i += kThreads) {
    const uint32_t last = i == words - 1 && V % 32 != 0 ? (1u << (V % 32)) - 1u : 0xFFFFFFFFu;
    any |= mask[i] & last;
  }
  return __syncthreads_or(any != 0) != 0;
}

struct __attribute__((packed, aligned(4))) Ids4 {
  int32_t id[4];
};

// 16 bytes of a row as they are in memory, `left` elements of which exist.
template <typename T>
struct Raw16 {
  u32x4 q;
};
template <typename T>
__device__ __forceinline__ void load_raw16(Raw16<T>& r, const T* p, int left) {
  constexpr int G = 16 / sizeof(T);
  if (left >= G) {
    r.q = load16(p);
  } else {
    T t[G];
#pragma unroll
    for (int e = 0; e < G; ++e) t[e] = e < left ? p[e] : (T)0.0f;
    __builtin_memcpy(&r, t, 16);
  }
}
template <typename T, int G>
__device__ __forceinline__ void widen_raw(const Raw16<T>& r, float (&v)[G]) {
  T t[G];
  __builtin_memcpy(t, &r, 16);
#pragma unroll
  for (int e = 0; e < G; ++e) v[e] = widen(t[e]);
}

template <typename T, typename O, bool HISTORY, bool BIASES, int kThreads>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a) {
  constexpr int G = 16 / sizeof(T), kGroups = kAdjustSlice / kThreads / G;  // a thread's groups of G tokens
  constexpr int kFirst = 512 / kThreads, kAhead = 4;  // 16-byte loads of history ids: before the logits, and then at a time
  __shared__ __align__(16) uint32_t table[HISTORY || BIASES ? kAdjustSlice : 4];
  __shared__ uint2 entry[BIASES ? kThreads : 1];
  __shared__ int found[2][kThreads / kWave];
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
  int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
  if (HISTORY && penalised) {
    h0 = a.hist_offsets[b];
    h1 = a.hist_offsets[b + 1];
  }
  if (BIASES) {
    b0 = a.bias_offsets[b];
    b1 = a.bias_offsets[b + 1];
  }
  if (slice == a.slices || (a.per_row == a.slices && slice == 0 && a.out_status != nullptr)) {
    if (status == ARCS_ROW_OK && mask != nullptr && !any_allowed<kThreads>(mask, a.V)) status = ARCS_ROW_NOTHING_ALLOWED;
    if (tid == 0) a.out_status[b] = status;
    if (slice == a.slices) return;
  }

  const int64_t lo = (int64_t)slice * kAdjustSlice;
  const int len = (int)(a.V - lo < kAdjustSlice ? a.V - lo : kAdjustSlice);
  const T* row = (const T*)a.logits + b * a.stride + lo;
  O* to = (O*)a.out + b * a.out_stride + lo;
  if (status == ARCS_ROW_BAD_MASK || status == ARCS_ROW_BAD_PENALTY) {
    for (int i = tid; i < len; i += kThreads) to[i] = (O)__builtin_nanf("");
    return;
  }

  // What is asked for first: mask bits, then the first ids of the lists.
  uint32_t keep[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int at = (g * kThreads + tid) * G;
    keep[g] = at < len ? (1u << G) - 1u : 0u;
    if (mask != nullptr && at < len) keep[g] = ((const uint8_t*)(mask + lo / 32))[at / 8];
  }
  const bool counted = HISTORY && h1 > h0, biased = BIASES && b1 > b0;
  // Ids are taken four at a time; lanes past the last four read them again, and do not count.
  const int64_t fours = counted ? (h1 - h0) / 4 : 0;
  auto four = [&](int64_t i) { return *(const Ids4*)(a.hist_ids + h0 + (i < fours ? i : fours - 1) * 4); };
  Ids4 first[kFirst];
  int32_t rest = -1;  // one of the last, fewer than four
  if (counted) {
    if (fours > 0) {
#pragma unroll
      for (int j = 0; j < kFirst; ++j) first[j] = four(j * kThreads + tid);
    }
    if (tid < (int)((h1 - h0) & 3)) rest = a.hist_ids[h0 + fours * 4 + tid];
  }
  int32_t bias_id = -1;
  float bias_value = 0.0f;
  if (biased && b0 + tid < b1) {
    bias_id = a.bias_ids[b0 + tid];
    bias_value = a.bias_values[b0 + tid];
  }
  // the groups' tokens that are left, and their logits as they are in memory
  Raw16<T> raw[kGroups];
  auto load = [&](int g) {
    const int at = (g * kThreads + tid) * G;
    if (keep[g] != 0) load_raw16(raw[g], row + at, len - at);
  };
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int at = (g * kThreads + tid) * G;
    if (G < 8) keep[g] = (keep[g] >> (mask != nullptr ? at % 8 : 0)) & ((1u << G) - 1u);
    if (!a.in_place) load(g);
  }
  bool here[kGroups];  // in place: the group's logits are loaded
#pragma unroll
  for (int g = 0; g < kGroups; ++g) here[g] = !a.in_place;

  auto fill = [&](uint32_t x) {
    const u32x4 v = {x, x, x, x};
#pragma unroll
    for (int i = 0; i < kAdjustSlice / 4 / kThreads; ++i) ((u32x4*)table)[i * kThreads + tid] = v;
    __syncthreads();
  };
  float z[kGroups][G];
  bool wide[kGroups] = {};  // the group's values are in z
  // how often each of the slice's tokens is in the history
  if (counted) {
    fill(0u);
    // an id outside [0, V) is in no slice: negative ones are 2^31 or more, slices begin below that
    auto add = [&](int32_t id) {
      const uint32_t at = (uint32_t)id - (uint32_t)lo;
      if (at < (uint32_t)len) atomicAdd(&table[at], 1u);
    };
    if (fours > 0) {
#pragma unroll
      for (int j = 0; j < kFirst; ++j)
        if (j * kThreads + tid < fours) {
#pragma unroll
          for (int e = 0; e < 4; ++e) add(first[j].id[e]);
        }
    }
    add(rest);
    for (int64_t i = kFirst * kThreads + tid; i - tid < fours; i += kAhead * kThreads) {
      Ids4 x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) x[j] = four(i + j * kThreads);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * kThreads < fours) {
#pragma unroll
          for (int e = 0; e < 4; ++e) add(x[j].id[e]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t* own = table + (g * kThreads + tid) * G;
      uint32_t c[G], any = 0;
#pragma unroll
      for (int e = 0; e < G; ++e) {
        c[e] = own[e];
        any |= c[e];
      }
      if (any == 0u) continue;
      if (!here[g]) load(g);
      here[g] = true;
      widen_raw(raw[g], z[g]);
      wide[g] = true;
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (c[e] != 0u) z[g][e] = penalize(z[g][e], c[e], pc);
    }
  }

  // The biases of the slice's tokens, kThreads entries of the list at a time: those of the slice in
  // list order in LDS; the first entry of a token adds all of its token's.
  if (biased) {
    if (counted) __syncthreads();
    fill(0x80000000u);  // -0: adding it changes nothing
    float* sums = (float*)table;
    int turn = 0;
    for (int64_t i0 = b0; i0 < b1; i0 += kThreads, turn ^= 1) {
      const int64_t i = i0 + tid;
      if (i0 != b0 && i < b1) {
        bias_id = a.bias_ids[i];
        bias_value = a.bias_values[i];
      }
      const uint32_t at = (uint32_t)bias_id - (uint32_t)lo;
      const bool in = i < b1 && at < (uint32_t)len;
      const uint64_t lanes = __ballot(in);
      if ((tid & 63) == 0) found[turn][tid >> 6] = __popcll(lanes);
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / kWave; ++w) {
        before += w < (tid >> 6) ? found[turn][w] : 0;
        all += found[turn][w];
      }
      if (all == 0) continue;
      before += __popcll(lanes & ((1ull << (tid & 63)) - 1ull));
      if (in) entry[before] = make_uint2(at, __float_as_uint(bias_value));
      __syncthreads();
      if (in) {
        bool later = false;
        float s = sums[at];
        for (int j = 0; j < all; ++j) {
          const uint2 x = entry[j];
          if (x.x != at) continue;
          later |= j < before;
          s += __uint_as_float(x.y);
        }
        bias_value = s;
        if (later) bias_id = -1;
      }
      __syncthreads();
      if (in && bias_id >= 0) sums[at] = bias_value;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float* own = sums + (g * kThreads + tid) * G;
      float s[G];
      bool any = false;
#pragma unroll
      for (int e = 0; e < G; ++e) {
        s[e] = own[e];
        any |= __float_as_uint(s[e]) != 0x80000000u;
      }
      if (!any) continue;
      if (!here[g]) load(g);
      here[g] = true;
      if (!wide[g]) widen_raw(raw[g], z[g]);
      wide[g] = true;
#pragma unroll
      for (int e = 0; e < G; ++e) z[g][e] += s[e];
    }
  }

#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int at = (g * kThreads + tid) * G, left = len - at;
    if (left <= 0) continue;
    if (!here[g]) {
      const uint32_t all = (1u << (left < G ? left : G)) - 1u;
      if ((keep[g] & all) == all) continue;
      load(g);
    }
    if (!wide[g]) widen_raw(raw[g], z[g]);
#pragma unroll
    for (int e = 0; e < G; ++e) z[g][e] = (keep[g] >> e) & 1u ? z[g][e] : -__builtin_inff();
    store_some<O, G>(to + at, left, z[g]);
  }
}

namespace {

template <typename T, typename O, int kThreads>
void launch(const AdjustArgs& a, unsigned blocks, hipStream_t stream) {
  const dim3 grid(blocks), threads(kThreads);
  if (a.hist_ids != nullptr) {
    if (a.bias_ids != nullptr) hipLaunchKernelGGL((adjust_kernel<T, O, true, true, kThreads>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((adjust_kernel<T, O, true, false, kThreads>), grid, threads, 0, stream, a);
  } else {
    if (a.bias_ids != nullptr) hipLaunchKernelGGL((adjust_kernel<T, O, false, true, kThreads>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((adjust_kernel<T, O, false, false, kThreads>), grid, threads, 0, stream, a);
  }
}

// Workgroups of 512 threads where the compute units hold them all (four each), so that the lists are
// gone over sooner: 37 rows x 50,001 float32 with 20,000 history ids each 14.7 us, 16.6 with 256;
// many take 256 threads, of which more workgroups fly at once: 256 rows x 129,280 33 us, 53 with 512.
template <typename T, typename O>
void launch(const AdjustArgs& a, unsigned blocks, hipStream_t stream) {
  if (blocks <= 1024) launch<T, O, 512>(a, blocks, stream);
  else launch<T, O, 256>(a, blocks, stream);
}

}  // namespace

bool adjust_fits(int64_t B, int64_t V) {
  return B * ((V + kAdjustSlice - 1) / kAdjustSlice + 1) <= 2147483647;
}

hipError_t launch_adjust(AdjustArgs a, int dtype, int out_dtype, int64_t B, hipStream_t stream) {
  a.slices = (int)((a.V + kAdjustSlice - 1) / kAdjustSlice);
  // one workgroup more a row looks the mask through where the status is wanted
  a.per_row = a.slices + (a.out_status != nullptr && a.mask != nullptr ? 1 : 0);
  // A launch holds fewer than 2^32 threads: more rows take several.
  const int64_t most = ((int64_t(1) << 24) - 1) / a.per_row, element = dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  const int64_t out_element = out_dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  for (int64_t b = 0; b < B; b += most) {
    const int64_t rows = B - b < most ? B - b : most;
    const unsigned blocks = (unsigned)(rows * a.per_row);
    if (dtype == ARCS_DTYPE_BF16) {
      if (out_dtype == ARCS_DTYPE_BF16) launch<__bf16, __bf16>(a, blocks, stream);
      else launch<__bf16, float>(a, blocks, stream);
    } else {
      if (out_dtype == ARCS_DTYPE_BF16) launch<float, __bf16>(a, blocks, stream);
      else launch<float, float>(a, blocks, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // the next rows' parts of what is listed by rows
    a.logits = (const char*)a.logits + rows * a.stride * element;
    a.out = (char*)a.out + rows * a.out_stride * out_element;
    if (a.params != nullptr) a.params += rows;
    if (a.hist_offsets != nullptr) a.hist_offsets += rows;
    if (a.bias_offsets != nullptr) a.bias_offsets += rows;
    if (a.mask_rows != nullptr) {
      a.mask_rows += rows;
    } else if (a.mask != nullptr) {
      a.mask += rows * a.mask_stride;
      a.masks -= rows;
    }
    if (a.out_status != nullptr) a.out_status += rows;
  }
  return hipSuccess;
}

}  // namespace arcs
