// The linear layer's smaller kernels and its launches: the forward pass of few rows, dz
// and dbias, and copies of rows that are not on the 16-byte grid.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.hpp"
#include "linear_device.hpp"
#include "launch.hpp"

namespace arcs {

// ---------------------------------------------------------------------------
// forward, few rows
// ---------------------------------------------------------------------------
// A workgroup makes 16 columns of the output for all rows: its waves take the steps of k in
// turn, weights and hidden states straight from memory to registers (16 bytes a lane: the
// lane's row, 8 k of bfloat16 or 4 of float32), and their sums meet in LDS.
constexpr int kFewWaves = 8;

template <typename T>
__device__ __forceinline__ u32x4 few_load(const T* row, int64_t k, int64_t D) {
  constexpr int kEach = 16 / sizeof(T);
  if (k + kEach <= D) return load16(row + k);
  u32x4 v = {0u, 0u, 0u, 0u};
  T t[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) t[e] = k + e < D ? row[k + e] : (T)0.0f;
  __builtin_memcpy(&v, t, 16);
  return v;
}

template <typename T>
__device__ __forceinline__ f32x4 few_product(u32x4 x, u32x4 y, f32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[e]), __uint_as_float(y[e]), c, 0, 0, 0);
    return c;
  }
}

template <typename T>
__global__ __launch_bounds__(kFewWaves * 64) void linear_few_kernel(LinearArgs a) {
  constexpr int kStep = 64 / sizeof(T);  // k of one product: 16 bytes in each of four lanes of a row
  __shared__ float part[kFewWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t v0 = (int64_t)blockIdx.x * 16;
  const int r = lane & 15, q = lane >> 4;
  // rows past the last one repeat it, and are not stored
  const int64_t v = v0 + r < a.V ? v0 + r : a.V - 1;
  const int64_t n = r < a.N ? r : a.N - 1;
  const T* w = (const T*)a.weight + v * a.weight_stride;
  const T* h = (const T*)a.hidden + n * a.hidden_stride;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int64_t k = (int64_t)wave * kStep; k < a.D; k += kFewWaves * kStep) {
    const int64_t at = k + q * (16 / (int)sizeof(T));
    acc = few_product<T>(few_load(w, at, a.D), few_load(h, at, a.D), acc);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) part[wave][q * 4 + e][r] = acc[e];
  __syncthreads();
  // thread: column v0 + tid % 16 of row tid / 16
  if (tid >= 256) return;
  const int c = tid & 15, row = tid >> 4;
  if (row >= a.N || v0 + c >= a.V) return;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < kFewWaves; ++i) z += part[i][c][row];
  if (a.bias != nullptr) z += widen(((const T*)a.bias)[v0 + c]);
  if (a.out_pre != nullptr) ((T*)a.out_pre)[row * a.V + v0 + c] = (T)z;
  float y = act_value(z, a.act, a.cap);
  if (a.residual != nullptr) y += widen(((const T*)a.residual)[row * a.residual_stride + v0 + c]);
  if (a.out_bf16) ((__bf16*)a.out)[row * a.out_stride + v0 + c] = (__bf16)y;
  else ((float*)a.out)[row * a.out_stride + v0 + c] = y;
}

// ---------------------------------------------------------------------------
// backward: dz and the columns' sums
// ---------------------------------------------------------------------------
// A thread has 8 columns of chunk_rows rows.  The sums take dz before it is rounded to T.
// dz may be NULL (only dbias is wanted, or grad_out is dz as it is), and so may the sums.
template <typename T, typename G>
__global__ __launch_bounds__(128) void linear_dz_kernel(LinearArgs a, T* dz, int64_t ldz, float* sums, int64_t chunk_rows) {
  const int64_t v = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 8;
  if (v >= ldz && v >= a.V) return;
  const int left = (int)(a.V - v < 8 ? a.V - v : 8);
  const int64_t n0 = (int64_t)blockIdx.y * chunk_rows, n1 = n0 + chunk_rows < a.N ? n0 + chunk_rows : a.N;
  float sum[8] = {};
  if (left > 0) {
#pragma unroll 2
    for (int64_t n = n0; n < n1; ++n) {
      float g[8];
      load_some<G, 8>((const G*)a.grad + n * a.grad_stride + v, left, g);
      if (a.act != ARCS_ACT_NONE) {
        float z[8];
        load_some<T, 8>((const T*)a.pre + n * a.V + v, left, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = e < left ? g[e] * act_slope(z[e], a.act, a.cap) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
      if (dz != nullptr) store_some<T, 8>(dz + n * ldz + v, 8, g);  // zeros past V, up to ldz
    }
    if (sums != nullptr) store_some<float, 8>(sums + blockIdx.y * a.V + v, left, sum);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void linear_dbias_kernel(const float* sums, int64_t V, int64_t chunks, T* out) {
  __shared__ double part[4][64];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t v = (int64_t)blockIdx.x * 64 + c;
  double s = 0.0;
  if (v < V)
    for (int64_t i = g; i < chunks; i += 4) s += (double)sums[i * V + v];
  part[g][c] = s;
  __syncthreads();
  if (g == 0 && v < V) out[v] = (T)(float)((part[0][c] + part[1][c]) + (part[2][c] + part[3][c]));
}

// Rows of `columns` elements to rows of ld, zeros behind them.
template <typename T>
__global__ __launch_bounds__(256) void linear_pack_kernel(const T* from, int64_t stride, int64_t columns, T* to, int64_t ld) {
  constexpr int kEach = 16 / sizeof(T);
  const int64_t row = blockIdx.x;
  const T* p = from + row * stride;
  for (int64_t c = threadIdx.x * kEach; c < ld; c += 256 * kEach) {
    const int64_t left = columns - c;
    float v[kEach];
    load_some<T, kEach>(p + c, (int)(left < kEach ? left > 0 ? left : 0 : kEach), v);
    store_some<T, kEach>(to + row * ld + c, kEach, v);
  }
}

namespace {

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
size_t padded(int64_t bytes) { return (size_t)((bytes + 255) / 256 * 256); }

size_t slab_bytes(int mode, int64_t M, int64_t N, int64_t K, bool bf16) {
  const LinearShape s = linear_shape(mode, M, N, K, bf16);
  if (s.workers == 0) return 0;
  return padded((s.workers + tiles(M, s.columns) * tiles(N, s.rows)) * s.columns * s.rows * 4);
}

template <typename T>
void pack(const void*& rows, int64_t& stride, int64_t count, int64_t columns, char* to, int64_t ld, hipStream_t stream) {
  hipLaunchKernelGGL(linear_pack_kernel<T>, dim3((unsigned)count), dim3(256), 0, stream, (const T*)rows, stride, columns,
                     (T*)to, ld);
  rows = to;
  stride = ld;
}

// Copies of the rows that are not on the grid.  Both operands' rows run along k in the forward
// pass, so a D off the grid needs both copies.
template <typename T>
void pack_operands(LinearArgs& a, const LinearPlan& plan, int dtype, hipStream_t stream) {
  if (!linear_rows_aligned(a.hidden, a.hidden_stride, a.D, dtype))
    pack<T>(a.hidden, a.hidden_stride, a.N, a.D, a.workspace + plan.hidden, plan.ldd, stream);
  if (!linear_rows_aligned(a.weight, a.weight_stride, a.D, dtype))
    pack<T>(a.weight, a.weight_stride, a.V, a.D, a.workspace + plan.weight, plan.ldd, stream);
}

template <typename T>
hipError_t forward(LinearArgs a, int dtype, bool aligned, hipStream_t stream) {
  if (a.N <= kLinearFewRows) {
    hipLaunchKernelGGL(linear_few_kernel<T>, dim3((unsigned)tiles(a.V, 16)), dim3(kFewWaves * 64), 0, stream, a);
    return hipGetLastError();
  }
  const LinearPlan plan = linear_plan(a.N, a.V, a.D, dtype, aligned, false);
  pack_operands<T>(a, plan, dtype, stream);
  LinearProduct p = {};
  p.a = a.weight;
  p.lda = a.weight_stride;
  p.b = a.hidden;
  p.ldb = a.hidden_stride;
  p.M = a.V;
  p.N = a.N;
  p.K = plan.ldd;
  p.out = a.out;
  p.ldo = a.out_stride;
  p.out_bf16 = a.out_bf16;
  p.slab = (float*)(a.workspace + plan.slab);
  p.shape = linear_shape(kLinForward, p.M, p.N, p.K, sizeof(T) == 2);
  p.bias = a.bias;
  p.residual = a.residual;
  p.ldr = a.residual_stride;
  p.pre = a.out_pre;
  p.ldp = a.V;
  p.act = a.act;
  p.cap = a.cap;
  return launch_linear_product(p, kLinForward, dtype, stream);
}

template <typename T>
hipError_t backward(LinearArgs a, int dtype, bool aligned, hipStream_t stream) {
  const LinearPlan plan = linear_plan(a.N, a.V, a.D, dtype, aligned, true);
  const bool same = a.grad_bf16 == (sizeof(T) == 2 ? 1 : 0);
  // without an activation grad_out is dz, if the products can read it where it is
  const bool direct = a.act == ARCS_ACT_NONE && same && linear_rows_aligned(a.grad, a.grad_stride, a.V, dtype);
  const bool products = a.out_dhidden != nullptr || a.out_dweight != nullptr;
  T* dz = products && !direct ? (T*)(a.workspace + plan.dz) : nullptr;
  float* sums = a.out_dbias != nullptr ? (float*)(a.workspace + plan.dbias) : nullptr;
  const int64_t chunks = tiles(a.N, plan.chunk_rows);
  if (dz != nullptr || sums != nullptr) {
    const dim3 grid((unsigned)tiles(a.V, 1024), (unsigned)chunks);
    if (a.grad_bf16)
      hipLaunchKernelGGL((linear_dz_kernel<T, __bf16>), grid, dim3(128), 0, stream, a, dz, plan.ldz, sums, plan.chunk_rows);
    else
      hipLaunchKernelGGL((linear_dz_kernel<T, float>), grid, dim3(128), 0, stream, a, dz, plan.ldz, sums, plan.chunk_rows);
  }
  if (sums != nullptr)
    hipLaunchKernelGGL(linear_dbias_kernel<T>, dim3((unsigned)tiles(a.V, 64)), dim3(256), 0, stream, sums, a.V, chunks,
                       (T*)a.out_dbias);
  LinearProduct p = {};
  p.slab = (float*)(a.workspace + plan.slab);
  p.out_bf16 = sizeof(T) == 2;
  p.M = a.D;
  p.ldo = a.D;
  p.b = direct ? a.grad : dz;
  p.ldb = direct ? a.grad_stride : plan.ldz;
  const LinearArgs given = a;
  hipError_t e = hipGetLastError();
  if (a.out_dhidden != nullptr && e == hipSuccess) {
    if (!linear_rows_aligned(a.weight, a.weight_stride, a.D, dtype))
      pack<T>(a.weight, a.weight_stride, a.V, a.D, a.workspace + plan.weight, plan.ldd, stream);
    p.a = a.weight;
    p.lda = a.weight_stride;
    p.N = a.N;
    p.K = a.V;
    p.out = given.out_dhidden;
    p.shape = linear_shape(kLinDhidden, p.M, p.N, p.K, sizeof(T) == 2);
    e = launch_linear_product(p, kLinDhidden, dtype, stream);
  }
  if (a.out_dweight != nullptr && e == hipSuccess) {
    if (!linear_rows_aligned(a.hidden, a.hidden_stride, a.D, dtype))
      pack<T>(a.hidden, a.hidden_stride, a.N, a.D, a.workspace + plan.hidden, plan.ldd, stream);
    p.a = a.hidden;
    p.lda = a.hidden_stride;
    p.N = a.V;
    p.K = a.N;
    p.out = given.out_dweight;
    p.shape = linear_shape(kLinDweight, p.M, p.N, p.K, sizeof(T) == 2);
    e = launch_linear_product(p, kLinDweight, dtype, stream);
  }
  return e;
}

}  // namespace

bool linear_rows_aligned(const void* p, int64_t stride, int64_t columns, int dtype) {
  // a tile's rows lie within 2^31 bytes
  const int64_t each = dtype == ARCS_DTYPE_BF16 ? 8 : 4, most = int64_t(1) << (dtype == ARCS_DTYPE_BF16 ? 22 : 21);
  return ((uintptr_t)p & 15u) == 0 && stride % each == 0 && columns % each == 0 && stride < most;
}

LinearPlan linear_plan(int64_t N, int64_t V, int64_t D, int dtype, bool aligned, bool backward) {
  const bool bf16 = dtype == ARCS_DTYPE_BF16;
  const int64_t each = bf16 ? 8 : 4, E = bf16 ? 2 : 4;
  LinearPlan p = {};
  p.ldd = tiles(D, each) * each;
  p.ldz = tiles(V, 8) * 8;  // linear_dz_kernel writes 8 columns at a time
  p.chunk_rows = N <= 16 * 256 ? 16 : tiles(N, 256);
  if (!backward && N <= kLinearFewRows) return p;
  size_t at = 0;
  auto part = [&](size_t bytes) {
    const size_t here = at;
    at += bytes;
    return here;
  };
  if (!aligned) {
    p.hidden = part(padded(N * p.ldd * E));
    p.weight = part(padded(V * p.ldd * E));
  }
  size_t slab;
  if (backward) {
    p.dz = part(padded(N * p.ldz * E));
    p.dbias = part(padded(tiles(N, p.chunk_rows) * V * 4));
    const size_t dh = slab_bytes(kLinDhidden, D, N, V, bf16), dw = slab_bytes(kLinDweight, D, V, N, bf16);
    slab = dh > dw ? dh : dw;
  } else {
    slab = slab_bytes(kLinForward, V, N, p.ldd, bf16);
  }
  p.slab = part(slab);
  p.total = at;
  return p;
}

hipError_t launch_linear(LinearArgs a, int dtype, bool aligned, hipStream_t stream) {
  return dtype == ARCS_DTYPE_BF16 ? forward<__bf16>(a, dtype, aligned, stream) : forward<float>(a, dtype, aligned, stream);
}

hipError_t launch_linear_backward(LinearArgs a, int dtype, bool aligned, hipStream_t stream) {
  return dtype == ARCS_DTYPE_BF16 ? backward<__bf16>(a, dtype, aligned, stream) : backward<float>(a, dtype, aligned, stream);
}

}  // namespace arcs
