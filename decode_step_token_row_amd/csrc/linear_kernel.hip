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
// A workgroup makes 16 R columns of the output for all rows: its waves take blocks of 128 bytes of k
// in turn, weights and hidden states straight from memory to registers (a line of each of
// 16 weight rows in two loads, 16 bytes a lane), U blocks in flight, and their sums meet in LDS.
// Reading the weights bounds it: one row x 32,000 x 2,048 takes 22.5 to 24 us (131 MB, 5.6 TB/s; a
// copy reaches 4.8 read and written), one row x 129,280 x 4,096 168 (6.3 TB/s); eight rows x 4,096
// x 4,096 take 9.8 to 10.3 us, of which about 4 are a launch with next to no work.  float32 takes
// twice the bytes: 54 us for the first (4.8 TB/s), 19 for the last.  Two, four and eight blocks in
// flight, bfloat16: 27.7, 24.2 and 29.9 us for the first; asked for half a line at a time and four
// steps ahead it took 27.9.
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

template <typename T, int U, int R>
__global__ __launch_bounds__(kFewWaves * 64) void linear_few_kernel(LinearArgs a) {
  constexpr int E = 16 / sizeof(T), kBlock = 8 * E;  // elements of a load, and of a block of k
  __shared__ float part[kFewWaves][R][16][17];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t v0 = (int64_t)blockIdx.x * (16 * R);
  const int r = lane & 15, q = lane >> 4;
  // rows past the last one repeat it, and are not stored
  const int64_t n = r < a.N ? r : a.N - 1;
  const T* h = (const T*)a.hidden + n * a.hidden_stride;
  const T* w[R];
  f32x4 acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t v = v0 + i * 16 + r;
    w[i] = (const T*)a.weight + (v < a.V ? v : a.V - 1) * a.weight_stride;
    acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int blocks = (int)(a.D / kBlock);  // whole ones
  for (int b0 = wave; b0 < blocks; b0 += kFewWaves * U) {
    u32x4 x[U][R][2], y[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * kFewWaves;
      if (b >= blocks) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < R; ++i) x[u][i][t] = load16(w[i] + b * kBlock + t * 4 * E + q * E);
        y[u][t] = load16(h + b * kBlock + t * 4 * E + q * E);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b0 + u * kFewWaves >= blocks) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] = few_product<T>(x[u][i][t], y[u][t], acc[i]);
    }
  }
  // what is left of k, by the wave whose turn it is
  if (wave == blocks % kFewWaves) {
    for (int64_t k = (int64_t)blocks * kBlock; k < a.D; k += 4 * E)
#pragma unroll
      for (int i = 0; i < R; ++i) acc[i] = few_product<T>(few_load(w[i], k + q * E, a.D), few_load(h, k + q * E, a.D), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][i][q * 4 + e][r] = acc[i][e];
  __syncthreads();
  // thread: column tid % (16 R) of row tid / (16 R)
  const int c = tid % (16 * R), row = tid / (16 * R);
  if (row >= a.N || v0 + c >= a.V) return;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < kFewWaves; ++i) z += part[i][c / 16][c % 16][row];
  if (a.bias != nullptr) z += widen(((const T*)a.bias)[v0 + c]);
  if (a.out_pre != nullptr) ((T*)a.out_pre)[row * a.V + v0 + c] = (T)z;
  float y[1] = {z};
  act_values(y, a.act, a.cap, a.inv_cap);
  if (a.residual != nullptr) y[0] += widen(((const T*)a.residual)[row * a.residual_stride + v0 + c]);
  if (a.out_bf16) ((__bf16*)a.out)[row * a.out_stride + v0 + c] = (__bf16)y[0];
  else ((float*)a.out)[row * a.out_stride + v0 + c] = y[0];
}

// ---------------------------------------------------------------------------
// backward: dz and the columns' sums
// ---------------------------------------------------------------------------
// A workgroup has 256 columns of ROWS * 8 rows: a thread 8 columns of ROWS rows, all loaded at
// once.  Reading grad_out and z and writing dz bounds it, and the activation's slope is close behind: 4,096 x
// 4,096 in bfloat16 takes 23 us with silu (100 MB; 54 with rows one after the other and the library's
// exp and division), 1,037 x 5,003 with gelu by tanh 14.  dz is rounded to T, as the matrix instructions
// of bfloat16 take both operands in it and float32's run at a tenth of their rate, and z was in the forward
// pass, as that halves what is kept between the two: the gradients are 0.0024 from the exact ones in the
// norm, 0.0023 were z in float32, and 0.0017 with nothing rounded but themselves.  The sums take dz
// before it is rounded to T; a workgroup's meet in LDS.  dz may be NULL (only dbias is wanted, or
// grad_out is dz as it is), and so may the sums.
template <typename T, typename G, int ROWS>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearArgs a, T* dz, int64_t ldz, float* sums, unsigned across) {
  __shared__ __align__(16) float part[8][256];
  const int tid = threadIdx.x, c = (tid & 31) * 8, r = tid >> 5;
  const unsigned down = blockIdx.x / across;  // more than a grid's y takes
  const int64_t v0 = (int64_t)(blockIdx.x - down * across) * 256, v = v0 + c;
  const int left = (int)(a.V - v < 8 ? a.V - v : 8);  // <= 0 past V
  const int64_t n0 = (int64_t)down * (ROWS * 8) + r;
  Raw8<G> g[ROWS];
  Raw8<T> z[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t n = n0 + i * 8;
    const int have = n < a.N ? left : 0;
    load_raw(g[i], (const G*)a.grad + n * a.grad_stride + v, have);
    if (a.act != ARCS_ACT_NONE) load_raw(z[i], (const T*)a.pre + n * a.V + v, have);
  }
  float sum[8] = {};
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float x[8];
    widen_raw(g[i], x);
    if (a.act != ARCS_ACT_NONE) {
      float y[8];
      widen_raw(z[i], y);
      act_slopes(x, y, a.act, a.inv_cap);  // past V both are 0
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += x[e];
    const int64_t n = n0 + i * 8;
    if (dz != nullptr && n < a.N && left > 0) store_some<T, 8>(dz + n * ldz + v, 8, x);  // zeros past V, up to ldz
  }
  if (sums == nullptr) return;
  *(f32x4*)&part[r][c] = f32x4{sum[0], sum[1], sum[2], sum[3]};
  *(f32x4*)&part[r][c + 4] = f32x4{sum[4], sum[5], sum[6], sum[7]};
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += part[i][tid];
  if (v0 + tid < a.V) sums[down * a.V + v0 + tid] = s;
}

// The chunks' sums added up, in an order of their numbers.
template <typename T>
__global__ __launch_bounds__(256) void linear_dbias_kernel(const float* sums, int64_t V, int64_t chunks, T* out) {
  __shared__ double part[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t v = (int64_t)blockIdx.x * 16 + c;
  double s = 0.0;
  if (v < V) {
#pragma unroll 8
    for (int64_t i = g; i < chunks; i += 16) s += (double)sums[i * V + v];
  }
  part[g][c] = s;
  __syncthreads();
  if (g != 0 || v >= V) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += part[i][c];
  out[v] = (T)(float)s;
}

// Rows of `columns` elements to rows of ld, zeros behind them.
template <typename T>
__global__ __launch_bounds__(256) void linear_pack_kernel(const T* from, int64_t stride, int64_t rows, int64_t columns, T* to,
                                                          int64_t ld) {
  constexpr int kEach = 16 / sizeof(T);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* p = from + row * stride;
    for (int64_t c = threadIdx.x * kEach; c < ld; c += 256 * kEach) {
      const int64_t left = columns - c;
      float v[kEach];
      load_some<T, kEach>(p + c, (int)(left < kEach ? left > 0 ? left : 0 : kEach), v);
      store_some<T, kEach>(to + row * ld + c, kEach, v);
    }
  }
}

namespace {

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
size_t padded(int64_t bytes) { return (size_t)((bytes + 255) / 256 * 256); }

// Rows of a workgroup of linear_dz_kernel: 32, or 8 where that leaves compute units without
// work (with 8 below 1,024 instead of 512 workgroups of 32, 2,000 x 3,000 13 us instead of 11 and
// 1,037 x 5,003 11.0 instead of 11.6, sums included).
int64_t dz_chunk_rows(int64_t N, int64_t V) { return tiles(N, 32) * tiles(V, 256) < 512 ? 8 : 32; }

size_t slab_bytes(int mode, int64_t M, int64_t N, int64_t K, bool bf16) {
  const LinearShape s = linear_shape(mode, M, N, K, bf16);
  if (s.workers == 0) return 0;
  return padded((s.workers + tiles(M, s.columns) * tiles(N, s.rows)) * s.columns * s.rows * 4);
}

template <typename T>
void pack(const void*& rows, int64_t& stride, int64_t count, int64_t columns, char* to, int64_t ld, hipStream_t stream) {
  // a launch holds fewer than 2^32 threads, the head's 2^24 rows have as many
  const int64_t blocks = count < (int64_t(1) << 20) ? count : int64_t(1) << 20;
  hipLaunchKernelGGL(linear_pack_kernel<T>, dim3((unsigned)blocks), dim3(256), 0, stream, (const T*)rows, stride, count,
                     columns, (T*)to, ld);
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
    // More rows read the hidden states for fewer columns at a time more often, few columns leave
    // compute units without work: 16 rows x 129,280 x 4,096 210 us with 32 columns a workgroup and
    // 248 with 16, 8 x 32,000 x 1,001 28 and 33, but one row x 129,280 193 and 168 and 8 x 4,096 x
    // 4,096 13.6 and 10.2.
    const dim3 threads(kFewWaves * 64);
    if (a.N > 4 && a.V >= 16384)
      hipLaunchKernelGGL((linear_few_kernel<T, 4, 2>), dim3((unsigned)tiles(a.V, 32)), threads, 0, stream, a);
    else
      hipLaunchKernelGGL((linear_few_kernel<T, 4, 1>), dim3((unsigned)tiles(a.V, 16)), threads, 0, stream, a);
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
  p.inv_cap = a.inv_cap;
  return launch_linear_product(p, kLinForward, dtype, stream);
}

template <typename T, typename G>
void launch_dz(const LinearArgs& a, T* dz, int64_t ldz, float* sums, int64_t chunk_rows, hipStream_t stream) {
  const unsigned across = (unsigned)tiles(a.V, 256);
  // below 2^24 workgroups, whose threads a launch holds: as many would be for 2^37 elements of grad_out and dz each
  const dim3 grid((unsigned)(across * tiles(a.N, chunk_rows)));
  if (chunk_rows == 8) hipLaunchKernelGGL((linear_dz_kernel<T, G, 1>), grid, dim3(256), 0, stream, a, dz, ldz, sums, across);
  else hipLaunchKernelGGL((linear_dz_kernel<T, G, 4>), grid, dim3(256), 0, stream, a, dz, ldz, sums, across);
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
    if (a.grad_bf16) launch_dz<T, __bf16>(a, dz, plan.ldz, sums, plan.chunk_rows, stream);
    else launch_dz<T, float>(a, dz, plan.ldz, sums, plan.chunk_rows, stream);
  }
  if (sums != nullptr)
    hipLaunchKernelGGL(linear_dbias_kernel<T>, dim3((unsigned)tiles(a.V, 16)), dim3(256), 0, stream, sums, a.V, chunks,
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

hipError_t launch_linear_product(const LinearProduct& p, int mode, int dtype, hipStream_t stream) {
  const bool bf16 = dtype == ARCS_DTYPE_BF16;
  if (mode == kLinForward) return bf16 ? launch_linear_forward_bf16(p, stream) : launch_linear_forward_f32(p, stream);
  if (mode == kLinDhidden) return bf16 ? launch_linear_dhidden_bf16(p, stream) : launch_linear_dhidden_f32(p, stream);
  return bf16 ? launch_linear_dweight_bf16(p, stream) : launch_linear_dweight_f32(p, stream);
}

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
  p.chunk_rows = dz_chunk_rows(N, V);
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
