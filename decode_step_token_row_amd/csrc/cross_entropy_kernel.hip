// Linear cross entropy: row list, reductions and the general matrix kernel.
//
// The general kernel runs every alignment and size: operands are widened to
// float32 on their way into LDS and multiplied with the float32 matrix
// instruction, so its products are those of float32 arithmetic.  Rows on the
// 16-byte grid go to cross_entropy_mfma.hip instead.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cross_entropy.hpp"
#include "cross_entropy_device.hpp"
#include "launch.hpp"

namespace arcs {

// ---------------------------------------------------------------------------
// The row list.  One workgroup: rows keep their order, so sums over rows do
// not depend on timing.
// ---------------------------------------------------------------------------
constexpr int kPrepNT = 1024;

template <bool BACKWARD>
__global__ __launch_bounds__(kPrepNT) void ce_prep_kernel(CeArgs a) {
  __shared__ int s_count[kPrepNT / kWave];
  __shared__ float s_max[kPrepNT / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float gmax = 1.0f;
  if (BACKWARD) {
    float m = 0.0f;
    for (int64_t n = tid; n < a.N; n += kPrepNT) {
      int32_t t;
      float T;
      if (ce_row_kind(a, n, t, T) != 0) continue;
      const float g = fabsf(a.grad_loss[n] / T);
      if (g < __builtin_inff() && g > m) m = g;
    }
    m = wave_max_f32(m);
    if (lane == 0) s_max[wave] = m;
    __syncthreads();
    for (int w = 0; w < kPrepNT / kWave; ++w) m = fmaxf(m, s_max[w]);
    if (m > 0.0f) gmax = m;
  }
  int base = 0;
  for (int64_t n0 = 0; n0 < a.N; n0 += kPrepNT) {
    const int64_t n = n0 + tid;
    int32_t t = 0;
    float T = 1.0f;
    const int k = n < a.N ? ce_row_kind(a, n, t, T) : 1;
    const uint64_t mask = __ballot(k == 0);
    __syncthreads();  // the last round's counts have been read
    if (lane == 0) s_count[wave] = __popcll(mask);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kPrepNT / kWave; ++w) {
      const int c = s_count[w];
      before += w < wave ? c : 0;
      all += c;
    }
    const int at = base + before + __popcll(mask & ((1ull << lane) - 1ull));
    base += all;
    if (n >= a.N) continue;
    if (k == 0) {
      CeRow r = {};
      if (BACKWARD) {
        r = ce_row(a, n, t, T, gmax);
      } else {
        r.row = (int32_t)n;
        r.target = t;
        r.a = kLog2e / T;
      }
      a.rows[at] = r;
    }
    if (BACKWARD) {
      a.place[n] = k == 0 ? at : -1;
    } else {
      if (k != 0) {
        const float v = k < 0 ? 0.0f : __builtin_nanf("");
        a.out_loss[n] = v;
        a.out_lse[n] = v;
      }
      if (a.out_status) a.out_status[n] = k < 0 ? 0 : k;
    }
  }
  if (tid == 0) {
    a.head->count = base;
    a.head->gmax = gmax;
  }
}

// ---------------------------------------------------------------------------
// Forward: the slices of a row joined, one workgroup per row (listed, or direct).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void ce_combine_kernel(CeArgs a, int direct) {
  __shared__ float2 s_part[4];
  const int64_t i = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t n = i;
  float scale;  // as the tiles had it
  if (direct) {
    int32_t target;
    float T;
    const int k = ce_row_kind(a, i, target, T);
    if (tid == 0 && a.out_status) a.out_status[i] = k < 0 ? 0 : k;
    if (k != 0) {
      if (tid == 0) a.out_loss[i] = a.out_lse[i] = k < 0 ? 0.0f : __builtin_nanf("");
      return;
    }
    scale = kLog2e / T;
  } else {
    if (i >= a.head->count) return;
    n = a.rows[i].row;
    scale = a.rows[i].a;
  }
  // each lane's slices, then the lanes', then the waves' (the first wave goes over the four)
  const float2* p = a.partial + i * a.slices;
  float m = -__builtin_inff(), sum = 0.0f;
  auto join = [&](float m2, float s2) {
    const float top = fmaxf(m, m2), z = finite_or_zero(top);
    sum = fmaf(sum, exp2_fast(m - z), s2 * exp2_fast(m2 - z));
    m = top;
  };
#pragma unroll 4
  for (int64_t s = tid; s < a.slices; s += 256) {
    const float2 q = p[s];
    join(q.x, q.y);
  }
  for (int o = 32; o > 0; o >>= 1) join(__shfl_xor(m, o, kWave), __shfl_xor(sum, o, kWave));
  if (lane == 0) s_part[wave] = make_float2(m, sum);
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < 4; ++w) join(s_part[w].x, s_part[w].y);
    // joined in 64 bits: each result is rounded once, at its own size, not at the maximum's
    int e;
    const float f = frexpf(sum, &e);
    const double l2 = (double)m + (double)e + (double)log2f(f);
    a.out_lse[n] = (float)(l2 * 0.69314718055994530942);
    a.out_loss[n] = (float)((l2 - (double)a.dtarget[i] * (double)scale) * 0.69314718055994530942);
  }
}

// ---------------------------------------------------------------------------
// Backward: dhidden rows from the slabs, and zeros for rows not listed.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(256) void ce_dhidden_kernel(CeArgs a) {
  const int64_t n = blockIdx.x, d = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (d >= a.D) return;
  const int i = a.place[n];
  float v = 0.0f;
  if (i >= 0) {
    const float* p = a.slab + (int64_t)i * a.D + d;
    const int64_t step = a.N * a.D;
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) v += p[s * step];
    v *= a.head->gmax;
  }
  if (BF16) ((__bf16*)a.out_dhidden)[n * a.D + d] = (__bf16)v;
  else ((float*)a.out_dhidden)[n * a.D + d] = v;
}

// ---------------------------------------------------------------------------
// The general matrix kernel: C[m, n] = sum_k A[m, k] B[n, k] on 128 x 128
// tiles, four waves of 64 x 64 (two by two 32x32x2 float32 products), 16 k at
// a time through two LDS buffers.  Elements are loaded one by one (rows lie
// anywhere), which bounds it; three workgroups a compute unit hide some of
// that.  Against the tile kernel, 1,024 rows x 50,001 x 1,001 and x 1,000: bfloat16
// 2,251 and 159 us forward, 5,186 and 414 backward, float32 1,575 and 823, 4,675 and
// 2,391.
// ---------------------------------------------------------------------------
constexpr int kGenTile = 128, kGenK = 16, kGenLd = kGenTile + 4;

// Eight consecutive elements of a row from `at` on, zeros from `len` on.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t at, int64_t len, float out[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = row != nullptr && at + e < len ? (float)row[at + e] : 0.0f;
}

template <typename T, int MODE>
__global__ __launch_bounds__(256, 3) void ce_general_kernel(CeArgs a, CePiece pc) {
  __shared__ float sA[2][kGenK * kGenLd], sB[2][kGenK * kGenLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t count = a.head->count;
  constexpr bool kLogits = MODE == kCeStats || MODE == kCeDs;
  const int64_t M = kLogits ? pc.len : a.D;
  const int64_t N = MODE == kCeDweight ? pc.len : count;
  const int64_t m0 = (int64_t)(MODE == kCeDweight ? blockIdx.y : blockIdx.x) * kGenTile;
  const int64_t n0 = (int64_t)(MODE == kCeDweight ? blockIdx.x : blockIdx.y) * kGenTile;
  if (n0 >= N) return;
  int64_t k_lo = 0, k_hi = kLogits ? a.D : MODE == kCeDhidden ? pc.len : count;
  if (MODE == kCeDhidden) {  // this split's part of the piece
    const int64_t part = ((k_hi + a.splits - 1) / a.splits + kGenK - 1) / kGenK * kGenK;
    k_lo = part * blockIdx.z;
    k_hi = k_lo + part < k_hi ? k_lo + part : k_hi;
  }
  const T* W = (const T*)a.weight + pc.v0 * a.weight_stride;
  const T* H = (const T*)a.hidden;
  const float* S = (const float*)a.ds;
  constexpr bool kAOuter = !kLogits, kBOuter = MODE == kCeDweight;  // k is the row index in memory

  // this thread's eight elements of a tile: along k of one m, or along m of one k
  const int in_r = tid >> 1, in_k = (tid & 1) * 8;
  const int out_k = tid >> 4, out_m = (tid & 15) * 8;
  const int64_t bn = n0 + in_r;
  const T* hrow = kLogits && bn < N ? H + (int64_t)a.rows[bn].row * a.hidden_stride : nullptr;
  // row, place in it and its length of this thread's eight elements at k0
  auto a_row = [&](int64_t k0, int64_t& at, int64_t& len) -> const T* {
    at = kAOuter ? m0 + out_m : k0 + in_k;
    len = kAOuter ? M : k_hi;
    if (!kAOuter) return m0 + in_r < M ? W + (m0 + in_r) * a.weight_stride : nullptr;
    const int64_t k = k0 + out_k;
    if (k >= k_hi) return nullptr;
    return MODE == kCeDhidden ? W + k * a.weight_stride : H + (int64_t)a.rows[k].row * a.hidden_stride;
  };
  auto s_row = [&](int64_t k0, int64_t& at, int64_t& len) -> const float* {  // dz: zeros from the piece's end on
    at = kBOuter ? n0 + out_m : k0 + in_k;
    len = a.ds_ld;
    const int64_t r = kBOuter ? k0 + out_k : bn;
    return r < (kBOuter ? k_hi : N) ? S + r * a.ds_ld : nullptr;
  };
  auto put = [&](float* s, bool outer, const float v[8]) {
    if (outer) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[out_k * kGenLd + out_m + e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[(in_k + e) * kGenLd + in_r] = v[e];
    }
  };
  float va[8], vb[8];
  auto load = [&](int64_t k0) {
    int64_t at, len;
    const T* ra = a_row(k0, at, len);
    load8<T>(ra, at, len, va);
    if constexpr (kLogits) {
      load8<T>(hrow, k0 + in_k, k_hi, vb);
    } else {
      const float* rs = s_row(k0, at, len);
      load8<float>(rs, at, len, vb);
    }
  };
  auto store = [&](int to) {
    put(sA[to], kAOuter, va);
    put(sB[to], kBOuter, vb);
  };

  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  const int fr = lane & 31, fk = lane >> 5;

  if (k_lo < k_hi) {
    load(k_lo);
    store(0);
  }
  __syncthreads();
  int at = 0;
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += kGenK, at ^= 1) {
    const bool more = k0 + kGenK < k_hi;
    if (more) load(k0 + kGenK);
#pragma unroll
    for (int kk = 0; kk < kGenK; kk += 2) {
      float fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = sA[at][(kk + fk) * kGenLd + wm + i * 32 + fr];
        fb[i] = sB[at][(kk + fk) * kGenLd + wn + i * 32 + fr];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    if (more) store(at ^ 1);
    __syncthreads();
  }

  // a lane holds column n = lane % 32 of each product, rows 8 (r / 4) + 4 (lane / 32) + r % 4
  auto row_of = [&](int i, int r) { return m0 + wm + i * 32 + 8 * (r >> 2) + 4 * fk + (r & 3); };
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = n0 + wn + j * 32 + fr;
    if (kLogits) {
      CeRow row;
      row.target = -1;
      row.a = row.c = row.lse2 = row.rest = 0.0f;
      if (n < N) row = a.rows[n];
      if (MODE == kCeStats) {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int64_t v = row_of(i, r);
            const float dot = acc[i][j][r], y = dot * row.a;
            if (v < M) {
              m = fmaxf(m, y);
              if (pc.v0 + v == row.target) a.dtarget[n] = dot;
            }
          }
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        const float mz = finite_or_zero(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (row_of(i, r) < M) sum += exp2_fast(fmaf(acc[i][j][r], row.a, -mz));
        sum += __shfl_xor(sum, 32, kWave);
        // a slice is a wave's 64 rows of the tile
        if (fk == 0 && n < N) a.partial[n * a.slices + 2 * (int64_t)blockIdx.x + (wave & 1)] = make_float2(m, sum);
      } else if (n < N) {
        float* out = (float*)a.ds + n * a.ds_ld;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int64_t v = row_of(i, r);
            float p = exp2_fast(fmaf(acc[i][j][r], row.a, -row.lse2)) * row.rest;
            if (pc.v0 + v == row.target) p -= 1.0f;
            out[v] = v < M ? p * row.c : 0.0f;  // ds_ld is a multiple of the tile
          }
      }
    } else if (n < N) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t m = row_of(i, r);
          if (m >= M) continue;
          if (MODE == kCeDhidden) {
            float* out = a.slab + ((int64_t)blockIdx.z * a.N + n) * a.D + m;
            *out = pc.first ? acc[i][j][r] : *out + acc[i][j][r];
          } else {
            ((T*)a.out_dweight)[(pc.v0 + n) * a.D + m] = (T)(acc[i][j][r] * a.head->gmax);
          }
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
namespace {

constexpr int64_t kMaxTiles = int64_t(1) << 23;  // of a launch (its threads fit 32 bits)
constexpr int64_t kPieceBytes = int64_t(1) << 28;  // dz of one piece, about
constexpr int64_t kMaxPiece = int64_t(1) << 24;  // 64 rows of dz lie within 2^31 bytes

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

}  // namespace

CePlan cross_entropy_plan(int64_t N, int64_t V, int64_t D, int dtype, bool backward) {
  CePlan p = {};
  p.fits = N > 0 && V > 0 && D > 0 && tiles(N, kGenTile) <= 65535 &&
           (unsigned __int128)tiles(N, kGenTile) * (unsigned __int128)tiles(V > D ? V : D, kGenTile) <= kMaxTiles;
  if (!p.fits) return p;
  unsigned __int128 at = sizeof(CeHeader);
  auto take = [&](unsigned __int128 bytes) {
    const size_t off = (size_t)at;
    at += (bytes + 255) / 256 * 256;
    return off;
  };
  typedef unsigned __int128 u128;
  const bool bf16 = dtype == ARCS_DTYPE_BF16;
  p.rows = take((u128)N * sizeof(CeRow));
  p.hc = take((u128)N * D * (bf16 ? 2 : 4));
  p.splits = 1;
  if (!backward) {
    p.slices = 8 * tiles(V, 256);
    p.dtarget = take((u128)N * 4);
    p.partial = take((u128)N * p.slices * sizeof(float2));
  } else {
    // dz of a piece: bfloat16 in the matrix kernels, float32 in the general one
    int64_t piece = kPieceBytes / 4 / N / 256 * 256;
    if (piece < 1024) piece = 1024;
    if (piece > kMaxPiece) piece = kMaxPiece;
    const int64_t whole = tiles(V, 256) * 256;
    p.piece = piece < whole ? piece : whole;
    const int64_t t = tiles(N, kGenTile) * tiles(D, kGenTile);
    int64_t splits = 512 / t, most = p.piece / 512;
    if (splits > most) splits = most;
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.place = take((u128)N * 4);
    p.ds = take((u128)N * p.piece * 4);
    // dhidden's partial sums: the general kernel's splits or the matrix kernels' parts
    u128 slab = (u128)p.splits * N * D * 4;
    const int64_t rows = ce_rows_of_tile(N, bf16), columns = ce_columns_of_tile(N, bf16);
    // as many workgroups as the compute units hold, unless that leaves them less than 512 of k
    const int64_t jobs = tiles(N, rows) * tiles(D, columns), share = jobs * tiles(p.piece, 512), full = columns == 128 ? 512 : 256;
    p.workers = (int)(share < full ? tiles(share, 8) * 8 : full);
    const u128 parts = (u128)(p.workers + jobs) * rows * columns * 4;
    if (parts > slab) slab = parts;
    p.slab = take(slab);
  }
  if (at > (u128)INT64_MAX) p.fits = false;
  p.total = (size_t)at;
  return p;
}

void launch_cross_entropy_prep(const CeArgs& a, bool backward, hipStream_t stream) {
  if (backward) hipLaunchKernelGGL(ce_prep_kernel<true>, dim3(1), dim3(kPrepNT), 0, stream, a);
  else hipLaunchKernelGGL(ce_prep_kernel<false>, dim3(1), dim3(kPrepNT), 0, stream, a);
}

void launch_cross_entropy_combine(const CeArgs& a, bool direct, hipStream_t stream) {
  hipLaunchKernelGGL(ce_combine_kernel, dim3((unsigned)a.N), dim3(256), 0, stream, a, direct ? 1 : 0);
}

void launch_cross_entropy_dhidden(const CeArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)a.N, (unsigned)tiles(a.D, 256));
  if (bf16) hipLaunchKernelGGL(ce_dhidden_kernel<true>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(ce_dhidden_kernel<false>, grid, dim3(256), 0, stream, a);
}

template <typename T>
static hipError_t launch_general(CeArgs a, bool backward, hipStream_t stream) {
  const dim3 block(256);
  const unsigned nt = (unsigned)tiles(a.N, kGenTile), dt = (unsigned)tiles(a.D, kGenTile);
  if (!backward) {
    const CePiece pc = {0, a.V, 1, 0, 0};
    a.slices = 2 * tiles(a.V, kGenTile);
    hipLaunchKernelGGL((ce_general_kernel<T, kCeStats>), dim3((unsigned)tiles(a.V, kGenTile), nt), block, 0, stream, a, pc);
    launch_cross_entropy_combine(a, false, stream);
    return hipGetLastError();
  }
  for (int64_t v0 = 0; v0 < a.V; v0 += a.ds_ld) {
    const CePiece pc = {v0, a.V - v0 < a.ds_ld ? a.V - v0 : a.ds_ld, v0 == 0, 0, 0};
    const unsigned vt = (unsigned)tiles(pc.len, kGenTile);
    hipLaunchKernelGGL((ce_general_kernel<T, kCeDs>), dim3(vt, nt), block, 0, stream, a, pc);
    if (a.out_dhidden)
      hipLaunchKernelGGL((ce_general_kernel<T, kCeDhidden>), dim3(dt, nt, (unsigned)a.splits), block, 0, stream, a, pc);
    if (a.out_dweight)
      hipLaunchKernelGGL((ce_general_kernel<T, kCeDweight>), dim3(vt, dt), block, 0, stream, a, pc);
  }
  if (a.out_dhidden) launch_cross_entropy_dhidden(a, sizeof(T) == 2, stream);
  return hipGetLastError();
}

hipError_t launch_cross_entropy(const CeArgs& a, int dtype, bool backward, hipStream_t stream) {
  if (cross_entropy_matrix_path(a, dtype)) return launch_cross_entropy_matrix(a, dtype, backward, stream);
  launch_cross_entropy_prep(a, backward, stream);
  return dtype == ARCS_DTYPE_BF16 ? launch_general<__bf16>(a, backward, stream) : launch_general<float>(a, backward, stream);
}

}  // namespace arcs
