// Head logits from 4-bit weights with group scales.
//
//   logits[b, v] = sum_g scale[v, g] * sum_{d in g} (q[v, d] - zero[v, g]) hidden[b, d]
//
// q is two weights a byte, the lower d in the low nibble.  The products run
// on the bfloat16 matrix instruction with the batch as its rows and 16
// vocabulary rows as its columns, so a lane needs the scale of one row only.
// A nibble becomes an exact bfloat16 with an offset: 16 + q by an AND and an
// OR on two weights at a time (0x4180 is 16.0 and bit 3 of its mantissa is 1),
// or, with zero points, 48 + q - z by an AND and an addition of the row's
// constant (0x4200 is 32.0, bit 2 is 1).  The offset's part of a group's sum,
// 24 or 48 times the sum of the hidden state over the group, is what the
// product's accumulator starts from, negated:
//   sum (q - z) h = -48 sum h + sum (48 + q - z) h.
// Scales are applied to the group's float32 sums, so no weight is rounded.
//
// Batches of at most 16 rows take one launch: hidden states go through LDS, four
// steps of 128 k at a time in two buffers, and weights from memory to registers
// four steps ahead.  Larger batches have the hidden states prepared first, in the
// workspace: in the nibbles' order and as the LDS holds them, with the groups'
// sums beside them, so that a step is a plain copy to LDS that takes no registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "arcs.h"
#include "device_common.hpp"
#include "launch.hpp"
#include "lds_load.hpp"

namespace arcs {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kW4FewRows = 16;
constexpr int kW4Step = 128;  // k of one step: 16 bytes of a weight row in each of four lanes

// Eight nibbles as bfloat16, in the order 0 4 1 5 2 6 3 7: 16 + q, or with zero
// points (add = 0x42004200 + 4 (16 - z) in both halves) 48 + q - z.
template <bool ZERO>
__device__ __forceinline__ bf16x8 w4_unpack(uint32_t w, uint32_t add) {
  u32x4 d;
  if (ZERO) {
    d[0] = ((w << 2) & 0x003C003Cu) + add;
    d[1] = ((w >> 2) & 0x003C003Cu) + add;
    d[2] = ((w >> 6) & 0x003C003Cu) + add;
    d[3] = ((w >> 10) & 0x003C003Cu) + add;
  } else {
    d[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    d[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    d[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    d[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
  }
  return __builtin_bit_cast(bf16x8, d);
}

// Eight bfloat16 in the same order.
__device__ __forceinline__ u32x4 w4_order(u32x4 x) {
  u32x4 d;
  d[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
  d[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
  d[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
  d[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
  return d;
}

// w[i] of lane group j <-> w[j] of lane group i (groups of 16 lanes).
__device__ __forceinline__ u32x4 w4_turn(u32x4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// GROUP 128: a lane's 16 bytes are 32 consecutive k and one product takes 8 of
// each lane group's.  GROUP 32, 64: the 16 bytes are exchanged between the four
// lane groups first, so that a product's 32 k are consecutive and lie in one group.
template <int GROUP, bool ZERO, bool SF32>
struct W4 {
  static constexpr int kGroups = kW4Step / GROUP;           // of a step
  static constexpr int kProducts = 4 / kGroups;             // of 32 k, in a group
  static constexpr bool kTurn = GROUP < 128;
  static constexpr int kScale = SF32 ? 4 : 2;               // bytes of a scale
  static constexpr int kScales = (kGroups * kScale + 3) / 4;  // words of a step's scales
  static constexpr float kOffset = ZERO ? -48.0f : -24.0f;

  // Where lane group j finds the 8 k of product n of a step, in units of 8.
  static __device__ __forceinline__ int chunk(int n, int j) { return kTurn ? n * 4 + j : j * 4 + n; }

  // RT tiles of 16 weight rows: a uniform base, and a lane's row in each.
  template <int RT>
  struct Rows {
    const char *qb, *sb, *zb;
    uint32_t qo[RT], so[RT], zo[RT];
    __device__ __forceinline__ Rows(const W4Args& a, int64_t v0, int r, int j) {
      const int64_t base = v0 < a.V ? v0 : a.V - 1;
      qb = (const char*)a.qweight + base * a.qweight_stride;
      sb = (const char*)a.scales + base * a.scale_stride * kScale;
      zb = (const char*)a.zeros + base * a.zero_stride;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const uint32_t v = (uint32_t)(base + t * 16 + r < a.V ? t * 16 + r : a.V - 1 - base);
        qo[t] = v * (uint32_t)a.qweight_stride + j * 16;
        so[t] = v * (uint32_t)a.scale_stride * kScale;
        zo[t] = v * (uint32_t)a.zero_stride;
      }
    }
  };

  // The weights, scales and zero points of RT tiles over NS steps from one on.
  // All of a row's 64 NS bytes are asked for at once: a line is used while it is
  // in the cache, and a wave's loads keep NS * RT KB on their way.
  template <int RT, int NS>
  struct Part {
    static constexpr int kN = NS * kGroups;                  // scales of a row
    static constexpr int kWords = (kN * kScale + 3) / 4, kZeroWords = (kN + 3) / 4;
    u32x4 w[NS][RT];
    uint32_t s[RT][kWords], z[RT][kZeroWords];

    __device__ __forceinline__ void load(const W4Args& a, const Rows<RT>& rows, int step, int j) {
      const int64_t k = (int64_t)step * kW4Step, first = k / GROUP;
      if (k + NS * kW4Step <= a.D) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int c = 0; c < NS; ++c) w[c][t] = *(const u32x4*)(rows.qb + (k >> 1) + c * 64 + rows.qo[t]);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          __builtin_memcpy(s[t], rows.sb + first * kScale + rows.so[t], kN * kScale);
          if (ZERO) __builtin_memcpy(z[t], rows.zb + first + rows.zo[t], kN);
        }
        return;
      }
      // the row's end
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          w[c][t] = u32x4{0, 0, 0, 0};
          if (k + c * kW4Step + j * 32 < a.D) w[c][t] = *(const u32x4*)(rows.qb + (k >> 1) + c * 64 + rows.qo[t]);
        }
#pragma unroll
        for (int g = 0; g < kWords; ++g) s[t][g] = 0;
#pragma unroll
        for (int g = 0; g < kZeroWords; ++g) z[t][g] = 0;
#pragma unroll
        for (int g = 0; g < kN; ++g) {
          if (k + g * GROUP >= a.D) continue;
          const char* p = rows.sb + (first + g) * kScale + rows.so[t];
          if (SF32) s[t][g] = *(const uint32_t*)p;
          else s[t][g / 2] |= (uint32_t) * (const uint16_t*)p << (g % 2 * 16);
          if (ZERO) z[t][g / 4] |= (uint32_t) * (const uint8_t*)(rows.zb + first + g + rows.zo[t]) << (g % 4 * 8);
        }
      }
    }
    __device__ __forceinline__ float scale(int t, int g) const {
      return SF32 ? __uint_as_float(s[t][g]) : g % 2 ? bf16_hi(s[t][g / 2]) : bf16_lo(s[t][g / 2]);
    }
    __device__ __forceinline__ uint32_t add(int t, int g) const {
      return ZERO ? 0x42404240u - ((z[t][g / 4] >> (g % 4 * 8)) & 15u) * 0x00040004u : 0u;
    }
  };

  // A lane's 8 k of a hidden row: their order, and (in the group's first lane) the group's sum.
  static __device__ __forceinline__ float group_sum(u32x4 v) {
    float s = (bf16_lo(v[0]) + bf16_hi(v[0])) + (bf16_lo(v[1]) + bf16_hi(v[1]));
    s += (bf16_lo(v[2]) + bf16_hi(v[2])) + (bf16_lo(v[3]) + bf16_hi(v[3]));
    s = add_dpp<0xB1>(s);                   // lanes 1 apart
    s = add_dpp<0x4E>(s);                   // 2 apart
    if (GROUP > 32) s = add_dpp<0x141>(s);  // the other four of eight
    if (GROUP > 64) s = add_dpp<0x140>(s);  // the other eight of sixteen
    return kOffset * s;
  }
};

template <int MT, int RT, bool OF32>
__device__ __forceinline__ void w4_write(const W4Args& a, const f32x4 (&total)[MT][RT], int64_t b0, int64_t v0, int r, int j) {
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t v = v0 + t * 16 + r;
    if (v >= a.V) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t row = b0 + m * 16 + j * 4 + e;
        if (row >= a.B) continue;
        if (OF32) ((float*)a.logits)[row * a.row_stride + v] = total[m][t][e];
        else ((__bf16*)a.logits)[row * a.row_stride + v] = (__bf16)total[m][t][e];
      }
  }
}

// ---------------------------------------------------------------------------
// At most 16 rows: four waves of RT * 16 weight rows each.
// ---------------------------------------------------------------------------
constexpr int kW4Stage = 4;  // steps

template <int RT, int GROUP, bool ZERO, bool SF32, bool OF32>
__global__ __launch_bounds__(256, 2) void w4_rows_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, SF32>;
  constexpr int SC = kW4Stage, kRows = 16, kPer = kRows * SC * 16 / 256;
  __shared__ __align__(16) char s_x[2][SC * kRows * 256];
  __shared__ __align__(16) float s_sum[2][SC * K::kGroups][kRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, j = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * (RT * 16);
  const int steps = (int)((a.D + kW4Step - 1) / kW4Step), stages = (steps + SC - 1) / SC;
  const typename K::template Rows<RT> rows(a, v0, r, j);

  // the stage's hidden states: piece p of a thread is 8 k of one row, 64 pieces a row
  u32x4 xr[kPer];
  auto fetch_x = [&](int stage) {
    const int64_t k = (int64_t)stage * SC * kW4Step + lane * 8;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int row = wave + p * 4;
      if (row < a.B) xr[p] = k < a.D ? *(const u32x4*)(a.hidden + row * a.hidden_stride + k) : u32x4{0, 0, 0, 0};
    }
  };
  auto store_x = [&](int stage) {
    char* x = s_x[stage & 1] + (lane >> 4) * (kRows * 256);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int row = wave + p * 4;
      if (row >= a.B) continue;
      const float s = K::group_sum(xr[p]);
      *(u32x4*)(x + row * 256 + (((lane & 15) ^ row) * 16)) = w4_order(xr[p]);
      if (lane % (GROUP / 8) == 0) s_sum[stage & 1][lane / (GROUP / 8)][row] = s;
    }
  };

  typename K::template Part<RT, SC> next;
  f32x4 total[1][RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) total[0][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  fetch_x(0);
  next.load(a, rows, 0, j);
  store_x(0);
  __syncthreads();
  for (int stage = 0; stage < stages; ++stage) {
    typename K::template Part<RT, SC> now = next;
    if (stage + 1 < stages) {
      fetch_x(stage + 1);
      next.load(a, rows, (stage + 1) * SC, j);
    }
    const char* x = s_x[stage & 1];
#pragma unroll
    for (int c = 0; c < SC; ++c) {
      if (c > 0 && stage * SC + c >= steps) break;
#pragma unroll
      for (int t = 0; t < RT; ++t)
        if (K::kTurn) now.w[c][t] = w4_turn(now.w[c][t]);
#pragma unroll
      for (int g = 0; g < K::kGroups; ++g) {
        const int gs = c * K::kGroups + g;
        const f32x4 start = *(const f32x4*)&s_sum[stage & 1][gs][j * 4];
        bf16x8 xf[K::kProducts];
#pragma unroll
        for (int i = 0; i < K::kProducts; ++i)
          xf[i] = *(const bf16x8*)(x + (c * kRows + r) * 256 + ((K::chunk(g * K::kProducts + i, j) ^ r) * 16));
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4 acc = start;
#pragma unroll
          for (int i = 0; i < K::kProducts; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                xf[i], w4_unpack<ZERO>(now.w[c][t][g * K::kProducts + i], now.add(t, gs)), acc, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) total[0][t][e] = fmaf(now.scale(t, gs), acc[e], total[0][t][e]);
        }
      }
    }
    if (stage + 1 < stages) store_x(stage + 1);
    __syncthreads();
  }
  w4_write<1, RT, OF32>(a, total, 0, v0, r, j);
}

// ---------------------------------------------------------------------------
// More rows.  The prepared hidden states of one step are 4096 bytes for every 16
// rows: row x 256 bytes, chunk c of 8 k at c ^ row; rows past B are zeros.  The
// sums are [step][group][row].
// ---------------------------------------------------------------------------
template <int GROUP, bool ZERO>
__global__ __launch_bounds__(256) void w4_prepare_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, false>;
  const int row = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int64_t step = blockIdx.x, tile = blockIdx.y, b = tile * 16 + row, k = step * kW4Step + c * 8;
  u32x4 v = {0, 0, 0, 0};
  if (b < a.B && k < a.D) v = *(const u32x4*)(a.hidden + b * a.hidden_stride + k);
  const float s = K::group_sum(v);
  const int64_t tiles = a.padded_rows / 16;
  *(u32x4*)(a.prepared + (step * tiles + tile) * 4096 + row * 256 + ((c ^ row) * 16)) = w4_order(v);
  if (c % (GROUP / 8) == 0) a.sums[(step * K::kGroups + c / (GROUP / 8)) * a.padded_rows + b] = s;
}

constexpr int kW4Part = 2;  // steps between two barriers

template <int MT, int RT, int WB, int WV, int GROUP, bool ZERO, bool SF32, bool OF32>
__global__ __launch_bounds__(WB* WV * 64, 2) void w4_batch_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, SF32>;
  constexpr int NS = kW4Part, kWaves = WB * WV, kRows = WB * MT * 16;
  constexpr int kLoads = NS * kRows / 4, kPer = kLoads / kWaves;  // of 1024 bytes
  constexpr int kN = NS * K::kGroups;                             // groups of a part
  constexpr int kSumLoads = (kN * kRows * 4 + 1023) / 1024;
  constexpr int kSumAt = NS * kRows * 256, kStage = kSumAt + kSumLoads * 1024;
  static_assert(kSumLoads <= kWaves && kLoads % kWaves == 0, "loads of a part over the waves");
  __shared__ __align__(1024) char lds[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, j = lane >> 4;
  const int wb = wave % WB, wv = wave / WB;
  // blocks go round the eight dies in turn; a die gets neighbouring tiles, the
  // batch's tiles of the same weights one after the other
  const int per = (a.tiles + 7) / 8, at = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= per || at >= a.tiles) return;
  const int64_t b0 = (int64_t)(at % a.batch_tiles) * kRows;
  const int64_t v0 = ((int64_t)(at / a.batch_tiles) * WV + wv) * (RT * 16);
  const int parts = (int)((a.D + NS * kW4Step - 1) / (NS * kW4Step));
  const typename K::template Rows<RT> rows(a, v0, r, j);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(ARCS_LDS char*)lds;
  const int64_t step_x = a.padded_rows * 256;
  const char* px = a.prepared + b0 * 256;
  const char* ps = (const char*)(a.sums + b0);
  constexpr int kSumLanes = kRows / 4;  // lanes of one group's sums
  const int sum_group = (wave * 64 + lane) / kSumLanes;
  const uint32_t sum_off =
      sum_group < kN ? (uint32_t)(sum_group * a.padded_rows * 4 + (wave * 64 + lane) % kSumLanes * 16) : kNoLoad;
  auto issue = [&](int part) {
    const uint32_t to = lds0 + (uint32_t)(part & 1) * kStage;
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      const int load = wave + t * kWaves, step = load / (kRows / 4), in = load % (kRows / 4);
      load_to_lds(to + load * 1024u, (uint32_t)(in * 1024 + lane * 16),
                  buffer_of(px + ((int64_t)part * NS + step) * step_x, kRows * 256));
    }
    if (wave < kSumLoads)
      load_to_lds(to + kSumAt + wave * 1024u, sum_off, buffer_of(ps + (int64_t)part * kN * a.padded_rows * 4, kBufMost));
  };

  f32x4 total[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t) total[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  typename K::template Part<RT, NS> next;
  issue(0);
  next.load(a, rows, 0, j);
  for (int part = 0; part < parts; ++part) {
    wait_loads<0>();  // this part's hidden states are in LDS, its weights in registers
    wait_lds();
    __builtin_amdgcn_s_barrier();
    typename K::template Part<RT, NS> now = next;
    if (part + 1 < parts) {
      issue(part + 1);
      next.load(a, rows, (part + 1) * NS, j);
    }
    const char* x = lds + (part & 1) * kStage;
    const float* sums = (const float*)(x + kSumAt);
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      u32x4 w[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) w[t] = K::kTurn ? w4_turn(now.w[c][t]) : now.w[c][t];
#pragma unroll
      for (int g = 0; g < K::kGroups; ++g) {
        const int gs = c * K::kGroups + g;
        f32x4 acc[MT][RT];
#pragma unroll
        for (int i = 0; i < K::kProducts; ++i) {
          bf16x8 xf[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int row = (wb * MT + m) * 16;
            if (i == 0) {
              const f32x4 start = *(const f32x4*)(sums + gs * kRows + row + j * 4);
#pragma unroll
              for (int t = 0; t < RT; ++t) acc[m][t] = start;
            }
            xf[m] = *(const bf16x8*)(x + (c * kRows + row + r) * 256 + ((K::chunk(g * K::kProducts + i, j) ^ r) * 16));
          }
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const bf16x8 wf = w4_unpack<ZERO>(w[t][g * K::kProducts + i], now.add(t, gs));
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[m], wf, acc[m][t], 0, 0, 0);
          }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[m][t][e] = fmaf(now.scale(t, gs), acc[m][t][e], total[m][t][e]);
        __builtin_amdgcn_sched_barrier(0);  // one group's operands at a time in registers
      }
    }
  }
  w4_write<MT, RT, OF32>(a, total, b0 + wb * MT * 16, v0, r, j);
}

namespace {

// Steps of the prepared hidden states: whole parts, zeros past D.
int64_t w4_steps(int64_t D) { return (D + kW4Part * kW4Step - 1) / (kW4Part * kW4Step) * kW4Part; }

template <int RT, int GROUP, bool ZERO, bool SF32>
void launch_w4_rows(const W4Args& a, bool f32, hipStream_t stream) {
  const dim3 grid((unsigned)((a.V + 64 * RT - 1) / (64 * RT))), block(256);
  if (f32) hipLaunchKernelGGL((w4_rows_kernel<RT, GROUP, ZERO, SF32, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((w4_rows_kernel<RT, GROUP, ZERO, SF32, false>), grid, block, 0, stream, a);
}

template <int MT, int RT, int WB, int WV, int GROUP, bool ZERO, bool SF32>
void launch_w4_batch(W4Args a, bool f32, hipStream_t stream) {
  constexpr int kRows = WB * MT * 16, kCols = WV * RT * 16;
  a.batch_tiles = (int)((a.B + kRows - 1) / kRows);
  const int64_t tiles = (a.V + kCols - 1) / kCols * a.batch_tiles;
  a.tiles = (int)tiles;
  hipLaunchKernelGGL((w4_prepare_kernel<GROUP, ZERO>),
                     dim3((unsigned)w4_steps(a.D), (unsigned)(a.padded_rows / 16)), dim3(256), 0, stream, a);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8)), block(WB * WV * 64);
  if (f32) hipLaunchKernelGGL((w4_batch_kernel<MT, RT, WB, WV, GROUP, ZERO, SF32, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((w4_batch_kernel<MT, RT, WB, WV, GROUP, ZERO, SF32, false>), grid, block, 0, stream, a);
}

template <int GROUP, bool ZERO, bool SF32>
void launch_w4_typed(W4Args a, bool f32, hipStream_t stream) {
  if (a.B <= kW4FewRows) {
    if (a.V <= 65536) launch_w4_rows<1, GROUP, ZERO, SF32>(a, f32, stream);
    else launch_w4_rows<2, GROUP, ZERO, SF32>(a, f32, stream);
  } else if (a.B <= 32) {
    launch_w4_batch<2, 4, 1, 4, GROUP, ZERO, SF32>(a, f32, stream);
  } else if (a.B <= 64) {
    launch_w4_batch<4, 2, 1, 8, GROUP, ZERO, SF32>(a, f32, stream);
  } else {
    launch_w4_batch<8, 2, 1, 8, GROUP, ZERO, SF32>(a, f32, stream);
  }
}

template <int GROUP>
void launch_w4_group(const W4Args& a, bool sf32, bool f32, hipStream_t stream) {
  if (a.zeros) {
    if (sf32) launch_w4_typed<GROUP, true, true>(a, f32, stream);
    else launch_w4_typed<GROUP, true, false>(a, f32, stream);
  } else {
    if (sf32) launch_w4_typed<GROUP, false, true>(a, f32, stream);
    else launch_w4_typed<GROUP, false, false>(a, f32, stream);
  }
}

// Rows the workspace holds: the batch rounded up to a workgroup's.
int64_t padded_rows(int64_t B) {
  const int64_t to = B <= 32 ? 32 : B <= 64 ? 64 : 128;
  return (B + to - 1) / to * to;
}

}  // namespace

size_t w4_workspace_bytes(int64_t B, int64_t D, int group) {
  if (B <= kW4FewRows) return 0;
  return (size_t)(padded_rows(B) * w4_steps(D) * (256 + 4 * (kW4Step / group)));
}

hipError_t launch_w4_logits(W4Args a, int scale_dtype, int logits_dtype, int group, void* workspace, hipStream_t stream) {
  const bool sf32 = scale_dtype == ARCS_DTYPE_F32, f32 = logits_dtype == ARCS_DTYPE_F32;
  if (a.B > kW4FewRows) {
    a.padded_rows = padded_rows(a.B);
    a.prepared = (char*)workspace;
    a.sums = (float*)(a.prepared + a.padded_rows * w4_steps(a.D) * 256);
  }
  if (group == 32) launch_w4_group<32>(a, sf32, f32, stream);
  else if (group == 64) launch_w4_group<64>(a, sf32, f32, stream);
  else launch_w4_group<128>(a, sf32, f32, stream);
  return hipGetLastError();
}

}  // namespace arcs
