// Head logits from 4-bit weights with group scales.
//
//   logits[b, v] = sum_g scale[v, g] * sum_{d in g} (q[v, d] - zero[v, g]) hidden[b, d]
//
// q is two weights a byte, the lower d in the low nibble.  The products run
// on the bfloat16 matrix instruction with the batch as its rows and 16
// vocabulary rows as its columns, so a lane needs the scale of one row only.
// A nibble becomes the level q - z itself, exactly, in bfloat16 times 2^-19 (w4_unpack),
// and the logits are multiplied by 2^19 at the end.  So a level of zero adds
// nothing, an infinite hidden state keeps its level's sign and sums are no larger
// than the definition's.  (Levels with an offset of 16 or 48, taken away again
// through the accumulator's start, took 8 or 12 operations for 8 weights instead of
// 17 to 19 but lost four to six bits of a sum to the offset's, and all of it with one
// large hidden state.)  Scales are applied to the group's float32 sums, so no
// weight is rounded.
//
// Batches of at most 16 rows take one launch: hidden states go through LDS, four
// steps of 128 k at a time in two buffers, and weights from memory to registers
// four steps ahead.  What bounds them is reading the weights, beside which the
// unpacking does not hide whole: one row x 129,280 x 4,096 (277 MB) takes 60 us,
// 4.6 TB/s (a large copy reaches 5.1; levels with an offset took 54).  It took nearly
// twice that while a row's 64 bytes of one step were asked for at a time: each line
// of weights and scales had left the L2 before its other half was wanted.
//
// Larger batches have the hidden states prepared first, in the workspace: in the
// nibbles' order and as the LDS holds them, so that a step is a plain copy to LDS
// that takes no registers.  There the unpacking, the scaling of the groups' sums, the
// LDS reads and the products take about the same time each, and overlap only in part:
// 256 rows x 129,280 x 7,168 in groups of 64 with zero points take 550 to 560 us (850
// TFLOP/s).  A tile of 128 rows x 32 columns a wave unpacks each weight twice for 256
// rows; 64 x 64 a wave unpacks it four times and took 590 us where this one took 570.
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

// Eight nibbles less their zero point, times 2^-19, as bfloat16 in the order 0 4 1 5 2 6 3 7.
// Two nibbles at a time become the binary16 numbers 128 + q / 8 (or, from the bits four
// higher, 8 + q / 8); adding -(128 + z / 8) or -(8 + z / 8) gives (q - z) / 8 exactly.  Its
// exponent field is 0 or 12 .. 15, whose upper three bits are 011, and its lower seven
// mantissa bits are 0: with its lower twelve bits moved down by three, under the upper four
// as they were, it is the bfloat16 with the exponent field 011 011xx, that is 2^-16 times the
// number.  `zero` holds z in bits 0 .. 3 of both halves.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The masks are registers to the compiler: an AND and an OR of two literals are two
// instructions, of a register and a literal one (21 operations for 8 weights, 17 so).
struct W4Masks {
  uint32_t low = 0x000F000Fu, high = 0x00F000F0u;
  __device__ __forceinline__ W4Masks() {
    asm("" : "+v"(low));
    asm("" : "+v"(high));
  }
};

template <bool ZERO>
__device__ __forceinline__ bf16x8 w4_unpack(uint32_t w, uint32_t zero, const W4Masks& mask) {
  const uint32_t low = ZERO ? zero | 0xD800D800u : 0xD808D808u, high = ZERO ? (zero << 4) | 0xC800C800u : 0xC880C880u;
  auto level = [](uint32_t q, uint32_t less) {
    const f16x2 x = __builtin_bit_cast(f16x2, q) + __builtin_bit_cast(f16x2, less);
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return ((b >> 3) & 0x0FFF0FFFu) | (b & 0xF000F000u);
  };
  const uint32_t w8 = w >> 8;
  u32x4 d;
  d[0] = level((w & mask.low) | 0x58005800u, low);
  d[1] = level((w & mask.high) | 0x48004800u, high);
  d[2] = level((w8 & mask.low) | 0x58005800u, low);
  d[3] = level((w8 & mask.high) | 0x48004800u, high);
  return __builtin_bit_cast(bf16x8, d);
}

constexpr float kW4Unit = 0x1p19f;  // what the sums of w4_unpack's levels are multiplied by

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

  // Chunk c of 8 k of a step is lane group j's in product n; the LDS slot of (n, j) is 4 n + j
  // in a row of 16 chunks, then turned by the row, so that no two lanes of a read share a bank.
  static __device__ __forceinline__ int slot(int c) { return kTurn ? c : (c & 3) * 4 + (c >> 2); }

  // RT tiles of 16 weight rows of a wave, through a buffer descriptor: what lies
  // past D in a row meets hidden states that are zero there, and what lies past
  // the last row is not read.
  template <int RT>
  struct Rows {
    const char* base;
    int64_t bytes;
    uint32_t off[RT];
    __device__ __forceinline__ Rows(const W4Args& a, int64_t v0, int r, int j) {
      const int64_t v = v0 < a.V ? v0 : a.V - 1;
      base = (const char*)a.qweight + v * a.qweight_stride;
      bytes = (a.V - 1 - v) * a.qweight_stride + a.D / 2;
#pragma unroll
      for (int t = 0; t < RT; ++t)
        off[t] = (uint32_t)(v + t * 16 + r < a.V ? t * 16 + r : a.V - 1 - v) * (uint32_t)a.qweight_stride + j * 16;
    }
    // 16 bytes a lane of each tile: k 128 step on
    __device__ __forceinline__ void load(u32x4 (&w)[RT], int step) const {
      // a part's last step can begin past the end of the last row: nothing is left there
      const int64_t at = (int64_t)step * (kW4Step / 2), left = bytes > at ? bytes - at : 0;
      const __amdgpu_buffer_rsrc_t d = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(base + at), (short)0, (int)(left < (int64_t)kBufMost ? left : (int64_t)kBufMost), 0x00020000);
#pragma unroll
      for (int t = 0; t < RT; ++t) w[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(d, off[t], 0, 0));
    }
  };

  // The scales of a workgroup's ROWS weight rows over kN groups, and their
  // zero points, on their way to LDS as [group][row] pairs.
  // fetch only loads (a conversion beside a load would wait for it there).  Groups
  // past the end get a scale of zero: the last group's may be infinite, and meets zeros.
  template <int ROWS, int kN, int THREADS>
  struct Scales {
    static_assert(ROWS * kN % THREADS == 0, "scales of a part over the threads");
    static constexpr int kPer = ROWS * kN / THREADS;
    const char *sb, *zb;
    uint32_t so[kPer], zo[kPer];
    uint32_t s[kPer], z[kPer];
    int groups;
    bool past;
    __device__ __forceinline__ Scales(const W4Args& a, int64_t v0) {
      const int64_t v = v0 < a.V ? v0 : a.V - 1;
      sb = (const char*)a.scales + v * a.scale_stride * kScale;
      zb = (const char*)a.zeros + v * a.zero_stride;
      groups = (int)(a.D / GROUP);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = (threadIdx.x + i * THREADS) / kN;
        const uint32_t at = (uint32_t)(v + row < a.V ? row : a.V - 1 - v);
        so[i] = at * (uint32_t)a.scale_stride * kScale;
        zo[i] = at * (uint32_t)a.zero_stride;
      }
    }
    __device__ __forceinline__ void fetch(int part) {
      int g = part * kN + threadIdx.x % kN;  // THREADS is a multiple of kN
      past = g >= groups;
      g = past ? groups - 1 : g;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const char* p = sb + (so[i] + (uint32_t)g * kScale);
        s[i] = SF32 ? *(const uint32_t*)p : *(const uint16_t*)p;
        if (ZERO) z[i] = *(const uint8_t*)(zb + (zo[i] + (uint32_t)g));
      }
    }
    __device__ __forceinline__ void store(uint2* to) const {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x + i * THREADS;
        to[e % kN * ROWS + e / kN] =
            make_uint2(past ? 0 : SF32 ? s[i] : s[i] << 16, ZERO ? (z[i] & 15u) * 0x00010001u : 0u);
      }
    }
  };
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
        const float x = total[m][t][e] * kW4Unit;
        if (OF32) ((float*)a.logits)[row * a.row_stride + v] = x;
        else ((__bf16*)a.logits)[row * a.row_stride + v] = (__bf16)x;
      }
  }
}

// ---------------------------------------------------------------------------
// At most 16 rows: four waves of RT * 16 weight rows each.
// ---------------------------------------------------------------------------
constexpr int kW4Stage = 4;  // steps

template <int GROUP, bool ZERO, bool SF32, bool OF32>
__global__ __launch_bounds__(256, 4) void w4_rows_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, SF32>;
  constexpr int SC = kW4Stage, kRows = 16, kPer = kRows * SC * 16 / 256, kN = SC * K::kGroups;
  __shared__ __align__(16) char s_x[2][SC * kRows * 256];
  __shared__ __align__(16) uint2 s_scale[2][64 * kN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, j = lane >> 4;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + wave) * 16;
  const int steps = (int)((a.D + kW4Step - 1) / kW4Step), stages = (steps + SC - 1) / SC;
  const typename K::template Rows<1> rows(a, v0, r, j);
  typename K::template Scales<64, kN, 256> scales(a, (int64_t)blockIdx.x * 64);

  // the stage's hidden states: piece p of a thread is 8 k of one row, 64 pieces a row
  u32x4 xr[kPer];
  auto fetch_x = [&](int stage) {
    const int64_t k = (int64_t)stage * SC * kW4Step + lane * 8;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int row = wave + p * 4;
      if (row < a.B) xr[p] = *(const u32x4*)(a.hidden + row * a.hidden_stride + (k < a.D ? k : 0));
    }
  };
  auto store_x = [&](int stage) {
    char* x = s_x[stage & 1] + (lane >> 4) * (kRows * 256);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int row = wave + p * 4;
      if (row >= a.B) continue;
      if ((int64_t)stage * SC * kW4Step + lane * 8 >= a.D) xr[p] = u32x4{0, 0, 0, 0};
      *(u32x4*)(x + row * 256 + ((K::slot(lane & 15) ^ row) * 16)) = w4_order(xr[p]);
    }
  };

  const W4Masks mask;
  u32x4 next[SC][1];
  f32x4 total[1][1] = {{{0.0f, 0.0f, 0.0f, 0.0f}}};
  fetch_x(0);
  scales.fetch(0);
#pragma unroll
  for (int c = 0; c < SC; ++c) rows.load(next[c], c < steps ? c : 0);
  store_x(0);
  scales.store(s_scale[0]);
  __syncthreads();
  for (int stage = 0; stage < stages; ++stage) {
    u32x4 now[SC];
#pragma unroll
    for (int c = 0; c < SC; ++c) now[c] = next[c][0];
    if (stage + 1 < stages) {
      fetch_x(stage + 1);
      scales.fetch(stage + 1);
      // all of a row's 256 bytes are asked for at once: a line is used while it is cached
#pragma unroll
      for (int c = 0; c < SC; ++c) rows.load(next[c], (stage + 1) * SC + c < steps ? (stage + 1) * SC + c : 0);
    }
    const char* x = s_x[stage & 1];
    const uint2* scale = &s_scale[stage & 1][wave * 16 + r];
#pragma unroll
    for (int c = 0; c < SC; ++c) {
      if (c > 0 && stage * SC + c >= steps) break;
      const u32x4 w = K::kTurn ? w4_turn(now[c]) : now[c];
#pragma unroll
      for (int g = 0; g < K::kGroups; ++g) {
        const int gs = c * K::kGroups + g;
        const uint2 sc = scale[gs * 64];
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < K::kProducts; ++i) {
          const bf16x8 xf = *(const bf16x8*)(x + (c * kRows + r) * 256 + ((((g * K::kProducts + i) * 4 + j) ^ r) * 16));
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, w4_unpack<ZERO>(w[g * K::kProducts + i], sc.y, mask), acc, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) total[0][0][e] = fmaf(__uint_as_float(sc.x), acc[e], total[0][0][e]);
        asm volatile("" : "+v"(total[0][0]));  // the sums are not left for later
      }
    }
    if (stage + 1 < stages) {
      store_x(stage + 1);
      scales.store(s_scale[(stage + 1) & 1]);
    }
    __syncthreads();
  }
  w4_write<1, 1, OF32>(a, total, 0, v0, r, j);
}

// ---------------------------------------------------------------------------
// More rows.  The prepared hidden states of one step are 4096 bytes for every 16
// rows: row x 256 bytes, chunk c of 8 k at slot(c) ^ row; rows past B are zeros.
// ---------------------------------------------------------------------------
template <int GROUP, bool ZERO>
__global__ __launch_bounds__(256) void w4_prepare_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, false>;
  const int row = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int64_t step = blockIdx.x, tile = blockIdx.y, b = tile * 16 + row, k = step * kW4Step + c * 8;
  u32x4 v = {0, 0, 0, 0};
  if (b < a.B && k < a.D) v = *(const u32x4*)(a.hidden + b * a.hidden_stride + k);
  const int64_t tiles = a.padded_rows / 16;
  *(u32x4*)(a.prepared + (step * tiles + tile) * 4096 + row * 256 + ((K::slot(c) ^ row) * 16)) = w4_order(v);
}

// Steps between two barriers: a row's 128 bytes, as far as LDS reaches.
constexpr int w4_part(int rows, int group) { return rows == 128 && group == 32 ? 1 : 2; }

template <int MT, int RT, int WB, int WV, int GROUP, bool ZERO, bool SF32, bool OF32>
__global__ __launch_bounds__(WB* WV * 64, MT == 2 ? 3 : 2) void w4_batch_kernel(W4Args a) {
  using K = W4<GROUP, ZERO, SF32>;
  constexpr int NS = w4_part(WB * MT * 16, GROUP), kThreads = WB * WV * 64, kCols = WV * RT * 16;
  constexpr int kWaves = WB * WV, kRows = WB * MT * 16;
  constexpr int kLoads = NS * kRows / 4, kPer = kLoads / kWaves;  // of 1024 bytes
  constexpr int kN = NS * K::kGroups;                             // groups of a part
  constexpr int kStage = NS * kRows * 256;
  static_assert(kLoads % kWaves == 0, "loads of a part over the waves");
  __shared__ __align__(1024) char lds[2 * kStage];
  __shared__ __align__(16) uint2 s_scale[2][kCols * kN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, j = lane >> 4;
  const int wb = wave % WB, wv = wave / WB;
  // blocks go round the eight dies in turn; a die gets neighbouring tiles, the
  // batch's tiles of the same weights one after the other
  const int per = (a.tiles + 7) / 8, at = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (((int)blockIdx.x >> 3) >= per || at >= a.tiles) return;
  const int64_t b0 = (int64_t)(at % a.batch_tiles) * kRows;
  const int64_t vb = (int64_t)(at / a.batch_tiles) * kCols, v0 = vb + wv * (RT * 16);
  const int parts = (int)((a.D + NS * kW4Step - 1) / (NS * kW4Step));
  const typename K::template Rows<RT> rows(a, v0, r, j);
  typename K::template Scales<kCols, kN, kThreads> scales(a, vb);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(ARCS_LDS char*)lds;
  const int64_t step_x = a.padded_rows * 256;
  const char* px = a.prepared + b0 * 256;
  auto issue = [&](int part) {
    const uint32_t to = lds0 + (uint32_t)(part & 1) * kStage;
#pragma unroll
    for (int t = 0; t < kPer; ++t) {
      const int load = wave + t * kWaves, step = load / (kRows / 4), in = load % (kRows / 4);
      load_to_lds(to + load * 1024u, (uint32_t)lane * 16,
                  buffer_of(px + ((int64_t)part * NS + step) * step_x + in * 1024, 1024));
    }
  };

  f32x4 total[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t) total[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const W4Masks mask;
  u32x4 next[NS][RT];
  scales.fetch(0);
  issue(0);
#pragma unroll
  for (int c = 0; c < NS; ++c) rows.load(next[c], c);
  scales.store(s_scale[0]);
  for (int part = 0; part < parts; ++part) {
    // This part's hidden states are in LDS: only its weights, NS * RT loads issued
    // after them, may be on their way.
    wait_loads<NS * RT>();
    wait_lds();
    __builtin_amdgcn_s_barrier();
    if (part + 1 < parts) {
      scales.fetch(part + 1);
      issue(part + 1);
    }
    const int ahead = part + 1 < parts ? (part + 1) * NS : 0;  // the last part's loads are not used
    const char* x = lds + (part & 1) * kStage;
    const uint2* scale = &s_scale[part & 1][wv * RT * 16 + r];
    // Products p = 0 .. 4 NS - 1 of 32 k each; the hidden states of the next one are
    // read while one runs.  Groups past D meet zeros, and a scale of zero.
    constexpr int kAll = 4 * NS;
    bf16x8 xf[2][MT];
    auto read_x = [&](int p) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xf[p & 1][m] = *(const bf16x8*)(x + ((p >> 2) * kRows + (wb * MT + m) * 16 + r) * 256 + ((((p & 3) * 4 + j) ^ r) * 16));
    };
    u32x4 w[RT];
    uint2 sc[RT];
    f32x4 acc[MT][RT];
    read_x(0);
#pragma unroll
    for (int p = 0; p < kAll; ++p) {
      const int c = p / 4, gs = p / K::kProducts, i = p % K::kProducts;
      if (p % 4 == 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t) w[t] = K::kTurn ? w4_turn(next[c][t]) : next[c][t];
        rows.load(next[c], ahead + c);
      }
      if (i == 0) {
#pragma unroll
        for (int t = 0; t < RT; ++t) sc[t] = scale[gs * kCols + t * 16];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      if (p + 1 < kAll) read_x(p + 1);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const bf16x8 wf = w4_unpack<ZERO>(w[t][p % 4], sc[t].y, mask);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[p & 1][m], wf, acc[m][t], 0, 0, 0);
      }
      if (i == K::kProducts - 1) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int e = 0; e < 4; ++e) total[m][t][e] = fmaf(__uint_as_float(sc[t].x), acc[m][t][e], total[m][t][e]);
            asm volatile("" : "+v"(total[m][t]));  // one group at a time in registers: its sums are not left for later
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (part + 1 < parts) scales.store(s_scale[(part + 1) & 1]);
  }
  wait_loads<0>();
  w4_write<MT, RT, OF32>(a, total, b0 + wb * MT * 16, v0, r, j);
}

namespace {

// Steps of the prepared hidden states: whole parts of two, zeros past D.
int64_t w4_steps(int64_t D) { return (D + 2 * kW4Step - 1) / (2 * kW4Step) * 2; }

template <int GROUP, bool ZERO, bool SF32>
void launch_w4_rows(const W4Args& a, bool f32, hipStream_t stream) {
  const dim3 grid((unsigned)((a.V + 63) / 64)), block(256);
  if (f32) hipLaunchKernelGGL((w4_rows_kernel<GROUP, ZERO, SF32, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((w4_rows_kernel<GROUP, ZERO, SF32, false>), grid, block, 0, stream, a);
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
  // The smallest tile that holds the batch, and from 65 rows on 128 rows a tile.  Against
  // 129,280 x 7,168, in the tile taken and in the next larger one, without and with zero
  // points (us):
  //            groups of 32           64                     128
  //   16 rows  162/157, 178/183       132/141, 143/165       127/133, 130/144
  //   32 rows  163/301, 188/333       146/175, 170/198       138/154, 148/162
  //   64 rows  304/332, 336/367       186/262, 210/273       165/237, 174/247
  // (16 rows in groups of 32 are the one pair that is no better; against 4,096 it is
  // 108/104 and 106/106.)
  if (a.B <= kW4FewRows) {
    launch_w4_rows<GROUP, ZERO, SF32>(a, f32, stream);
  } else if (a.B <= 32) {
    launch_w4_batch<2, 2, 1, 4, GROUP, ZERO, SF32>(a, f32, stream);
  } else if (a.B <= 64) {
    launch_w4_batch<4, 4, 1, 4, GROUP, ZERO, SF32>(a, f32, stream);
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

size_t w4_workspace_bytes(int64_t B, int64_t D) {
  if (B <= kW4FewRows) return 0;
  return (size_t)(padded_rows(B) * w4_steps(D) * 256);
}

hipError_t launch_w4_logits(W4Args a, int scale_dtype, int logits_dtype, int group, void* workspace, hipStream_t stream) {
  const bool sf32 = scale_dtype == ARCS_DTYPE_F32, f32 = logits_dtype == ARCS_DTYPE_F32;
  if (a.B > kW4FewRows) {
    a.padded_rows = padded_rows(a.B);
    a.prepared = (char*)workspace;
  }
  if (group == 32) launch_w4_group<32>(a, sf32, f32, stream);
  else if (group == 64) launch_w4_group<64>(a, sf32, f32, stream);
  else launch_w4_group<128>(a, sf32, f32, stream);
  return hipGetLastError();
}

}  // namespace arcs
