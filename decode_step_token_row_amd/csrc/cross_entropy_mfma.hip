// Linear cross entropy on the matrix instructions (bfloat16 and float32 rows on
// the 16-byte grid).
//
// One tile kernel runs the four products of the general kernel (STATS, DS,
// DHIDDEN, DWEIGHT): C[m, n] = sum_k A[m, k] B[n, k], 128 bytes of k at a time.
// Tiles go from memory to LDS by the buffer loads that write LDS directly, S
// tiles deep, one barrier a tile.  An operand whose rows run along k is read
// back 16 bytes a lane; one whose rows run along m or n (the head in DHIDDEN,
// both operands in DWEIGHT) through the transposing LDS read (bfloat16) or word
// by word (float32), so no operand is stored twice.  The load writes LDS in lane
// order, so bank conflicts (none are counted in the loop, up to 7 % of the LDS
// cycles in the results' way through LDS) are avoided by permuting the lanes'
// global addresses:
//   along k: a row's 128 bytes are 8 chunks, chunk c of row r at c ^ (r / 2 % 8);
//   along m: a row's 32-byte chunks, chunk q of row k at q ^ 2 (k % 4).
//
// What bounds it: the products.  4,096 rows x 129,280 x 4,096 take 3.4 to 3.6 ms
// forward, by machine (1,210 to 1,270 TFLOP/s; a large library product reaches 1,445),
// 256 x 256 tiles of eight waves of 128 x 64.  Steps, at that size, each beside the one
// before on one machine: the plain loop 3.75 ms;
// fragments read one k step ahead of the products, across the barrier too,
// 3.58; the next tile's loads between the products instead of before them, 3.52;
// workgroups that stay and load their next tile before they write the last one
// out, 3.37.  Slower: four waves of 128 x 128 (4.0), the head three tiles deep
// (3.67).  Few rows are bound by reading the head: one row x 32,000 x 2,048 takes
// 29 us with its launches (131 MB, 26 us at the rate of a copy).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cross_entropy.hpp"
#include "cross_entropy_device.hpp"
#include "launch.hpp"
#include "lds_load.hpp"
#include "mfma_tile.hpp"

namespace arcs {

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
struct CeTile {
  static constexpr int kThreads = WM * WN * 64, kWaves = WM * WN;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr bool kLogits = MODE == kCeStats || MODE == kCeDs;
  static constexpr bool kAOuter = !kLogits, kBOuter = MODE == kCeDweight;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kTK = 128 / sizeof(T);  // k of one tile
  static constexpr int kABytes = BM * 128, kBBytes = BN * 128, kStage = kABytes + kBBytes;
  static constexpr int kALoads = BM / 8, kBLoads = BN / 8;  // of 1024 bytes each
  static constexpr int kAPer = (kALoads + kWaves - 1) / kWaves, kBPer = (kBLoads + kWaves - 1) / kWaves;
  static constexpr int kPer = kAPer + kBPer;
  // bfloat16 results go out through 32 rows of kOutM columns a wave
  static constexpr bool kOut = kBf16 && (MODE == kCeDs || MODE == kCeDweight);
  static constexpr int kOutM = MT % 2 == 0 && S * kStage + kWaves * 32 * 64 * 2 <= 163840 ? 64 : 32;
  static constexpr int kOutBytes = 32 * kOutM * 2, kLds = S * kStage + (kOut ? kWaves * kOutBytes : 0);
};

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
__global__ __launch_bounds__(WM* WN * 64, 2) void ce_tile_kernel(CeArgs a, CePiece pc) {
  using C = CeTile<T, MODE, WM, WN, MT, NT, S>;
  constexpr int BM = C::BM, BN = C::BN, kTK = C::kTK;
  constexpr int64_t E = sizeof(T);
  __shared__ __align__(1024) char lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool direct = MODE == kCeStats && pc.direct;
  const int64_t count = direct ? a.N : a.head->count;
  const int64_t M = C::kLogits ? pc.len : a.D;
  const int64_t N = MODE == kCeDweight ? pc.len : count;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(ARCS_LDS char*)lds;

  // The tiles of this workgroup.  Workgroups go round the eight dies in turn; a
  // die gets neighbouring tiles, eight along m by some along n, which share
  // their operands in its L2.  DHIDDEN has few tiles of a long k: there
  // a.workers workgroups share them out evenly, worker w the tiles from
  // w T / workers on, the first and last of them in part.
  const int mt = (int)((M + BM - 1) / BM), nt = (int)((N + BN - 1) / BN), all = mt * nt;
  int job, job_end, job_step = 1, worker = 0;
  if (MODE == kCeDhidden) {
    worker = ((int)blockIdx.x & 7) * (a.workers / 8) + ((int)blockIdx.x >> 3);
    job = (int)((int64_t)worker * all / a.workers);
    job_end = (int)(((int64_t)(worker + 1) * all + a.workers - 1) / a.workers);
  } else {
    const int chunk = (all + 7) / 8, first = ((int)blockIdx.x & 7) * chunk;
    job = first + ((int)blockIdx.x >> 3);
    job_end = first + chunk < all ? first + chunk : all;
    job_step = (int)gridDim.x / 8;
  }
  if (job >= job_end) return;

  // The tile that is loaded: descriptors at its first k, and the lanes' offsets.
  int64_t m0, n0;
  int nk, shift = 0;
  const char *pa, *pb;
  int64_t na, nb;
  uint32_t oa[C::kAPer], ob[C::kBPer];
  const T* W = (const T*)a.weight + pc.v0 * a.weight_stride;
  const T* H = (const T*)(pc.gather ? a.hidden : a.hc);
  const T* Z = (const T*)a.ds;
  const int64_t step_a = C::kLogits ? 128 : MODE == kCeDhidden ? kTK * a.weight_stride * E : kTK * a.D * E;
  const int64_t step_b = MODE == kCeDweight ? kTK * a.ds_ld * E : 128;
  auto place = [&](int job) {
    tile_place(job, mt, nt, m0, n0);
    m0 *= BM;
    n0 *= BN;
    int64_t k_lo = 0, k_hi = C::kLogits ? a.D : MODE == kCeDhidden ? pc.len : count;
    if (MODE == kCeDhidden) {
      // where worker w begins, in tiles' k: a fraction of the workers, the same in every piece
      const int64_t tiles_k = (pc.len + kTK - 1) / kTK;
      const int64_t from = (int64_t)worker * all - (int64_t)job * a.workers, to = from + all;
      if (from > 0) k_lo = from * tiles_k / a.workers * kTK;
      if (to < a.workers) k_hi = to * tiles_k / a.workers * kTK;
    }
    nk = k_hi > k_lo ? (int)((k_hi - k_lo + kTK - 1) / kTK) : 0;
    // With one tile of rows every workgroup reads other weight rows, and begun together
    // all ask for the same columns of rows a power of two apart, so for few of the
    // memory's channels at a time: each begins its walk along k elsewhere (one row x
    // 32,000 tokens, D = 2048: 34.3 us without, 28.7 with; 64 rows x 128,000: 270 and
    // 273).  Tiles of the same weight rows share their loads, and begin together.
    if (C::kLogits) shift = nt == 1 ? (int)((uint32_t)job * 2654435761u >> 16) % nk : 0;
    na = nb = kBufMost;
#pragma unroll
    for (int t = 0; t < C::kAPer; ++t) {
      const int inst = (wave + t * C::kWaves) % C::kALoads;
      int r, c;
      if (!C::kAOuter) {
        inner_place<T>(inst, lane, r, c);
        const int64_t left = M - 1 - m0;
        oa[t] = (uint32_t)((r < left ? r : left) * a.weight_stride * E + c * E);
      } else {
        outer_place<T, BM>(inst, lane, r, c);
        const int64_t ld = MODE == kCeDhidden ? a.weight_stride : a.D;
        oa[t] = m0 + c < M ? (uint32_t)(r * ld * E + c * E) : kNoLoad;
      }
    }
#pragma unroll
    for (int t = 0; t < C::kBPer; ++t) {
      const int inst = (wave + t * C::kWaves) % C::kBLoads;
      int r, c;
      if (!C::kBOuter) {
        inner_place<T>(inst, lane, r, c);
        const int64_t left = N - 1 - n0, n = r < left ? r : left;
        if (C::kLogits) ob[t] = (uint32_t)((direct ? (n0 + n) * a.hidden_stride : pc.gather ? (int64_t)a.rows[n0 + n].row * a.hidden_stride : n * a.D) * E + c * E);
        else ob[t] = (uint32_t)(n * a.ds_ld * E + c * E);
      } else {
        outer_place<T, BN>(inst, lane, r, c);
        ob[t] = (uint32_t)(r * a.ds_ld * E + c * E);
      }
    }
    if (C::kLogits) {
      pa = (const char*)(W + m0 * a.weight_stride);
      pb = (const char*)(pc.gather ? H : H + n0 * a.D);
    } else if (MODE == kCeDhidden) {
      pa = (const char*)(W + k_lo * a.weight_stride + m0);
      na = ((pc.len - k_lo) * a.weight_stride - m0) * E;
      pb = (const char*)(Z + n0 * a.ds_ld + k_lo);
    } else {
      pa = (const char*)(H + m0);
      na = (count * a.D - m0) * E;
      pb = (const char*)(Z + n0);
      nb = (count * a.ds_ld - n0) * E;
    }
  };
  // along k: the lane's first element's k in a tile, the same for each second load
  uint32_t ka[2], kb[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    int r, c;
    inner_place<T>((wave + t * C::kWaves) % C::kALoads, lane, r, c);
    ka[t] = (uint32_t)c;
    inner_place<T>((wave + t * C::kWaves) % C::kBLoads, lane, r, c);
    kb[t] = (uint32_t)c;
  }

  // Load t of tile kt, of the kPer a wave has; tiles past the last read nothing
  // (zeros go to a buffer that is free), so that the waits always count the same.
  struct Source {
    u32x4 a, b;
    uint32_t to, left;
  };
  auto source = [&](int kt) {
    Source s;
    const bool none = kt >= nk;
    s.to = lds0 + (uint32_t)(kt % S) * C::kStage;
    if (C::kLogits) {
      kt += shift;
      kt = kt >= nk ? kt - nk : kt;
    }
    const int64_t k = (int64_t)kt * kTK;
    s.a = uniform4(buffer_of(pa + kt * step_a, none ? 0 : C::kAOuter ? na - kt * step_a : (int64_t)kBufMost));
    s.b = uniform4(buffer_of(pb + kt * step_b, none ? 0 : C::kBOuter ? nb - kt * step_b : (int64_t)kBufMost));
    // logits: the columns of the last tile past D are zeros
    s.left = (uint32_t)(a.D - k < kTK ? a.D - k : kTK);
    return s;
  };
  auto issue_one = [&](const Source& s, int t) {
    if (t < C::kAPer) {
      const uint32_t off = C::kLogits && ka[t & 1] >= s.left ? kNoLoad : oa[t];
      const uint32_t to = s.to + ((wave + t * C::kWaves) % C::kALoads) * 1024u;
      if (t == 0) load_to_lds<true>(to, off, s.a);
      else load_to_lds<false>(to, off, s.a);
    } else {
      t -= C::kAPer;
      const uint32_t off = C::kLogits && kb[t & 1] >= s.left ? kNoLoad : ob[t];
      const uint32_t to = s.to + C::kABytes + ((wave + t * C::kWaves) % C::kBLoads) * 1024u;
      if (t == 0) load_to_lds<true>(to, off, s.b);
      else load_to_lds<false>(to, off, s.b);
    }
  };
  auto issue_first = [&]() {
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const Source from = source(t);
#pragma unroll
      for (int l = 0; l < C::kPer; ++l) issue_one(from, l);
    }
  };

  const int wm = (wave % WM) * MT * 32, wn = (wave / WM) * NT * 32;
  const int fr = lane & 31, fh = lane >> 5;
  // A lane's fragments in a stage, as LDS addresses: along k one place for each
  // k step (tiles of 32 rows are 4096 bytes apart), along m one for each tile
  // (k steps are 16 rows apart).
  uint32_t pa_lds[4], pb_lds[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t inner = fr * 128 + (((t * 2 + fh) ^ ((lane >> 1) & 7)) * 16);
    auto outer = [&](int width, int at) {
      if (!C::kBf16) return (uint32_t)((fh * 4 * width + at + fr) * 4);
      const int k = fh * 8 + ((lane & 15) >> 2);
      const int turn = width >= 128 ? (k & 3) << 1 : width == 64 ? ((k >> 1) & 1) << 1 : 0;
      return (uint32_t)(k * width * 2 + (((at >> 4) + ((lane >> 4) & 1)) ^ turn) * 32 + (lane & 3) * 8);
    };
    pa_lds[t] = lds0 + (C::kAOuter ? outer(BM, wm + t * 32) : wm * 128 + inner);
    pb_lds[t] = lds0 + C::kABytes + (C::kBOuter ? outer(BN, wn + t * 32) : wn * 128 + inner);
  }
  // A fragment is 16 bytes: 8 k of bfloat16 for one 32 x 32 x 16 product, or 4 k of
  // float32 for four of 32 x 32 x 2.
  auto frag_inner = [](uint32_t at) { return *(const ARCS_LDS u32x4*)(uintptr_t)at; };
  auto frag_outer = [](uint32_t at, int width) {
    if constexpr (C::kBf16) {
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ARCS_LDS s16x4*)(uintptr_t)at);
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ARCS_LDS s16x4*)(uintptr_t)(at + 8 * width));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      u32x4 f;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = *(const ARCS_LDS uint32_t*)(uintptr_t)(at + e * width * 4);
      return f;
    }
  };
  auto product = [](u32x4 x, u32x4 y, f32x16 c) {
    if constexpr (C::kBf16) {
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(x[e]), __uint_as_float(y[e]), c, 0, 0, 0);
      return c;
    }
  };

  // Fragments of step ks + 1 are read while step ks multiplies.  The last step of
  // a tile reads from the next one: there the workgroup meets, once a tile, the
  // next tile has landed and this one's buffer is filled again.
  f32x16 acc[MT][NT];
  u32x4 fa[2][MT], fb[2][NT];
  auto read = [&](int kt, int ks) {
    const uint32_t at = (uint32_t)(kt % S) * C::kStage;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      fa[ks & 1][i] = C::kAOuter ? frag_outer(pa_lds[i] + at + ks * 32 * BM, BM) : frag_inner(pa_lds[ks] + at + i * 4096);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      fb[ks & 1][j] = C::kBOuter ? frag_outer(pb_lds[j] + at + ks * 32 * BN, BN) : frag_inner(pb_lds[ks] + at + j * 4096);
  };
  auto multiply = [&](int ks) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[i][j] = product(fa[ks & 1][i], fb[ks & 1][j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };

  place(job);
  issue_first();
  while (true) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    wait_loads<(S - 1) * C::kPer>();
    __builtin_amdgcn_s_barrier();
    read(0, 0);
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int ks = 0; ks < 3; ++ks) {
        read(kt, ks + 1);
        multiply(ks);
      }
      const Source from = source(kt + S);
      wait_loads<(S - 2) * C::kPer>();  // tile kt + 1 has landed
      wait_lds();                       // this wave's reads of tile kt are done
      __builtin_amdgcn_s_barrier();
      read(kt + 1, 0);
      // the loads go between the products, which run on while one is issued
      constexpr int kProducts = MT * NT, kEach = (C::kPer + kProducts - 1) / kProducts;
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        acc[p / NT][p % NT] = product(fa[1][p / NT], fb[1][p % NT], acc[p / NT][p % NT]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int l = p * kEach; l < (p + 1) * kEach && l < C::kPer; ++l) issue_one(from, l);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_loads<0>();  // no load into LDS outlives its tile
    wait_lds();
    __builtin_amdgcn_s_barrier();

    // The next tile's first loads fly while this one's results go out.
    const int64_t em0 = m0, en0 = n0;
    const int done = job;
    job += job_step;
    const bool more = job < job_end;
    if (more) {
      place(job);
      issue_first();
    }

    // A lane holds column n = lane % 32 of each 32 x 32 product and rows
    // 8 (r / 4) + 4 (lane / 32) + r % 4: in the lane's wave, row_of + mw of the tile.
    auto row_of = [](int i, int r) { return i * 32 + 8 * (r >> 2) + (r & 3); };
    const int mw = wm + 4 * fh;
    const int m_left = (int)(M - em0 < BM ? M - em0 : BM) - mw;  // rows of the lane that exist
    if (MODE == kCeStats) {
      const bool ragged = M - em0 < BM;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t n = en0 + wn + j * 32 + fr;
        CeRow row;
        row.target = -1;
        row.a = 1.0f;
        if (n < N && !direct) row = a.rows[n];
        if (n < N && direct) {
          float temperature;
          const int kind = ce_row_kind(a, n, row.target, temperature);
          row.a = kLog2e / (kind == 0 ? temperature : 1.0f);
          if (kind != 0) row.target = -1;
        }
        if (ragged) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (row_of(i, r) >= m_left) acc[i][j][r] = -__builtin_inff();
        }
        float m = acc[0][j][0];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) m = fmaxf(m, acc[i][j][r]);
        m = fmaxf(m, __shfl_xor(m, 32, kWave)) * row.a;  // y = dot * a, a > 0
        const float mz = finite_or_zero(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) sum += exp2_fast(fmaf(acc[i][j][r], row.a, -mz));
        sum += __shfl_xor(sum, 32, kWave);
        // a slice is a wave's rows of the tile
        if (fh == 0 && n < N) a.partial[n * a.slices + em0 / BM * WM + wave % WM] = make_float2(m, sum);
        // few tiles hold a row's target
        const int64_t to_target = (int64_t)row.target - em0 - mw;
        const bool mine = to_target >= 0 && to_target < MT * 32 && (to_target & 4) == 0;
        if (__any(mine)) {
          float t = 0.0f;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) t = row_of(i, r) == (int)to_target ? acc[i][j][r] : t;
          if (mine) a.dtarget[n] = t;
        }
      }
    }
    if (MODE == kCeDhidden) {
      // part worker + job of the slab, [BN][BM]: each pair of them is met once
      float* part = a.slab + (int64_t)(worker + done) * (BM * BN);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int nl = wn + j * 32 + fr;
        if (en0 + nl >= N) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (row_of(i, q * 4) >= m_left) continue;
            f32x4* out = (f32x4*)(part + nl * BM + mw + row_of(i, q * 4));
            f32x4 v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
            if (!pc.first) v += *out;
            *out = v;
          }
      }
    }
    if (!C::kBf16 && (MODE == kCeDs || MODE == kCeDweight)) {
      const float g = MODE == kCeDweight ? a.head->gmax : 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t n = en0 + wn + j * 32 + fr;
        if (n >= N) continue;
        CeRow row;
        row.target = -1;
        row.a = row.c = row.lse2 = row.rest = 0.0f;
        if (MODE == kCeDs) row = a.rows[n];
        const int64_t to_target = (int64_t)row.target - pc.v0 - em0 - mw;
        const int target = to_target >= 0 && to_target < MT * 32 ? (int)to_target : -1;
        float* to = MODE == kCeDs ? (float*)a.ds + n * a.ds_ld + em0 + mw : (float*)a.out_dweight + (pc.v0 + n) * a.D + em0 + mw;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4 out;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int id = row_of(i, q * 4 + e);
              float v = acc[i][j][q * 4 + e];
              if (MODE == kCeDs) {
                v = exp2_fast(fmaf(v, row.a, -row.lse2)) * row.rest;
                v = id == target ? v - 1.0f : v;
                v = id < m_left ? v * row.c : 0.0f;
              } else {
                v *= g;
              }
              out[e] = v;
            }
            if (MODE == kCeDs || row_of(i, q * 4) < m_left) *(f32x4*)(to + row_of(i, q * 4)) = out;
          }
      }
    }
    if (C::kOut) {
      // bfloat16 results: 32 rows n of kOutM columns at a time through the wave's own
      // part of LDS, so that whole lines are stored.  16-byte chunk c of row n at c ^ n.
      constexpr int kOutM = C::kOutM, kChunks = kOutM / 8, kTiles = kOutM / 32;
      char* own = lds + S * C::kStage + wave * C::kOutBytes;
      const float g = MODE == kCeDweight ? a.head->gmax : 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        CeRow row;
        row.target = -1;
        row.a = row.c = row.lse2 = row.rest = 0.0f;
        if (MODE == kCeDs && en0 + wn + j * 32 + fr < N) row = a.rows[en0 + wn + j * 32 + fr];
        const int64_t to_target = (int64_t)row.target - pc.v0 - em0 - mw;
        const int target = to_target >= 0 && to_target < MT * 32 ? (int)to_target : -1;
#pragma unroll
        for (int i0 = 0; i0 < MT; i0 += kTiles) {
#pragma unroll
          for (int i = i0; i < i0 + kTiles; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              bf16x4 out;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float v = acc[i][j][q * 4 + e];
                if (MODE == kCeDs) {
                  const int id = row_of(i, q * 4 + e);
                  v = exp2_fast(fmaf(v, row.a, -row.lse2)) * row.rest;
                  v = id == target ? v - 1.0f : v;
                  v = id < m_left ? v * row.c : 0.0f;
                } else {
                  v *= g;
                }
                out[e] = (__bf16)v;
              }
              const int ml = row_of(i - i0, q * 4) + 4 * fh;
              *(bf16x4*)(own + fr * (kOutM * 2) + (((ml >> 3) ^ (fr & (kChunks - 1))) * 16) + (ml & 4) * 2) = out;
            }
          wait_lds();
          const int64_t ms = em0 + wm + i0 * 32;
#pragma unroll
          for (int t = 0; t < 32 * kChunks / 64; ++t) {
            const int nl = (t * 64 + lane) / kChunks, c = (t * 64 + lane) % kChunks;
            const int64_t n = en0 + wn + j * 32 + nl, m = ms + c * 8;
            const u32x4 v = *(const u32x4*)(own + nl * (kOutM * 2) + ((c ^ (nl & (kChunks - 1))) * 16));
            if (n >= N) continue;
            if (MODE == kCeDs) *(u32x4*)((uint16_t*)a.ds + n * a.ds_ld + m) = v;
            else if (m < M) *(u32x4*)((uint16_t*)a.out_dweight + (pc.v0 + n) * a.D + m) = v;
          }
          wait_lds();  // read before the next columns are written
        }
      }
    }
    if (!more) break;
  }
}

// dhidden rows: the parts of each tile added up in the workers' order; zeros for
// rows that are not listed.
template <typename T, int BM>
__global__ __launch_bounds__(256) void ce_dhidden_parts_kernel(CeArgs a, int BN) {
  const int64_t n = blockIdx.x;
  const int64_t d = (int64_t)blockIdx.y * 1024 + threadIdx.x * 4;
  if (d >= a.D) return;
  const int i = a.place[n], m = (int)(d / BM);
  const int mt = (int)((a.D + BM - 1) / BM), nt = (a.head->count + BN - 1) / BN, all = mt * nt;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i >= 0) {
    const int job = tile_index(m, i / BN, mt, nt);
    const int lo = (int)((int64_t)job * a.workers / all), hi = (int)(((int64_t)(job + 1) * a.workers + all - 1) / all);
    const float* p = a.slab + ((int64_t)job * BN + i % BN) * BM + d % BM;
#pragma unroll 4
    for (int w = lo; w < hi; ++w) v += *(const f32x4*)(p + (int64_t)w * (BN * BM));
    v *= a.head->gmax;
  }
  if constexpr (sizeof(T) == 2) {
    bf16x4 out;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (__bf16)v[e];
    *(bf16x4*)((__bf16*)a.out_dhidden + n * a.D + d) = out;
  } else {
    *(f32x4*)((float*)a.out_dhidden + n * a.D + d) = v;
  }
}

// Backward of at most kCeFewRows rows: the row list and the listed rows' hidden states
// in one launch.  Each workgroup goes over all rows to place its own (both gradients, 64
// rows x 8,000 x 1,024: 36.6 us, 39.4 with a list and then a copy).
constexpr int kCeFewRows = 1024;

template <typename T>
__global__ __launch_bounds__(256) void ce_list_copy_kernel(CeArgs a) {
  __shared__ int s_before[4], s_all[4];
  __shared__ float s_max[4];
  const int64_t n = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0, all = 0;
  float m = 0.0f;
  for (int64_t o0 = 0; o0 < a.N; o0 += 256) {
    const int64_t o = o0 + tid;
    int32_t t;
    float temperature;
    const bool listed = o < a.N && ce_row_kind(a, o, t, temperature) == 0;
    if (listed) {
      const float g = fabsf(a.grad_loss[o] / temperature);
      if (g < __builtin_inff() && g > m) m = g;
    }
    all += __popcll(__ballot(listed));
    before += __popcll(__ballot(listed && o < n));
  }
  m = wave_max_f32(m);
  if (lane == 0) {
    s_before[wave] = before;
    s_all[wave] = all;
    s_max[wave] = m;
  }
  __syncthreads();
  before = s_before[0] + s_before[1] + s_before[2] + s_before[3];
  all = s_all[0] + s_all[1] + s_all[2] + s_all[3];
  m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float gmax = m > 0.0f ? m : 1.0f;
  int32_t target;
  float temperature;
  const bool listed = ce_row_kind(a, n, target, temperature) == 0;
  if (tid == 0) {
    if (n == 0) {
      a.head->count = all;
      a.head->gmax = gmax;
    }
    a.place[n] = listed ? before : -1;
    if (listed) a.rows[before] = ce_row(a, n, target, temperature, gmax);
  }
  if (!listed) return;
  const u32x4* from = (const u32x4*)((const T*)a.hidden + n * a.hidden_stride);
  u32x4* to = (u32x4*)((T*)a.hc + before * a.D);
  for (int64_t c = tid; c < a.D * (int64_t)sizeof(T) / 16; c += 256) to[c] = from[c];
}

// The hidden states of the listed rows, one after the other.
template <typename T>
__global__ __launch_bounds__(256) void ce_copy_kernel(CeArgs a) {
  const int64_t i = blockIdx.x;
  if (i >= a.head->count) return;
  const u32x4* from = (const u32x4*)((const T*)a.hidden + (int64_t)a.rows[i].row * a.hidden_stride);
  u32x4* to = (u32x4*)((T*)a.hc + i * a.D);
  for (int64_t c = threadIdx.x; c < a.D * (int64_t)sizeof(T) / 16; c += 256) to[c] = from[c];
}

namespace {

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
void launch_tile(const CeArgs& a, const CePiece& pc, hipStream_t stream) {
  using C = CeTile<T, MODE, WM, WN, MT, NT, S>;
  const int64_t m = C::kLogits ? pc.len : a.D, n = MODE == kCeDweight ? pc.len : a.N;
  // as many workgroups as the compute units hold (by LDS), at most
  constexpr int64_t kMost = 256 * (163840 / C::kLds);
  const int64_t all = tiles(m, C::BM) * tiles(n, C::BN);
  const int64_t blocks = MODE == kCeDhidden ? a.workers : all < kMost ? tiles(all, 8) * 8 : kMost;
  hipLaunchKernelGGL((ce_tile_kernel<T, MODE, WM, WN, MT, NT, S>), dim3((unsigned)blocks), dim3(C::kThreads), 0, stream, a, pc);
}

// Whether the tiles of logits are too few for the compute units: then tiles of 64 (32)
// rows x 64 take less time.  Forward, with them and without: bfloat16, D = 1,024, 64 rows x
// 8,000 (32 tiles) 11.5 and 16.6 us, 300 x 8,000 (64) 21.6 and 35.4, D = 2,048, 300 x 15,000
// (118) 46 and 55, but 900 x 7,000 (112) 38 and 36; float32, D = 512, 64 x 25,000 (98) 29
// and 43, 20 x 25,000 (196) 26.5 and 19.8, and in the square tiles 200 x 12,000 x 1,024
// (188) 66 and 75, 512 x 8,000 x 1,024 (252) 89 and 84.
bool few_tiles(int64_t len, int64_t N, bool bf16) {
  const int rows = ce_rows_of_tile(N, bf16);
  return tiles(len, rows == 32 ? 128 : ce_columns_of_tile(N, bf16)) * tiles(N, rows) < (!bf16 && rows == 128 ? 192 : 128);
}

// The tile of a call: by its rows, so that few rows are not padded to many.  Against
// 129,280 x 4,096 in bfloat16, in the tile taken and in the next larger one: 32 rows
// 190 and 190 us forward, 694 and 701 backward; 64 rows 186 and 189, 724 and 730;
// 128 rows 192 and 251, 841 and 876.
//   bfloat16  32 x 256 (32 x 128 where that leaves compute units without a tile: one
//             row x 32,000 x 2,048 28.6 us, 33.3 with 256), 64 x 256, 128 x 256, 256 x 256
//   float32   the first three, and 128 x 128 for more rows: their products take so
//             long that smaller tiles, two workgroups a compute unit, cost no time in
//             loads and spread over the card more evenly (training step of 384 rows x
//             32,000 x 1,024: 815 us, 925 with 128 x 256)
template <typename T, int MODE>
void launch_rows(const CeArgs& a, const CePiece& pc, hipStream_t stream) {
  const int rows = ce_rows_of_tile(a.N, sizeof(T) == 2);
  if constexpr (MODE == kCeStats || MODE == kCeDs) {
    if (few_tiles(pc.len, a.N, sizeof(T) == 2)) {
      if (rows == 32) return launch_tile<T, MODE, 2, 1, 1, 1, 4>(a, pc, stream);
      return launch_tile<T, MODE, 2, 2, 1, 1, 4>(a, pc, stream);
    }
  }
  if constexpr (sizeof(T) == 2) {
    if constexpr (MODE == kCeDweight) {
      // two tiles of 128 x 128 run on a compute unit at once and even out a short launch (both
      // gradients, 900 rows x 7,000 x 1,024: 96 us, 102 with 256 x 256); of a long one the larger
      // tiles read less (512 x 30,000 x 2,048: 245 us, 250 with 128 x 128)
      if (tiles(a.D, 256) * tiles(pc.len, 256) < 512) return launch_tile<T, MODE, 2, 2, 2, 2, 2>(a, pc, stream);
      return launch_tile<T, MODE, 2, 4, 4, 2, 2>(a, pc, stream);
    }
    else if (rows == 256) return launch_tile<T, MODE, 2, 4, 4, 2, 2>(a, pc, stream);
    else if (rows == 128) return launch_tile<T, MODE, 4, 2, 2, 2, 3>(a, pc, stream);
  } else {
    if constexpr (MODE == kCeDweight) return launch_tile<T, MODE, 2, 2, 2, 2, 2>(a, pc, stream);
    else if (rows == 128) return launch_tile<T, MODE, 2, 2, 2, 2, 2>(a, pc, stream);
  }
  if constexpr (MODE != kCeDweight) {
    if (rows == 64) return launch_tile<T, MODE, 4, 2, 2, 1, 3>(a, pc, stream);
    if constexpr (MODE != kCeDhidden)
      if (tiles(pc.len, 256) < 256) return launch_tile<T, MODE, 4, 1, 1, 1, 4>(a, pc, stream);
    launch_tile<T, MODE, 8, 1, 1, 1, 4>(a, pc, stream);
  }
}

// Slices of a row in STATS: the waves along m of its tiles.
int64_t slices_of(int64_t V, int64_t N, bool bf16) {
  const int rows = ce_rows_of_tile(N, bf16);
  if (few_tiles(V, N, bf16)) return tiles(V, 64) * 2;
  if (rows == 32) return tiles(V, 256) < 256 ? tiles(V, 128) * 4 : tiles(V, 256) * 8;
  if (rows == 64) return tiles(V, 256) * 4;
  if (rows == 128) return bf16 ? tiles(V, 256) * 4 : tiles(V, 128) * 2;
  return tiles(V, 256) * 2;
}

template <typename T>
hipError_t launch_matrix(CeArgs a, bool backward, hipStream_t stream) {
  constexpr bool kBf16 = sizeof(T) == 2;
  CePiece pc = {0, a.V, 1, 0, 0};
  // forward: rows are read where they are if one descriptor reaches them all
  pc.gather = !backward && (unsigned __int128)a.N * (unsigned __int128)a.hidden_stride * sizeof(T) < kBufMost;
  // a tile's worth of rows or less: a list would save no product
  pc.direct = pc.gather && a.N <= 256;
  const bool few = backward && a.N <= kCeFewRows;
  if (few) hipLaunchKernelGGL(ce_list_copy_kernel<T>, dim3((unsigned)a.N), dim3(256), 0, stream, a);
  else if (!pc.direct) launch_cross_entropy_prep(a, backward, stream);
  if (!pc.gather && !few) hipLaunchKernelGGL(ce_copy_kernel<T>, dim3((unsigned)a.N), dim3(256), 0, stream, a);
  if (!backward) {
    a.slices = slices_of(a.V, a.N, kBf16);
    launch_rows<T, kCeStats>(a, pc, stream);
    launch_cross_entropy_combine(a, pc.direct, stream);
    return hipGetLastError();
  }
  for (int64_t v0 = 0; v0 < a.V; v0 += a.ds_ld) {
    pc.v0 = v0;
    pc.len = a.V - v0 < a.ds_ld ? a.V - v0 : a.ds_ld;
    pc.first = v0 == 0;
    launch_rows<T, kCeDs>(a, pc, stream);
    if (a.out_dhidden) launch_rows<T, kCeDhidden>(a, pc, stream);
    if (a.out_dweight) launch_rows<T, kCeDweight>(a, pc, stream);
  }
  if (a.out_dhidden) {
    const dim3 grid((unsigned)a.N, (unsigned)tiles(a.D, 1024));
    const int rows = ce_rows_of_tile(a.N, kBf16);
    if (ce_columns_of_tile(a.N, kBf16) == 128)
      hipLaunchKernelGGL((ce_dhidden_parts_kernel<T, 128>), grid, dim3(256), 0, stream, a, rows);
    else
      hipLaunchKernelGGL((ce_dhidden_parts_kernel<T, 256>), grid, dim3(256), 0, stream, a, rows);
  }
  return hipGetLastError();
}

}  // namespace

bool cross_entropy_matrix_path(const CeArgs& a, int dtype) {
  // rows on the 16-byte grid, and a tile's rows within 2^31 bytes
  const int64_t each = dtype == ARCS_DTYPE_BF16 ? 8 : 4, most = int64_t(1) << (dtype == ARCS_DTYPE_BF16 ? 22 : 21);
  if (a.D % each != 0 || a.hidden_stride % each != 0 || a.weight_stride % each != 0 || a.weight_stride >= most) return false;
  return (((uintptr_t)a.hidden | (uintptr_t)a.weight | (uintptr_t)a.out_dweight | (uintptr_t)a.out_dhidden) & 15u) == 0;
}

hipError_t launch_cross_entropy_matrix(const CeArgs& a, int dtype, bool backward, hipStream_t stream) {
  return dtype == ARCS_DTYPE_BF16 ? launch_matrix<__bf16>(a, backward, stream) : launch_matrix<float>(a, backward, stream);
}

}  // namespace arcs
