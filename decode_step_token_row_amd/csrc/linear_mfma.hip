// The linear layer's products on the matrix instructions.
//
//   C[m, n] = sum_k A[m, k] B[n, k],  stored at out[n][m]
//
// with the operands' rows along k or along m (n), see linear.hpp.  Tiles of 128 bytes of k
// go from memory to LDS by the loads that write LDS directly, S deep, one barrier a
// tile; operands whose rows run along m are read back transposed.  FORWARD's results go
// through bias, activation and residual in registers.  Where whole tiles would leave
// compute units without work, all workgroups share the tiles evenly, each a part of k of
// one or more: their float32 parts go to the workspace and linear_join_kernel adds them up
// in the workgroups' order, so that results do not depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.hpp"
#include "linear_device.hpp"
#include "lds_load.hpp"
#include "mfma_tile.hpp"

namespace arcs {

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
struct LinTile {
  static constexpr int kThreads = WM * WN * 64, kWaves = WM * WN;
  static constexpr int BM = WM * MT * 32, BN = WN * NT * 32;
  static constexpr bool kAOuter = MODE != kLinForward, kBOuter = MODE == kLinDweight;
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int kTK = 128 / sizeof(T);  // k of one tile
  static constexpr int kABytes = BM * 128, kBBytes = BN * 128, kStage = kABytes + kBBytes;
  static constexpr int kALoads = BM / 8, kBLoads = BN / 8;  // of 1024 bytes each
  static constexpr int kAPer = (kALoads + kWaves - 1) / kWaves, kBPer = (kBLoads + kWaves - 1) / kWaves;
  static constexpr int kPer = kAPer + kBPer;
  // bfloat16 results go out through 32 rows of kOutM columns a wave
  static constexpr int kOutM = MT % 2 == 0 && S * kStage + kWaves * 32 * 64 * 2 <= 163840 ? 64 : 32;
  static constexpr int kOutBytes = 32 * kOutM * 2;
  static constexpr int kLds = S * kStage + kWaves * kOutBytes;
};

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S, bool SHARED>
__global__ __launch_bounds__(WM* WN * 64, 2) void linear_tile_kernel(LinearProduct p) {
  using C = LinTile<T, MODE, WM, WN, MT, NT, S>;
  constexpr int BM = C::BM, BN = C::BN, kTK = C::kTK;
  constexpr int64_t E = sizeof(T);
  __shared__ __align__(1024) char lds[SHARED ? S * C::kStage : C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t M = p.M, N = p.N, K = p.K;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(ARCS_LDS char*)lds;

  // The tiles of this workgroup.  Workgroups go round the eight dies in turn; a die gets
  // neighbouring tiles, which share their operands in its L2.  SHARED: worker w has the
  // tiles from w T / workers on, the first and last of them in part.
  const int mt = (int)((M + BM - 1) / BM), nt = (int)((N + BN - 1) / BN), all = mt * nt;
  int job, job_end, job_step = 1, worker = 0;
  if (SHARED) {
    worker = ((int)blockIdx.x & 7) * (p.shape.workers / 8) + ((int)blockIdx.x >> 3);
    job = (int)((int64_t)worker * all / p.shape.workers);
    job_end = (int)(((int64_t)(worker + 1) * all + p.shape.workers - 1) / p.shape.workers);
  } else {
    const int chunk = (all + 7) / 8, first = ((int)blockIdx.x & 7) * chunk;
    job = first + ((int)blockIdx.x >> 3);
    job_end = first + chunk < all ? first + chunk : all;
    job_step = (int)gridDim.x / 8;
  }
  if (job >= job_end) return;

  // The tile that is loaded: its first k, descriptors there, and the lanes' offsets.
  int64_t m0, n0, k_lo;
  int nk, shift = 0;
  const char *pa, *pb;
  int64_t na, nb;
  uint32_t oa[C::kAPer], ob[C::kBPer];
  const T *A = (const T*)p.a, *B = (const T*)p.b;
  const int64_t step_a = C::kAOuter ? kTK * p.lda * E : 128;
  const int64_t step_b = C::kBOuter ? kTK * p.ldb * E : 128;
  auto place = [&](int job) {
    tile_place(job, mt, nt, m0, n0);
    m0 *= BM;
    n0 *= BN;
    k_lo = 0;
    int64_t k_hi = K;
    if (SHARED) {
      const int64_t tiles_k = (K + kTK - 1) / kTK;
      const int64_t from = (int64_t)worker * all - (int64_t)job * p.shape.workers, to = from + all;
      if (from > 0) k_lo = from * tiles_k / p.shape.workers * kTK;
      if (to < p.shape.workers) k_hi = to * tiles_k / p.shape.workers * kTK;
    }
    nk = k_hi > k_lo ? (int)((k_hi - k_lo + kTK - 1) / kTK) : 0;
    // With one tile of rows every workgroup reads other weight rows, and begun together all
    // ask for the same columns of rows a power of two apart, so for few of the memory's
    // channels at a time: each begins its walk along k elsewhere.
    if (!C::kAOuter && !SHARED) shift = nt == 1 ? (int)((uint32_t)job * 2654435761u >> 16) % nk : 0;
    na = nb = kBufMost;
#pragma unroll
    for (int t = 0; t < C::kAPer; ++t) {
      const int inst = (wave + t * C::kWaves) % C::kALoads;
      int r, c;
      if (!C::kAOuter) {
        inner_place<T>(inst, lane, r, c);
        const int64_t left = M - 1 - m0;
        oa[t] = (uint32_t)((r < left ? r : left) * p.lda * E + c * E);
      } else {
        outer_place<T, BM>(inst, lane, r, c);
        oa[t] = m0 + c < M ? (uint32_t)(r * p.lda * E + c * E) : kNoLoad;
      }
    }
#pragma unroll
    for (int t = 0; t < C::kBPer; ++t) {
      const int inst = (wave + t * C::kWaves) % C::kBLoads;
      int r, c;
      if (!C::kBOuter) {
        inner_place<T>(inst, lane, r, c);
        const int64_t left = N - 1 - n0;
        ob[t] = (uint32_t)((r < left ? r : left) * p.ldb * E + c * E);
      } else {
        outer_place<T, BN>(inst, lane, r, c);
        ob[t] = n0 + c < N ? (uint32_t)(r * p.ldb * E + c * E) : kNoLoad;
      }
    }
    if (C::kAOuter) {
      pa = (const char*)(A + k_lo * p.lda + m0);
      na = ((K - k_lo) * p.lda - m0) * E;
    } else {
      pa = (const char*)(A + m0 * p.lda + k_lo);
    }
    if (C::kBOuter) {
      pb = (const char*)(B + k_lo * p.ldb + n0);
      nb = ((K - k_lo) * p.ldb - n0) * E;
    } else {
      pb = (const char*)(B + n0 * p.ldb + k_lo);
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
    if (!C::kAOuter && !SHARED) {
      kt += shift;
      kt = kt >= nk ? kt - nk : kt;
    }
    s.a = uniform4(buffer_of(pa + kt * step_a, none ? 0 : C::kAOuter ? na - kt * step_a : (int64_t)kBufMost));
    s.b = uniform4(buffer_of(pb + kt * step_b, none ? 0 : C::kBOuter ? nb - kt * step_b : (int64_t)kBufMost));
    // rows along k: the columns of the last tile past K are zeros
    const int64_t left = K - k_lo - (int64_t)kt * kTK;
    s.left = (uint32_t)(left < kTK ? left > 0 ? left : 0 : kTK);
    return s;
  };
  auto issue_one = [&](const Source& s, int t) {
    if (t < C::kAPer) {
      const uint32_t off = !C::kAOuter && ka[t & 1] >= s.left ? kNoLoad : oa[t];
      const uint32_t to = s.to + ((wave + t * C::kWaves) % C::kALoads) * 1024u;
      if (t == 0) load_to_lds<true>(to, off, s.a);
      else load_to_lds<false>(to, off, s.a);
    } else {
      t -= C::kAPer;
      const uint32_t off = !C::kBOuter && kb[t & 1] >= s.left ? kNoLoad : ob[t];
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
      for (int q = 0; q < kProducts; ++q) {
        acc[q / NT][q % NT] = product(fa[1][q / NT], fb[1][q % NT], acc[q / NT][q % NT]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int l = q * kEach; l < (q + 1) * kEach && l < C::kPer; ++l) issue_one(from, l);
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
    if (SHARED) {
      // part worker + job of the slab, [BN][BM]: each pair of them is met once
      float* part = p.slab + (int64_t)(worker + done) * (BM * BN);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int nl = wn + j * 32 + fr;
        if (en0 + nl >= N) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (row_of(i, q * 4) >= m_left) continue;
            const f32x4 v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
            *(f32x4*)(part + nl * BM + mw + row_of(i, q * 4)) = v;
          }
      }
    } else {
      // out = residual + act(acc + bias); pass 0 writes acc + bias where it is wanted
      const bool plain = MODE != kLinForward;
      for (int pass = plain || p.pre == nullptr ? 1 : 0; pass < 2; ++pass) {
        void* to = pass == 0 ? p.pre : p.out;
        const int64_t ldo = pass == 0 ? p.ldp : p.ldo;
        const bool to_bf16 = pass == 0 || MODE != kLinForward ? C::kBf16 : p.out_bf16 != 0;
        const bool biased = !plain && p.bias != nullptr, added = !plain && pass == 1 && p.residual != nullptr;
        auto finish = [&](int i, int j, int q, float (&v)[4]) {
          const int ml = row_of(i, q * 4), left = m_left - ml;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][q * 4 + e];
          if (plain || left <= 0) return;
          if (biased) {
            float b[4];
            load_some<T, 4>((const T*)p.bias + em0 + mw + ml, left, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += b[e];
          }
          if (pass == 1 && p.act != ARCS_ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = act_value(v[e], p.act, p.cap);
          }
          const int64_t n = en0 + wn + j * 32 + fr;
          if (added && n < N) {
            float r[4];
            load_some<T, 4>((const T*)p.residual + n * p.ldr + em0 + mw + ml, left, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += r[e];
          }
        };
        if (!to_bf16) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int64_t n = en0 + wn + j * 32 + fr;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float v[4];
                finish(i, j, q, v);
                const int left = m_left - row_of(i, q * 4);
                if (n < N && left > 0) store_some<float, 4>((float*)to + n * ldo + em0 + mw + row_of(i, q * 4), left, v);
              }
          }
        } else {
          // 32 rows n of kOutM columns at a time through the wave's own part of LDS, so
          // that whole lines are stored.  16-byte chunk c of row n at c ^ n.
          constexpr int kOutM = C::kOutM, kChunks = kOutM / 8, kTiles = kOutM / 32;
          char* own = lds + (SHARED ? 0 : S * C::kStage + wave * C::kOutBytes);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i0 = 0; i0 < MT; i0 += kTiles) {
#pragma unroll
              for (int i = i0; i < i0 + kTiles; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  float v[4];
                  finish(i, j, q, v);
                  bf16x4 w;
#pragma unroll
                  for (int e = 0; e < 4; ++e) w[e] = (__bf16)v[e];
                  const int ml = row_of(i - i0, q * 4) + 4 * fh;
                  *(bf16x4*)(own + fr * (kOutM * 2) + (((ml >> 3) ^ (fr & (kChunks - 1))) * 16) + (ml & 4) * 2) = w;
                }
              wait_lds();
              const int64_t ms = em0 + wm + i0 * 32;
#pragma unroll
              for (int t = 0; t < 32 * kChunks / 64; ++t) {
                const int nl = (t * 64 + lane) / kChunks, c = (t * 64 + lane) % kChunks;
                const int64_t n = en0 + wn + j * 32 + nl, m = ms + c * 8;
                const u32x4 v = *(const u32x4*)(own + nl * (kOutM * 2) + ((c ^ (nl & (kChunks - 1))) * 16));
                if (n >= N || m >= M) continue;
                uint16_t* at = (uint16_t*)to + n * ldo + m;
                if (m + 8 <= M) {
                  store16(at, v);
                } else {
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    if (m + e < M) at[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                }
              }
              wait_lds();  // read before the next columns are written
            }
        }
      }
    }
    if (!more) break;
  }
}

// Shared tiles: the parts of each added up in the workers' order, and the epilogue.
template <typename T, bool FORWARD>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearProduct p) {
  const int64_t n = blockIdx.x, m = (int64_t)blockIdx.y * 1024 + threadIdx.x * 4;
  if (m >= p.M) return;
  const int BM = p.shape.columns, BN = p.shape.rows, workers = p.shape.workers;
  const int mt = (int)((p.M + BM - 1) / BM), nt = (int)((p.N + BN - 1) / BN), all = mt * nt;
  const int job = tile_index((int)(m / BM), (int)(n / BN), mt, nt);
  const int lo = (int)((int64_t)job * workers / all), hi = (int)(((int64_t)(job + 1) * workers + all - 1) / all);
  const float* part = p.slab + ((int64_t)job * BN + n % BN) * BM + m % BM;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int w = lo; w < hi; ++w) sum += *(const f32x4*)(part + (int64_t)w * (BN * BM));
  const int left = (int)(p.M - m < 4 ? p.M - m : 4);
  float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  if (FORWARD) {
    if (p.bias != nullptr) {
      float b[4];
      load_some<T, 4>((const T*)p.bias + m, left, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b[e];
    }
    if (p.pre != nullptr) store_some<T, 4>((T*)p.pre + n * p.ldp + m, left, v);
    if (p.act != ARCS_ACT_NONE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value(v[e], p.act, p.cap);
    }
    if (p.residual != nullptr) {
      float r[4];
      load_some<T, 4>((const T*)p.residual + n * p.ldr + m, left, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += r[e];
    }
    if (p.out_bf16) store_some<__bf16, 4>((__bf16*)p.out + n * p.ldo + m, left, v);
    else store_some<float, 4>((float*)p.out + n * p.ldo + m, left, v);
  } else {
    store_some<T, 4>((T*)p.out + n * p.ldo + m, left, v);
  }
}

namespace {

int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
void launch_tile(const LinearProduct& p, hipStream_t stream) {
  using C = LinTile<T, MODE, WM, WN, MT, NT, S>;
  if (p.shape.workers > 0) {
    hipLaunchKernelGGL((linear_tile_kernel<T, MODE, WM, WN, MT, NT, S, true>), dim3((unsigned)p.shape.workers),
                       dim3(C::kThreads), 0, stream, p);
    hipLaunchKernelGGL((linear_join_kernel<T, MODE == kLinForward>), dim3((unsigned)p.N, (unsigned)tiles(p.M, 1024)),
                       dim3(256), 0, stream, p);
    return;
  }
  // as many workgroups as the compute units hold (by LDS), at most
  constexpr int64_t kMost = 256 * (163840 / C::kLds);
  const int64_t all = tiles(p.M, C::BM) * tiles(p.N, C::BN);
  const int64_t blocks = all < kMost ? tiles(all, 8) * 8 : kMost;
  hipLaunchKernelGGL((linear_tile_kernel<T, MODE, WM, WN, MT, NT, S, false>), dim3((unsigned)blocks),
                     dim3(C::kThreads), 0, stream, p);
}

template <typename T, int MODE>
void launch_mode(const LinearProduct& p, hipStream_t stream) {
  launch_tile<T, MODE, 2, 2, 2, 2, 2>(p, stream);
}

}  // namespace

LinearShape linear_shape(int mode, int64_t M, int64_t N, int64_t K, bool bf16) {
  (void)mode;
  (void)bf16;
  const int64_t all = tiles(M, 128) * tiles(N, 128), tiles_k = tiles(K, bf16 ? 64 : 32);
  LinearShape s = {128, 128, 0};
  if (all < 256 && all * tiles_k >= 512) s.workers = 256;
  return s;
}

hipError_t launch_linear_product(const LinearProduct& p, int mode, int dtype, hipStream_t stream) {
  if (dtype == ARCS_DTYPE_BF16) {
    if (mode == kLinForward) launch_mode<__bf16, kLinForward>(p, stream);
    else if (mode == kLinDhidden) launch_mode<__bf16, kLinDhidden>(p, stream);
    else launch_mode<__bf16, kLinDweight>(p, stream);
  } else {
    if (mode == kLinForward) launch_mode<float, kLinForward>(p, stream);
    else if (mode == kLinDhidden) launch_mode<float, kLinDhidden>(p, stream);
    else launch_mode<float, kLinDweight>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace arcs
