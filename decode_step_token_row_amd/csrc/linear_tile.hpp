// The linear layer's products on the matrix instructions.
//
//   C[m, n] = sum_k A[m, k] B[n, k],  stored at out[n][m]
//
// with the operands' rows along k or along m (n), see linear.hpp.  Tiles of 128 bytes of k
// go from memory to LDS by the loads that write LDS directly, S deep; operands whose rows run
// along m are read back transposed.  Results go out through LDS, eight columns of a row a
// lane, FORWARD's through bias, activation and residual on their way; what those read is asked
// for two products ahead.  Where whole tiles would leave compute units without work, all
// workgroups share the tiles evenly, each a part of k of one or more: their float32 parts
// go to the workspace and linear_join_kernel adds them up in the workgroups' order, so that
// results do not depend on timing.
//
// What bounds it, at 4,096 x 4,096 x 4,096 in bfloat16 (256 tiles of 256 x 256, one a compute
// unit): forward 114 to 120 us (1,150 to 1,200 TFLOP/s), dhidden 109 to 116, dweight 110 to 115; a large
// library product reaches 1,450 TFLOP/s.  The matrix units are busy 60 % of a gradient's cycles; the rest is
// the way of 1.07 GB from L2 to LDS, as far as the products do not cover it.  Steps that counted: the
// next loads halfway through the third of the four steps instead of in the last, with a second meeting of
// the workgroup for it (head of 256 rows 306 -> 286 us); priority for the multiplying workgroup of two
// on a compute unit.  Steps that did not: loads spread over the whole tile with a third place for A (121
// us), four waves of 128 x 128 (116 to 125), walks along k begun at different places, other cache policies
// of the loads.  Rows of a power-of-two length cost the forward pass more than the others (4,032
// columns of k were 13 % faster before the second meeting).
// The epilogue with bias, silu, residual and z written beside the output adds 9 to 14 us to the forward
// pass of that size (100 MB more, 20 us at the rate of a copy); it added 45 while every
// element had its own branch on the activation and its residual was waited for.  One kernel has all of
// the epilogue's choices, and the 256 x 256 forward one keeps 15 vector registers in scratch memory for
// them (64 bytes a lane, filled before and read after the loop over k), the 128 x 128 one 129 scalar
// registers in lanes of vector registers: the former writes 83 MB for 67 MB of results, the gradients,
// which keep theirs, 35.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear.hpp"
#include "linear_device.hpp"
#include "lds_load.hpp"
#include "mfma_tile.hpp"

namespace arcs {

// The epilogue on E consecutive results of row n, `left` of which exist:
// FORWARD: out = residual + act(v + bias), pre = v + bias.
template <typename T, bool FORWARD, int E>
__device__ __forceinline__ void linear_finish(const LinearProduct& p, int64_t n, int64_t m, int left, float (&v)[E],
                                              const float (&bias)[E], const float (&residual)[E]) {
  if constexpr (FORWARD) {
    if (p.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += bias[e];
    }
    if (p.pre != nullptr) store_some<T, E>((T*)p.pre + n * p.ldp + m, left, v);
    act_values(v, p.act, p.cap, p.inv_cap);
    if (p.residual != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += residual[e];
    }
    if (p.out_bf16) store_some<__bf16, E>((__bf16*)p.out + n * p.ldo + m, left, v);
    else store_some<float, E>((float*)p.out + n * p.ldo + m, left, v);
  } else {
    store_some<T, E>((T*)p.out + n * p.ldo + m, left, v);
  }
}

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
  static constexpr int kOutBytes = 32 * 32 * 4;  // of a wave, for results on their way out
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
    // A die gets workers that begin near each other along k, in whichever tiles, so that they share
    // rows of both operands in its L2: worker w begins w T mod workers into a tile, and with
    // T = g odd, g dividing workers, the workers sorted by that are rank / g times the inverse of
    // odd, and those workers / g on (dhidden of 1,037 x 5,003 x 1,000 39 us, of 128 x 11,008 x 4,096
    // 31; 44 and 32 with neighbours in w; forward of 512 x 4,096 x 11,008 66 and 72, of 128 x 11,008 x
    // 4,096 39 and 38).
    const int workers = p.shape.workers, rank = ((int)blockIdx.x & 7) * (workers / 8) + ((int)blockIdx.x >> 3);
    const int low = all & -all, g = low < workers ? low : workers, q = workers / g;
    const uint32_t odd = (uint32_t)(all / g);
    uint32_t inverse = odd;  // modulo 2^3, 2^6, 2^12
    inverse *= 2u - odd * inverse;
    inverse *= 2u - odd * inverse;
    worker = (int)((uint32_t)(rank / g) * inverse & (uint32_t)(q - 1)) + rank % g * q;
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
  int nk, shift = 0, last;                     // last: columns of k of the last tile
  const char *pa, *pb;
  uint32_t na = kBufMost, nb = kBufMost, last_na = kBufMost, last_nb = kBufMost;  // bytes of a tile's descriptors
  // the next tile to load: how far along k, where its rows begin, its place in LDS
  int at, stage;
  const char *at_a, *at_b;
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
    // channels at a time: each begins its walk along k elsewhere.  Tiles of the same weight
    // rows share their loads, and begin together.
    if (!C::kAOuter && !SHARED) shift = nt == 1 ? (int)((uint32_t)job * 2654435761u >> 16) % nk : 0;
    const int64_t left_k = K - k_lo - (int64_t)(nk - 1) * kTK;
    last = (int)(left_k < kTK ? left_k : kTK);
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
      na = (uint32_t)((kTK * p.lda - m0) * E);
      last_na = (uint32_t)((last * p.lda - m0) * E);
    } else {
      pa = (const char*)(A + m0 * p.lda + k_lo);
    }
    if (C::kBOuter) {
      pb = (const char*)(B + k_lo * p.ldb + n0);
      nb = (uint32_t)((kTK * p.ldb - n0) * E);
      last_nb = (uint32_t)((last * p.ldb - n0) * E);
    } else {
      pb = (const char*)(B + n0 * p.ldb + k_lo);
    }
    at = shift;
    stage = 0;
    at_a = pa + shift * step_a;
    at_b = pb + shift * step_b;
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

  // The loads of the tile after the last one asked for, kt, of which a wave has kPer; tiles past
  // the last read nothing (zeros go to a buffer that is free), so that the waits always count the
  // same.
  struct Source {
    u32x4 a, b;
    uint32_t to, left;
  };
  auto source = [&](int kt) {
    Source s;
    s.to = lds0 + (uint32_t)stage;
    stage = stage == (S - 1) * C::kStage ? 0 : stage + C::kStage;
    const bool none = kt >= nk, ends = at == nk - 1;
    s.a = uniform4(buffer_of(at_a, none ? 0u : ends ? last_na : na));
    s.b = uniform4(buffer_of(at_b, none ? 0u : ends ? last_nb : nb));
    s.left = (uint32_t)(ends ? last : kTK);  // rows along k: the columns of the last tile past K are zeros
    ++at;
    at_a += step_a;
    at_b += step_b;
    if (!C::kAOuter && !SHARED && at == nk) {
      at = 0;
      at_a = pa;
      at_b = pb;
    }
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
  // Two deep, a tile's loads go out during the tile two before; deeper, into the place of the
  // tile before, while a tile multiplies (384 x 2,048 x 1,024 in float32 24.5 us, 27 with the loads
  // together at the end of the tile; all fragments of a tile read at once, with places for S
  // tiles, 28).
  constexpr int kAhead = S == 2 ? 2 : S - 1;
  auto issue_first = [&]() {
#pragma unroll
    for (int t = 0; t < kAhead; ++t) {
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
  // a tile reads from the next one: there the workgroup meets, once a tile, and the
  // next tile has landed.
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
    wait_loads<(kAhead - 1) * C::kPer>();
    __builtin_amdgcn_s_barrier();
    read(0, 0);
    for (int kt = 0; kt < nk; ++kt) {
      constexpr int kProducts = MT * NT;
      if constexpr (S == 2) {
        // Two deep, the next loads go out as soon as every wave has read its last fragments of
        // the tile: the workgroup meets once more for that, halfway through step 2.
        // Two workgroups share a compute unit in tiles of four waves: there the one that multiplies
        // goes first (512 x 11,008 x 4,096 68 us without, 63 with; 256 x 256 tiles 1 to 3 % slower with).
        constexpr bool kPriority = C::kWaves == 4;
        constexpr int kHalf = kProducts / 2, kEarly = C::kPer / 2;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          read(kt, ks + 1);
          if (kPriority) __builtin_amdgcn_s_setprio(1);
          multiply(ks);
          if (kPriority) __builtin_amdgcn_s_setprio(0);
        }
        read(kt, 3);
        const Source from = source(kt + S);
        if (kPriority) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int q = 0; q < kHalf; ++q)
          acc[q / NT][q % NT] = product(fa[0][q / NT], fb[0][q % NT], acc[q / NT][q % NT]);
        __builtin_amdgcn_sched_barrier(0);
        if (kPriority) __builtin_amdgcn_s_setprio(0);
        wait_lds();
        __builtin_amdgcn_s_barrier();
        constexpr int kRest = kProducts - kHalf, kEach1 = (kEarly + kRest - 1) / kRest;
#pragma unroll
        for (int q = kHalf; q < kProducts; ++q) {
          acc[q / NT][q % NT] = product(fa[0][q / NT], fb[0][q % NT], acc[q / NT][q % NT]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int l = (q - kHalf) * kEach1; l < (q - kHalf + 1) * kEach1 && l < kEarly; ++l) issue_one(from, l);
          __builtin_amdgcn_sched_barrier(0);
        }
        wait_loads<kEarly>();  // tile kt + 1 has landed
        __builtin_amdgcn_s_barrier();
        read(kt + 1, 0);
        constexpr int kEach2 = (C::kPer - kEarly + kProducts - 1) / kProducts;
#pragma unroll
        for (int q = 0; q < kProducts; ++q) {
          acc[q / NT][q % NT] = product(fa[1][q / NT], fb[1][q % NT], acc[q / NT][q % NT]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int l = kEarly + q * kEach2; l < kEarly + (q + 1) * kEach2 && l < C::kPer; ++l) issue_one(from, l);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        // every wave has read the tile before: its place is free
        const Source from = source(kt + kAhead);
        constexpr int kEach = (C::kPer + 3 * kProducts - 1) / (3 * kProducts);
#pragma unroll
        for (int ks = 0; ks < 3; ++ks) {
          read(kt, ks + 1);
#pragma unroll
          for (int q = 0; q < kProducts; ++q) {
            acc[q / NT][q % NT] = product(fa[ks & 1][q / NT], fb[ks & 1][q % NT], acc[q / NT][q % NT]);
            const int l0 = (ks * kProducts + q) * kEach;
#pragma unroll
            for (int l = l0; l < l0 + kEach && l < C::kPer; ++l) issue_one(from, l);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        wait_loads<(kAhead - 1) * C::kPer>();  // tile kt + 1 has landed
        wait_lds();                            // this wave's reads of tile kt are done
        __builtin_amdgcn_s_barrier();
        read(kt + 1, 0);
        multiply(3);
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
    // 8 (r / 4) + 4 (lane / 32) + r % 4.
    if constexpr (SHARED) {
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
            const int ml = wm + 4 * fh + i * 32 + q * 8;
            if (em0 + ml >= M) continue;
            const f32x4 v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
            *(f32x4*)(part + nl * BM + ml) = v;
          }
      }
    } else {
      // One product after the other goes through the wave's own part of LDS, 32 rows n of 32
      // float32, 16-byte chunk c of row n at c ^ (n % 8), so that a lane gets 8 columns of a row
      // and the epilogue stands in the code once.
      char* own = lds + S * C::kStage + wave * C::kOutBytes;
      // what the epilogue reads of a product's place: asked for two products ahead
      struct Beside {
        Raw8<T> bias, residual[2];
      };
      auto ask = [&](int block, Beside& x) {
        if constexpr (MODE == kLinForward) {
          const int64_t m = em0 + wm + block / NT * 32 + (lane & 3) * 8;
          const int left = (int)(M - m < 8 ? M - m : 8);
          if (p.bias != nullptr) load_raw(x.bias, (const T*)p.bias + m, left);
          if (p.residual != nullptr) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int64_t n = en0 + wn + block % NT * 32 + t * 16 + (lane >> 2);
              load_raw(x.residual[t], (const T*)p.residual + n * p.ldr + m, n < N ? left : 0);
            }
          }
        }
      };
      auto finish = [&](int block, const Beside& x) {
        asm volatile("" : "+s"(block));  // a branch for each product, not a select of their registers
#pragma unroll
        for (int c = 0; c < MT * NT; ++c) {
          if (block != c) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& y = acc[c / NT][c % NT];
            const f32x4 v = {y[q * 4], y[q * 4 + 1], y[q * 4 + 2], y[q * 4 + 3]};
            *(f32x4*)(own + fr * 128 + (((q * 2 + fh) ^ (fr & 7)) * 16)) = v;
          }
        }
        wait_lds();
        const int64_t m = em0 + wm + block / NT * 32 + (lane & 3) * 8;
        const int left = (int)(M - m < 8 ? M - m : 8);
        float bias[8], residual[8];
        widen_raw(x.bias, bias);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int nl = t * 16 + (lane >> 2), c = (lane & 3) * 2;
          const int64_t n = en0 + wn + block % NT * 32 + nl;
          const f32x4 y0 = *(const f32x4*)(own + nl * 128 + ((c ^ (nl & 7)) * 16));
          const f32x4 y1 = *(const f32x4*)(own + nl * 128 + (((c + 1) ^ (nl & 7)) * 16));
          float v[8] = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
          widen_raw(x.residual[t], residual);
          if (n < N && left > 0) linear_finish<T, MODE == kLinForward, 8>(p, n, m, left, v, bias, residual);
        }
        wait_lds();  // read before the next product is written
      };
      constexpr int kBlocks = MT * NT;
      Beside x = {}, y = {};
      ask(0, x);
      if constexpr (kBlocks > 1) {
        ask(1, y);
        for (int block = 0; block < kBlocks; block += 2) {
          finish(block, x);
          if (block + 2 < kBlocks) ask(block + 2, x);
          finish(block + 1, y);
          if (block + 3 < kBlocks) ask(block + 3, y);
        }
      } else {
        finish(0, x);
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
  float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  const int left = (int)(p.M - m < 4 ? p.M - m : 4);
  float bias[4] = {}, residual[4] = {};
  if (FORWARD && p.bias != nullptr) load_some<T, 4>((const T*)p.bias + m, left, bias);
  if (FORWARD && p.residual != nullptr) load_some<T, 4>((const T*)p.residual + n * p.ldr + m, left, residual);
  linear_finish<T, FORWARD, 4>(p, n, m, left, v, bias, residual);
}

template <typename T, int MODE, int WM, int WN, int MT, int NT, int S>
bool launch_linear_tile(const LinearProduct& p, hipStream_t stream) {
  using C = LinTile<T, MODE, WM, WN, MT, NT, S>;
  if (p.shape.columns != C::BM || p.shape.rows != C::BN) return false;
  if (p.shape.workers > 0) {
    hipLaunchKernelGGL((linear_tile_kernel<T, MODE, WM, WN, MT, NT, S, true>), dim3((unsigned)p.shape.workers),
                       dim3(C::kThreads), 0, stream, p);
    hipLaunchKernelGGL((linear_join_kernel<T, MODE == kLinForward>),
                       dim3((unsigned)p.N, (unsigned)linear_tiles(p.M, 1024)), dim3(256), 0, stream, p);
    return true;
  }
  // as many workgroups as the compute units hold (by LDS), at most
  constexpr int64_t kMost = 256 * (163840 / C::kLds);
  const int64_t all = linear_tiles(p.M, C::BM) * linear_tiles(p.N, C::BN);
  const int64_t blocks = all < kMost ? linear_tiles(all, 8) * 8 : kMost;
  hipLaunchKernelGGL((linear_tile_kernel<T, MODE, WM, WN, MT, NT, S, false>), dim3((unsigned)blocks),
                     dim3(C::kThreads), 0, stream, p);
  return true;
}

}  // namespace arcs
