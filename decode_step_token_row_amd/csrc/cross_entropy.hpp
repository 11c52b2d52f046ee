// Host and device declarations shared by the linear cross entropy's kernels.
//
//   z = hidden weight^T / T          [N, V], never kept whole
//   loss_n = logsumexp(z_n) - z_n[t_n]
//   dz = (softmax(z) - onehot(t)) * grad_loss / T
//   dhidden = dz weight,  dweight = dz^T hidden
//
// Rows whose target is ignore_index (masked) or refused (a target outside the
// vocabulary, a temperature that is no positive finite number) are left out of
// every product: a row list built on the device holds the others.  (Forward calls
// of few rows compute all rows and write only the others' results.)  Either way
// NaN in a left-out row's hidden states reaches nothing.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "arcs.h"

namespace arcs {

// What the device knows of a call's rows once the list is built.
struct CeHeader {
  int32_t count;  // rows in the list
  float gmax;     // largest finite |grad_loss / T| of them (1 if that is 0)
  int32_t pad[62];
};
static_assert(sizeof(CeHeader) == 256, "workspace header");

// One listed row.
struct CeRow {
  int32_t row;     // its place in the call's arrays
  int32_t target;  // in [0, V)
  float a;         // log2(e) / T: logits in base 2 are dot * a
  float c;         // (grad_loss / T) / gmax
  float lse2;      // its logsumexp in base 2 (backward), rounded,
  float rest;      // and 2 to minus what the rounding left: p = 2^(dot * a - lse2) * rest
  int32_t pad[2];
};
static_assert(sizeof(CeRow) == 32, "row record");

struct CeArgs {
  const void* hidden;
  int64_t hidden_stride;
  const void* weight;
  int64_t weight_stride;
  int64_t N, V, D;
  const int32_t* targets;
  int32_t ignore_index;
  const float* temperature;  // [N] or NULL
  float* out_loss;           // forward
  float* out_lse;
  int32_t* out_status;       // or NULL
  const float* lse;          // backward
  const float* grad_loss;
  void* out_dhidden;         // [N, D] or NULL
  void* out_dweight;         // [V, D] or NULL
  // workspace
  CeHeader* head;
  CeRow* rows;      // [N]
  int32_t* place;   // [N] backward: a row's place in the list, -1 if it is not listed
  float2* partial;  // forward: [N][slices] (maximum, sum of 2^(y - maximum)) of y = z * log2(e)
  int64_t slices;
  float* dtarget;   // forward: [N] the target's dot product
  void* ds;         // backward: [N][ds_ld] dz / gmax of one piece of the vocabulary
  int64_t ds_ld;    // (also the piece's length)
  float* slab;      // backward: partial sums of dhidden / gmax: [splits][N][D], or parts of tiles (matrix kernels)
  int splits;       // general kernel: of k in dhidden
  int workers;      // matrix kernels: workgroups that share dhidden's tiles
  void* hc;         // matrix kernels: [N][D] hidden states of the listed rows (backward, and forward
                    // where one descriptor does not reach all rows)
};

// The workspace's parts, in bytes from its start.
struct CePlan {
  size_t rows, place, partial, dtarget, ds, slab, hc, total;
  int64_t slices, piece;
  int splits, workers;
  bool fits;  // the sizes fit size_t and the launch grids
};
CePlan cross_entropy_plan(int64_t N, int64_t V, int64_t D, int dtype, bool backward);

// Matrix kernels: a tile's n side (the call's rows) and, in dhidden, its m side.
inline int ce_rows_of_tile(int64_t N, bool bf16) { return N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 || !bf16 ? 128 : 256; }
inline int ce_columns_of_tile(int64_t N, bool bf16) { return !bf16 && N > 64 ? 128 : 256; }

hipError_t launch_cross_entropy(const CeArgs& a, int dtype, bool backward, hipStream_t stream);

}  // namespace arcs
