// C ABI of libarcs (declared in include/arcs.h): argument validation, launch
// configuration and nothing else.  No allocation, no synchronisation, no
// host reads of device memory: every call only enqueues kernels on the
// caller's stream (Arc PR #217, "What this does" and "Layering": the
// sampling step must not put a host round trip between decode steps).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <initializer_list>

#include "arcs.h"
#include "cross_entropy.hpp"
#include "launch.hpp"
#include "linear.hpp"

// Device scratch of arcs_sample_noalloc: one copy per GPU, held until the
// process ends, at its own address on each device.  Host code never uses the
// symbol itself (on the host it is only a stand-in): the address comes from
// hipGetSymbolAddress with that device current, cached per device.
static __device__ __align__(256) unsigned char scratch[ARCS_NOALLOC_SCRATCH_BYTES];
static_assert(arcs::split_max_workspace() <= ARCS_NOALLOC_SCRATCH_BYTES, "the scratch holds every split workspace");

namespace {

constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

// The current device's scratch address (looked up on the first call there).
// Two threads racing on a first call store the same address.
int noalloc_scratch(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return ARCS_ERR_LAUNCH;
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    void* q = nullptr;
    if (hipGetSymbolAddress(&q, HIP_SYMBOL(scratch)) != hipSuccess || q == nullptr) return ARCS_ERR_LAUNCH;
    g_scratch_ptr[dev].store(q, std::memory_order_release);
    p = q;
  }
  *out = p;
  return ARCS_OK;
}

constexpr int64_t kMaxDim = 2147483647;
// arcs_w4_logits: what the launch grids and 32-bit offsets in a tile hold
constexpr int64_t kMaxW4Stride = int64_t(1) << 21, kMaxW4Batch = int64_t(1) << 19, kMaxW4Vocab = int64_t(1) << 28;

int check_common(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                 const void* out_ids) {
  if (logits == nullptr || out_ids == nullptr) return ARCS_ERR_NULL_POINTER;
  if (dtype != ARCS_DTYPE_BF16 && dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (B <= 0 || B > kMaxDim) return ARCS_ERR_BAD_BATCH;
  if (V <= 0 || V > kMaxDim) return ARCS_ERR_BAD_VOCAB;
  if (row_stride < V) return ARCS_ERR_BAD_STRIDE;
  const int64_t es = dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  if (((uintptr_t)logits) % (uintptr_t)es != 0) return ARCS_ERR_MISALIGNED;
  return ARCS_OK;
}

// Rows start on a 16-byte boundary: the vector-load path applies.
bool rows_16b_aligned(const void* logits, int dtype, int64_t row_stride) {
  const int64_t es = dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  return ((uintptr_t)logits % 16u) == 0 && ((row_stride * es) % 16) == 0;
}

// Fixed-point fraction bits: V * 2^F < 2^63 so any sum of weights in [0, 1]
// fits an unsigned 64-bit integer.
int fixed_bits(int64_t V) {
  int lg = 0;
  while ((int64_t(1) << (lg + 1)) <= V) ++lg;  // floor(log2 V)
  int F = 62 - lg;
  return F > 62 ? 62 : F;
}

int sample_impl(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                uint64_t seed, uint64_t step, const uint64_t* key, int32_t* out_ids, int32_t* out_status,
                void* workspace, size_t workspace_bytes, const double* uniforms, float* out_probs,
                arcs_row_stats* out_stats, void* stream, const arcs_dry_params* dry = nullptr,
                const int32_t* breakers = nullptr, int n_breakers = 0) {
  int st = check_common(logits, dtype, B, V, row_stride, out_ids);
  if (st != ARCS_OK) return st;
  if (n_breakers < 0 || n_breakers > ARCS_DRY_MAX_BREAKERS || (n_breakers > 0 && breakers == nullptr))
    return ARCS_ERR_BAD_DRY;
  if (((uintptr_t)dry) % 4u != 0 || ((uintptr_t)breakers) % 4u != 0) return ARCS_ERR_MISALIGNED;
  if (params == nullptr) return ARCS_ERR_NULL_POINTER;
  if ((hist_ids == nullptr) != (hist_offsets == nullptr)) return ARCS_ERR_BAD_HISTORY;
  const size_t ws_need = arcs_sample_workspace_bytes(B, V, dtype);
  if (workspace_bytes < ws_need) return ARCS_ERR_WORKSPACE_TOO_SMALL;
  if (ws_need > 0 && workspace == nullptr) return ARCS_ERR_NULL_POINTER;
  if (ws_need > 0 && ((uintptr_t)workspace & 15u) != 0) return ARCS_ERR_MISALIGNED;
  arcs::SampleArgs a;
  a.logits = logits;
  a.V = V;
  a.stride = row_stride;
  a.params = params;
  a.hist_ids = hist_ids;
  a.hist_offsets = hist_offsets;
  a.seed = seed;
  a.step = step;
  a.key = key;
  a.out_ids = out_ids;
  a.out_status = out_status;
  a.uniforms = uniforms;
  a.out_probs = out_probs;
  a.stats = out_stats;
  a.F = fixed_bits(V);
  a.scale = (float)((double)(int64_t(1) << a.F));
  a.pen_tables = (hist_ids != nullptr && V <= ARCS_MAX_PENALTY_VOCAB) ? 1 : 0;
  a.bitmap_words = a.pen_tables ? (uint32_t)((V + 31) / 32) : 0u;
  a.deferred_only = 0;
  a.dry = dry;
  a.dry_breakers = breakers;
  a.n_breakers = n_breakers;
  // penalised launches: a workspace of arcs_long_history_workspace_bytes()
  // takes the rows whose penalties the LDS tables cannot hold
  const size_t long_need = arcs_long_history_workspace_bytes(B, V);
  a.long_ws = (hist_ids != nullptr && workspace != nullptr && workspace_bytes >= long_need &&
               ((uintptr_t)workspace & 15u) == 0)
                  ? (float*)workspace
                  : nullptr;
  const bool vec = rows_16b_aligned(logits, dtype, row_stride);
  // small batches: greedy rows and rows without filters are read by many
  // workgroups per row (not with debug outputs, which read the row whole)
  const bool split = ws_need > 0 && arcs::split_shape(B, V, dtype) && vec && !a.pen_tables &&
                     out_stats == nullptr && out_probs == nullptr;
  a.split_parts = split ? (arcs::SplitPart*)workspace : nullptr;
  a.split_P = split ? arcs::split_slices(B) : 0;
  hipError_t e = arcs::launch_sample(a, dtype, B, vec, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

bool misaligned(const void* p, uintptr_t to) { return ((uintptr_t)p) % to != 0; }

// Arguments the two directions of the linear cross entropy share.
int check_cross_entropy(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride,
                        int dtype, int64_t N, int64_t V, int64_t D, const int32_t* targets,
                        const float* temperature, const void* workspace, size_t workspace_bytes, bool backward,
                        arcs::CePlan* plan) {
  if (hidden == nullptr || weight == nullptr || targets == nullptr) return ARCS_ERR_NULL_POINTER;
  if (dtype != ARCS_DTYPE_BF16 && dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (N <= 0 || N > kMaxDim) return ARCS_ERR_BAD_BATCH;
  if (V <= 0 || V > kMaxDim) return ARCS_ERR_BAD_VOCAB;
  if (D <= 0 || D > ARCS_MAX_HIDDEN) return ARCS_ERR_BAD_HIDDEN;
  if (hidden_stride < D || weight_stride < D) return ARCS_ERR_BAD_STRIDE;
  const uintptr_t es = dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  if (misaligned(hidden, es) || misaligned(weight, es) || misaligned(targets, 4) || misaligned(temperature, 4))
    return ARCS_ERR_MISALIGNED;
  *plan = arcs::cross_entropy_plan(N, V, D, dtype, backward);
  if (!plan->fits) return ARCS_ERR_BAD_BATCH;
  if (workspace_bytes < plan->total) return ARCS_ERR_WORKSPACE_TOO_SMALL;
  if (workspace == nullptr) return ARCS_ERR_NULL_POINTER;
  if (misaligned(workspace, 256)) return ARCS_ERR_MISALIGNED;
  return ARCS_OK;
}

arcs::CeArgs cross_entropy_args(const void* hidden, int64_t hidden_stride, const void* weight,
                                int64_t weight_stride, int64_t N, int64_t V, int64_t D, const int32_t* targets,
                                int32_t ignore_index, const float* temperature, const arcs::CePlan& p,
                                void* workspace) {
  arcs::CeArgs a = {};
  a.hidden = hidden;
  a.hidden_stride = hidden_stride;
  a.weight = weight;
  a.weight_stride = weight_stride;
  a.N = N;
  a.V = V;
  a.D = D;
  a.targets = targets;
  a.ignore_index = ignore_index;
  a.temperature = temperature;
  char* w = (char*)workspace;
  a.head = (arcs::CeHeader*)w;
  a.rows = (arcs::CeRow*)(w + p.rows);
  a.place = (int32_t*)(w + p.place);
  a.partial = (float2*)(w + p.partial);
  a.slices = p.slices;
  a.dtarget = (float*)(w + p.dtarget);
  a.ds = w + p.ds;
  a.ds_ld = p.piece;
  a.slab = (float*)(w + p.slab);
  a.splits = p.splits;
  a.workers = p.workers;
  a.hc = w + p.hc;
  return a;
}

uintptr_t element_size(int dtype) { return dtype == ARCS_DTYPE_BF16 ? 2 : 4; }

// Sizes the linear layer takes: tile counts fit an int, and a tile's rows of dz 31 bits.
int linear_sizes(int64_t N, int64_t V, int64_t D, int dtype, bool backward) {
  if (dtype != ARCS_DTYPE_BF16 && dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (N <= 0 || N > int64_t(1) << 22) return ARCS_ERR_BAD_BATCH;
  if (V <= 0 || V > (backward ? (int64_t(1) << 21) - 8 : int64_t(1) << 24)) return ARCS_ERR_BAD_VOCAB;
  if (N * V > int64_t(1) << 40) return ARCS_ERR_BAD_BATCH;
  if (D <= 0 || D > ARCS_MAX_HIDDEN) return ARCS_ERR_BAD_HIDDEN;
  return ARCS_OK;
}

// Arguments the two directions of the linear layer share.
int check_linear(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride, int dtype,
                 int64_t N, int64_t V, int64_t D, int activation, float softcap, bool backward,
                 const void* workspace, size_t workspace_bytes, bool* aligned) {
  if (hidden == nullptr || weight == nullptr) return ARCS_ERR_NULL_POINTER;
  int st = linear_sizes(N, V, D, dtype, backward);
  if (st != ARCS_OK) return st;
  if (hidden_stride < D || weight_stride < D) return ARCS_ERR_BAD_STRIDE;
  if (activation < ARCS_ACT_NONE || activation > ARCS_ACT_SOFTCAP ||
      (activation == ARCS_ACT_SOFTCAP && !(softcap >= 0x1p-100f && softcap <= 0x1p100f)))
    return ARCS_ERR_BAD_ACTIVATION;
  if (misaligned(hidden, element_size(dtype)) || misaligned(weight, element_size(dtype))) return ARCS_ERR_MISALIGNED;
  *aligned = arcs::linear_rows_aligned(hidden, hidden_stride, D, dtype) &&
             arcs::linear_rows_aligned(weight, weight_stride, D, dtype);
  const size_t need = arcs::linear_plan(N, V, D, dtype, *aligned, backward).total;
  if (workspace_bytes < need) return ARCS_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && workspace == nullptr) return ARCS_ERR_NULL_POINTER;
  if (need > 0 && misaligned(workspace, 256)) return ARCS_ERR_MISALIGNED;
  return ARCS_OK;
}

// A row-major array as its bytes lie.
struct Rows {
  const void* p;
  int64_t stride, rows, columns, size;  // stride and columns in elements of `size` bytes
};

// Whether any two rows of two arrays share bytes.  Rows of equal strides may lie between
// each other's.
bool overlap(const Rows& x, const Rows& y) {
  if (x.p == nullptr || y.p == nullptr) return false;
  const __int128 x0 = (intptr_t)x.p, y0 = (intptr_t)y.p, xs = (__int128)x.stride * x.size, ys = (__int128)y.stride * y.size;
  const __int128 xl = (__int128)x.columns * x.size, yl = (__int128)y.columns * y.size;
  if (x0 + xs * (x.rows - 1) + xl <= y0 || y0 + ys * (y.rows - 1) + yl <= x0) return false;
  if (xs != ys || x.rows == 1 || y.rows == 1) return true;
  const __int128 d = ((y0 - x0) % xs + xs) % xs;
  return d < xl || xs - d < yl;
}
bool overlaps_any(const Rows& x, std::initializer_list<Rows> others) {
  for (const Rows& y : others)
    if (overlap(x, y)) return true;
  return false;
}

// A list of gradients, and how many pieces it has.
int check_tensors(const arcs_tensor* tensors, int64_t n, int64_t* pieces) {
  if (n < 0) return ARCS_ERR_BAD_BATCH;
  if (n > 0 && tensors == nullptr) return ARCS_ERR_NULL_POINTER;
  int64_t total = 0;
  *pieces = 0;
  for (int64_t i = 0; i < n; ++i) {
    const arcs_tensor& t = tensors[i];
    if ((t.dtype != ARCS_DTYPE_BF16 && t.dtype != ARCS_DTYPE_F32) ||
        (t.out_dtype != ARCS_DTYPE_BF16 && t.out_dtype != ARCS_DTYPE_F32))
      return ARCS_ERR_BAD_DTYPE;
    if (t.count < 0 || t.count > (int64_t(1) << 40) - total) return ARCS_ERR_BAD_PLAN;
    if (t.count > 0 && t.data == nullptr) return ARCS_ERR_NULL_POINTER;
    if (misaligned(t.data, element_size(t.dtype)) || misaligned(t.out, element_size(t.out_dtype)))
      return ARCS_ERR_MISALIGNED;
    if (t.count > 0 && t.out == t.data && t.out_dtype != t.dtype) return ARCS_ERR_OVERLAP;
    total += t.count;
    *pieces += (t.count + arcs::kNormPiece - 1) / arcs::kNormPiece;
  }
  return ARCS_OK;
}

size_t norm_workspace(size_t plan_bytes) {
  const int groups = arcs::norm_groups((int64_t)(plan_bytes / sizeof(arcs::NormPiece)));
  return groups > 0 ? ((size_t)groups * 8 + 255) / 256 * 256 : 0;
}

int norm_impl(const void* plan, size_t plan_bytes, double max_norm, float* out_norm, void* workspace,
              size_t workspace_bytes, bool clip, void* stream) {
  if (out_norm == nullptr || (plan == nullptr && plan_bytes > 0)) return ARCS_ERR_NULL_POINTER;
  if (plan_bytes % sizeof(arcs::NormPiece) != 0) return ARCS_ERR_BAD_PLAN;
  if (misaligned(plan, 8) || misaligned(out_norm, 4)) return ARCS_ERR_MISALIGNED;
  const size_t need = norm_workspace(plan_bytes);
  if (workspace_bytes < need) return ARCS_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && workspace == nullptr) return ARCS_ERR_NULL_POINTER;
  if (need > 0 && misaligned(workspace, 256)) return ARCS_ERR_MISALIGNED;
  arcs::NormArgs a = {};
  a.plan = (const arcs::NormPiece*)plan;
  a.pieces = (int64_t)(plan_bytes / sizeof(arcs::NormPiece));
  a.max_norm = max_norm;
  a.out_norm = out_norm;
  a.sums = (double*)workspace;
  hipError_t e = arcs::launch_norm(a, clip, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int arcs_argmax(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                int32_t* out_ids, void* stream) {
  int st = check_common(logits, dtype, B, V, row_stride, out_ids);
  if (st != ARCS_OK) return st;
  hipError_t e = arcs::launch_argmax(logits, dtype, B, V, row_stride,
                                     rows_16b_aligned(logits, dtype, row_stride), out_ids,
                                     (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_sample(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                uint64_t seed, uint64_t step, int32_t* out_ids, int32_t* out_status,
                void* workspace, size_t workspace_bytes, void* stream) {
  return sample_impl(logits, dtype, B, V, row_stride, params, hist_ids, hist_offsets, seed, step,
                     nullptr, out_ids, out_status, workspace, workspace_bytes, nullptr, nullptr, nullptr,
                     stream);
}

int arcs_sample_dry(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                    const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                    const arcs_dry_params* dry, const int32_t* breakers, int n_breakers, uint64_t seed,
                    uint64_t step, int32_t* out_ids, int32_t* out_status, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return sample_impl(logits, dtype, B, V, row_stride, params, hist_ids, hist_offsets, seed, step, nullptr,
                     out_ids, out_status, workspace, workspace_bytes, nullptr, nullptr, nullptr, stream, dry,
                     breakers, n_breakers);
}

int arcs_sample_noalloc(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                        const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                        uint64_t seed, uint64_t step, int32_t* out_ids, int32_t* out_status, void* stream) {
  int st = check_common(logits, dtype, B, V, row_stride, out_ids);
  if (st != ARCS_OK) return st;
  const size_t need = arcs_sample_workspace_bytes(B, V, dtype);
  if (need > (size_t)ARCS_NOALLOC_SCRATCH_BYTES) return ARCS_ERR_SCRATCH_TOO_SMALL;
  void* ws = nullptr;
  if (need > 0) {
    st = noalloc_scratch(&ws);
    if (st != ARCS_OK) return st;
  }
  return sample_impl(logits, dtype, B, V, row_stride, params, hist_ids, hist_offsets, seed, step, nullptr,
                     out_ids, out_status, ws, need, nullptr, nullptr, nullptr, stream);
}

int arcs_sample_keyed(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const arcs_row_params* params, const int32_t* hist_ids,
                      const int64_t* hist_offsets, uint64_t* key, int advance, int32_t* out_ids,
                      int32_t* out_status, void* workspace, size_t workspace_bytes, void* stream) {
  if (key == nullptr) return ARCS_ERR_NULL_POINTER;
  if (((uintptr_t)key) % 8u != 0) return ARCS_ERR_MISALIGNED;
  int st = sample_impl(logits, dtype, B, V, row_stride, params, hist_ids, hist_offsets, 0, 0, key,
                       out_ids, out_status, workspace, workspace_bytes, nullptr, nullptr, nullptr, stream);
  if (st != ARCS_OK || !advance) return st;
  return arcs::launch_advance_step(key, (hipStream_t)stream) == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_sample_debug(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const arcs_row_params* params, const int32_t* hist_ids,
                      const int64_t* hist_offsets, uint64_t seed, uint64_t step,
                      int32_t* out_ids, int32_t* out_status, void* workspace,
                      size_t workspace_bytes, const double* uniforms, float* out_probs,
                      arcs_row_stats* out_stats, void* stream) {
  return sample_impl(logits, dtype, B, V, row_stride, params, hist_ids, hist_offsets, seed, step,
                     nullptr, out_ids, out_status, workspace, workspace_bytes, uniforms, out_probs,
                     out_stats, stream);
}

int arcs_sample_hybrid_nucleus(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                               const float* temperature, const float* top_p, int budget, uint64_t seed,
                               uint64_t step, int32_t* out_ids, int32_t* out_kept, int32_t* out_status,
                               void* stream) {
  int st = check_common(logits, dtype, B, V, row_stride, out_ids);
  if (st != ARCS_OK) return st;
  if (temperature == nullptr || top_p == nullptr) return ARCS_ERR_NULL_POINTER;
  if (dtype != ARCS_DTYPE_BF16) return ARCS_ERR_BAD_DTYPE;
  if (V % 8 != 0 || V > 131072) return ARCS_ERR_BAD_VOCAB;
  if (!rows_16b_aligned(logits, dtype, row_stride)) return ARCS_ERR_MISALIGNED;
  if (((uintptr_t)temperature) % 4u != 0 || ((uintptr_t)top_p) % 4u != 0) return ARCS_ERR_MISALIGNED;
  if (budget < 0 || budget > 4096) return ARCS_ERR_BAD_BUDGET;
  arcs::HybridArgs a;
  a.logits = logits;
  a.V = V;
  a.stride = row_stride;
  a.temperature = temperature;
  a.top_p = top_p;
  a.budget = budget;
  a.seed = seed;
  a.step = step;
  a.out_ids = out_ids;
  a.out_kept = out_kept;
  a.out_status = out_status;
  return arcs::launch_hybrid_nucleus(a, B, (hipStream_t)stream) == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_top_logprobs(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const float* temperature, int n, int32_t* out_ids, float* out_logprobs,
                      int32_t* out_status, void* stream) {
  int st = check_common(logits, dtype, B, V, row_stride, out_ids);
  if (st != ARCS_OK) return st;
  if (out_logprobs == nullptr) return ARCS_ERR_NULL_POINTER;
  if (n < 1 || n > ARCS_MAX_TOP_LOGPROBS) return ARCS_ERR_BAD_TOP_N;
  if (V > ARCS_TOP_LOGPROBS_MAX_VOCAB) return ARCS_ERR_BAD_VOCAB;
  if (((uintptr_t)temperature) % 4u != 0) return ARCS_ERR_MISALIGNED;
  arcs::LogprobArgs a;
  a.logits = logits;
  a.V = V;
  a.stride = row_stride;
  a.temperature = temperature;
  a.n = n;
  a.out_ids = out_ids;
  a.out_logprobs = out_logprobs;
  a.out_status = out_status;
  hipError_t e = arcs::launch_top_logprobs(a, dtype, B, rows_16b_aligned(logits, dtype, row_stride),
                                           (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_w4_logits(const void* hidden, int64_t B, int64_t D, int64_t hidden_stride, const uint8_t* qweight,
                   int64_t V, int64_t qweight_stride, const void* scales, int scale_dtype,
                   int64_t scale_stride, const uint8_t* zeros, int64_t zero_stride, int group_size,
                   void* logits, int logits_dtype, int64_t row_stride, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (hidden == nullptr || qweight == nullptr || scales == nullptr || logits == nullptr) return ARCS_ERR_NULL_POINTER;
  if ((scale_dtype != ARCS_DTYPE_BF16 && scale_dtype != ARCS_DTYPE_F32) ||
      (logits_dtype != ARCS_DTYPE_BF16 && logits_dtype != ARCS_DTYPE_F32))
    return ARCS_ERR_BAD_DTYPE;
  if (B <= 0 || B > kMaxW4Batch) return ARCS_ERR_BAD_BATCH;
  if (V <= 0 || V > kMaxW4Vocab) return ARCS_ERR_BAD_VOCAB;
  if (B * V > int64_t(1) << 36) return ARCS_ERR_BAD_BATCH;
  if (D <= 0 || D > ARCS_MAX_HIDDEN) return ARCS_ERR_BAD_HIDDEN;
  if ((group_size != 32 && group_size != 64 && group_size != 128) || D % group_size != 0) return ARCS_ERR_BAD_GROUP;
  const int64_t groups = D / group_size;
  if (hidden_stride < D || qweight_stride < D / 2 || scale_stride < groups || row_stride < V ||
      (zeros != nullptr && zero_stride < groups))
    return ARCS_ERR_BAD_STRIDE;
  // a tile's rows are addressed with 32 bits
  if (qweight_stride > kMaxW4Stride || scale_stride > kMaxW4Stride || (zeros != nullptr && zero_stride > kMaxW4Stride))
    return ARCS_ERR_BAD_STRIDE;
  if (misaligned(hidden, 16) || hidden_stride % 8 != 0 || misaligned(qweight, 16) || qweight_stride % 16 != 0 ||
      misaligned(scales, scale_dtype == ARCS_DTYPE_BF16 ? 2 : 4) ||
      misaligned(logits, logits_dtype == ARCS_DTYPE_BF16 ? 2 : 4))
    return ARCS_ERR_MISALIGNED;
  const size_t need = arcs::w4_workspace_bytes(B, D);
  if (workspace_bytes < need) return ARCS_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && workspace == nullptr) return ARCS_ERR_NULL_POINTER;
  if (need > 0 && misaligned(workspace, 256)) return ARCS_ERR_MISALIGNED;
  arcs::W4Args a = {};
  a.hidden = (const uint16_t*)hidden;
  a.B = B;
  a.D = D;
  a.hidden_stride = hidden_stride;
  a.qweight = qweight;
  a.V = V;
  a.qweight_stride = qweight_stride;
  a.scales = scales;
  a.scale_stride = scale_stride;
  a.zeros = zeros;
  a.zero_stride = zero_stride;
  a.logits = logits;
  a.row_stride = row_stride;
  hipError_t e = arcs::launch_w4_logits(a, scale_dtype, logits_dtype, group_size, workspace, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

size_t arcs_w4_logits_workspace_bytes(int64_t B, int64_t D, int group_size) {
  if (B <= 0 || B > kMaxW4Batch || D <= 0 || D > ARCS_MAX_HIDDEN ||
      (group_size != 32 && group_size != 64 && group_size != 128))
    return 0;
  return arcs::w4_workspace_bytes(B, D);
}

int arcs_linear_cross_entropy(const void* hidden, int64_t hidden_stride, const void* weight,
                              int64_t weight_stride, int dtype, int64_t N, int64_t V, int64_t D,
                              const int32_t* targets, int32_t ignore_index, const float* temperature,
                              float* out_loss, float* out_lse, int32_t* out_status, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (out_loss == nullptr || out_lse == nullptr) return ARCS_ERR_NULL_POINTER;
  arcs::CePlan plan;
  int st = check_cross_entropy(hidden, hidden_stride, weight, weight_stride, dtype, N, V, D, targets, temperature,
                               workspace, workspace_bytes, false, &plan);
  if (st != ARCS_OK) return st;
  if (misaligned(out_loss, 4) || misaligned(out_lse, 4) || misaligned(out_status, 4)) return ARCS_ERR_MISALIGNED;
  arcs::CeArgs a = cross_entropy_args(hidden, hidden_stride, weight, weight_stride, N, V, D, targets, ignore_index,
                                      temperature, plan, workspace);
  a.out_loss = out_loss;
  a.out_lse = out_lse;
  a.out_status = out_status;
  hipError_t e = arcs::launch_cross_entropy(a, dtype, false, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_linear_cross_entropy_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                       int64_t weight_stride, int dtype, int64_t N, int64_t V, int64_t D,
                                       const int32_t* targets, int32_t ignore_index, const float* temperature,
                                       const float* lse, const float* grad_loss, void* out_dhidden,
                                       void* out_dweight, void* workspace, size_t workspace_bytes, void* stream) {
  if (lse == nullptr || grad_loss == nullptr || (out_dhidden == nullptr && out_dweight == nullptr))
    return ARCS_ERR_NULL_POINTER;
  arcs::CePlan plan;
  int st = check_cross_entropy(hidden, hidden_stride, weight, weight_stride, dtype, N, V, D, targets, temperature,
                               workspace, workspace_bytes, true, &plan);
  if (st != ARCS_OK) return st;
  const uintptr_t es = dtype == ARCS_DTYPE_BF16 ? 2 : 4;
  if (misaligned(lse, 4) || misaligned(grad_loss, 4) || misaligned(out_dhidden, es) || misaligned(out_dweight, es))
    return ARCS_ERR_MISALIGNED;
  arcs::CeArgs a = cross_entropy_args(hidden, hidden_stride, weight, weight_stride, N, V, D, targets, ignore_index,
                                      temperature, plan, workspace);
  a.lse = lse;
  a.grad_loss = grad_loss;
  a.out_dhidden = out_dhidden;
  a.out_dweight = out_dweight;
  hipError_t e = arcs::launch_cross_entropy(a, dtype, true, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

size_t arcs_linear_cross_entropy_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int backward) {
  if (N <= 0 || N > kMaxDim || V <= 0 || V > kMaxDim || D <= 0 || D > ARCS_MAX_HIDDEN ||
      (dtype != ARCS_DTYPE_BF16 && dtype != ARCS_DTYPE_F32))
    return 0;
  const arcs::CePlan p = arcs::cross_entropy_plan(N, V, D, dtype, backward != 0);
  return p.fits ? p.total : 0;
}

int arcs_linear(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride, int dtype,
                int64_t N, int64_t V, int64_t D, const void* bias, int activation, float softcap,
                const void* residual, int64_t residual_stride, void* out, int out_dtype, int64_t out_stride,
                void* out_pre, void* workspace, size_t workspace_bytes, void* stream) {
  if (out == nullptr) return ARCS_ERR_NULL_POINTER;
  bool aligned;
  int st = check_linear(hidden, hidden_stride, weight, weight_stride, dtype, N, V, D, activation, softcap, false,
                        workspace, workspace_bytes, &aligned);
  if (st != ARCS_OK) return st;
  if (out_dtype != ARCS_DTYPE_BF16 && out_dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (out_stride < V || (residual != nullptr && residual_stride < V)) return ARCS_ERR_BAD_STRIDE;
  const uintptr_t es = element_size(dtype);
  if (misaligned(bias, es) || misaligned(residual, es) || misaligned(out_pre, es) ||
      misaligned(out, element_size(out_dtype)))
    return ARCS_ERR_MISALIGNED;
  const int64_t size = (int64_t)es;
  const Rows h = {hidden, hidden_stride, N, D, size}, w = {weight, weight_stride, V, D, size}, b = {bias, V, 1, V, size};
  const Rows r = {residual, residual_stride, N, V, size}, pre = {out_pre, V, N, V, size};
  const Rows y = {out, out_stride, N, V, (int64_t)element_size(out_dtype)};
  const bool in_place = residual == out && out_dtype == dtype && (N == 1 || residual_stride == out_stride);
  if (overlaps_any(y, {h, w, b, pre}) || (!in_place && overlap(y, r)) || overlaps_any(pre, {h, w, b, r}))
    return ARCS_ERR_OVERLAP;
  arcs::LinearArgs a = {};
  a.hidden = hidden;
  a.hidden_stride = hidden_stride;
  a.weight = weight;
  a.weight_stride = weight_stride;
  a.N = N;
  a.V = V;
  a.D = D;
  a.act = activation;
  a.cap = softcap;
  a.inv_cap = activation == ARCS_ACT_SOFTCAP ? 1.0f / softcap : 0.0f;
  a.bias = bias;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.out_bf16 = out_dtype == ARCS_DTYPE_BF16;
  a.out_pre = out_pre;
  a.workspace = (char*)workspace;
  hipError_t e = arcs::launch_linear(a, dtype, aligned, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

int arcs_linear_backward(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride,
                         int dtype, int64_t N, int64_t V, int64_t D, int activation, float softcap,
                         const void* pre, const void* grad_out, int grad_dtype, int64_t grad_stride,
                         void* out_dhidden, void* out_dweight, void* out_dbias, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (grad_out == nullptr || (out_dhidden == nullptr && out_dweight == nullptr && out_dbias == nullptr))
    return ARCS_ERR_NULL_POINTER;
  bool aligned;
  int st = check_linear(hidden, hidden_stride, weight, weight_stride, dtype, N, V, D, activation, softcap, true,
                        workspace, workspace_bytes, &aligned);
  if (st != ARCS_OK) return st;
  if (activation != ARCS_ACT_NONE && pre == nullptr) return ARCS_ERR_NULL_POINTER;
  if (grad_dtype != ARCS_DTYPE_BF16 && grad_dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (grad_stride < V) return ARCS_ERR_BAD_STRIDE;
  const uintptr_t es = element_size(dtype);
  if (misaligned(pre, es) || misaligned(grad_out, element_size(grad_dtype)) || misaligned(out_dhidden, es) ||
      misaligned(out_dweight, es) || misaligned(out_dbias, es))
    return ARCS_ERR_MISALIGNED;
  const int64_t size = (int64_t)es;
  const Rows h = {hidden, hidden_stride, N, D, size}, w = {weight, weight_stride, V, D, size}, z = {pre, V, N, V, size};
  const Rows g = {grad_out, grad_stride, N, V, (int64_t)element_size(grad_dtype)};
  const Rows dh = {out_dhidden, D, N, D, size}, dw = {out_dweight, D, V, D, size}, db = {out_dbias, V, 1, V, size};
  if (overlaps_any(dh, {h, w, z, g, dw, db}) || overlaps_any(dw, {h, w, z, g, db}) || overlaps_any(db, {h, w, z, g}))
    return ARCS_ERR_OVERLAP;
  arcs::LinearArgs a = {};
  a.hidden = hidden;
  a.hidden_stride = hidden_stride;
  a.weight = weight;
  a.weight_stride = weight_stride;
  a.N = N;
  a.V = V;
  a.D = D;
  a.act = activation;
  a.cap = softcap;
  a.inv_cap = activation == ARCS_ACT_SOFTCAP ? 1.0f / softcap : 0.0f;
  a.pre = pre;
  a.grad = grad_out;
  a.grad_stride = grad_stride;
  a.grad_bf16 = grad_dtype == ARCS_DTYPE_BF16;
  a.out_dhidden = out_dhidden;
  a.out_dweight = out_dweight;
  a.out_dbias = out_dbias;
  a.workspace = (char*)workspace;
  hipError_t e = arcs::launch_linear_backward(a, dtype, aligned, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

size_t arcs_linear_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int rows_aligned) {
  return linear_sizes(N, V, D, dtype, false) == ARCS_OK ? arcs::linear_plan(N, V, D, dtype, rows_aligned != 0, false).total : 0;
}

size_t arcs_linear_backward_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int rows_aligned) {
  return linear_sizes(N, V, D, dtype, true) == ARCS_OK ? arcs::linear_plan(N, V, D, dtype, rows_aligned != 0, true).total : 0;
}

int arcs_adjust_logits(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                       const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                       const int32_t* bias_ids, const float* bias_values, const int64_t* bias_offsets,
                       const uint32_t* mask, int64_t masks, int64_t mask_stride, const int32_t* mask_rows,
                       void* out, int out_dtype, int64_t out_stride, int32_t* out_status, void* stream) {
  int st = check_common(logits, dtype, B, V, row_stride, out);
  if (st != ARCS_OK) return st;
  if (out_dtype != ARCS_DTYPE_BF16 && out_dtype != ARCS_DTYPE_F32) return ARCS_ERR_BAD_DTYPE;
  if (!arcs::adjust_fits(B, V)) return ARCS_ERR_BAD_BATCH;
  if (out_stride < V) return ARCS_ERR_BAD_STRIDE;
  if ((hist_ids == nullptr) != (hist_offsets == nullptr)) return ARCS_ERR_BAD_HISTORY;
  if (hist_ids != nullptr && params == nullptr) return ARCS_ERR_NULL_POINTER;
  if ((bias_ids == nullptr) != (bias_values == nullptr) || (bias_ids == nullptr) != (bias_offsets == nullptr))
    return ARCS_ERR_BAD_BIAS;
  if (mask == nullptr ? mask_rows != nullptr : masks < (mask_rows != nullptr ? 1 : B)) return ARCS_ERR_BAD_MASK;
  if (mask != nullptr && mask_stride < (V + 31) / 32) return ARCS_ERR_BAD_STRIDE;
  if (misaligned(params, 4) || misaligned(hist_ids, 4) || misaligned(hist_offsets, 8) || misaligned(bias_ids, 4) ||
      misaligned(bias_values, 4) || misaligned(bias_offsets, 8) || misaligned(mask, 4) || misaligned(mask_rows, 4) ||
      misaligned(out, element_size(out_dtype)) || misaligned(out_status, 4))
    return ARCS_ERR_MISALIGNED;
  const bool in_place = out == logits && out_dtype == dtype && (B == 1 || out_stride == row_stride);
  if (!in_place && overlap({logits, row_stride, B, V, (int64_t)element_size(dtype)},
                           {out, out_stride, B, V, (int64_t)element_size(out_dtype)}))
    return ARCS_ERR_OVERLAP;
  arcs::AdjustArgs a = {};
  a.logits = logits;
  a.V = V;
  a.stride = row_stride;
  a.params = params;
  a.hist_ids = hist_ids;
  a.hist_offsets = hist_offsets;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.bias_offsets = bias_offsets;
  a.mask = mask;
  a.masks = masks;
  a.mask_stride = mask_stride;
  a.mask_rows = mask_rows;
  a.out = out;
  a.out_stride = out_stride;
  a.in_place = in_place;
  a.out_status = out_status;
  hipError_t e = arcs::launch_adjust(a, dtype, out_dtype, B, (hipStream_t)stream);
  return e == hipSuccess ? ARCS_OK : ARCS_ERR_LAUNCH;
}

size_t arcs_gradient_plan_bytes(const arcs_tensor* tensors, int64_t n) {
  int64_t pieces;
  return check_tensors(tensors, n, &pieces) == ARCS_OK ? (size_t)pieces * sizeof(arcs::NormPiece) : 0;
}

int arcs_gradient_plan(const arcs_tensor* tensors, int64_t n, void* plan, size_t plan_bytes) {
  int64_t pieces;
  int st = check_tensors(tensors, n, &pieces);
  if (st != ARCS_OK) return st;
  if (plan_bytes != (size_t)pieces * sizeof(arcs::NormPiece)) return ARCS_ERR_BAD_PLAN;
  if (pieces > 0 && plan == nullptr) return ARCS_ERR_NULL_POINTER;
  if (misaligned(plan, 8)) return ARCS_ERR_MISALIGNED;
  arcs::NormPiece* to = (arcs::NormPiece*)plan;
  for (int64_t i = 0; i < n; ++i) {
    const arcs_tensor& t = tensors[i];
    for (int64_t at = 0; at < t.count; at += arcs::kNormPiece) {
      arcs::NormPiece p = {};
      p.from = (const char*)t.data + at * element_size(t.dtype);
      p.to = t.out == nullptr ? nullptr : (char*)t.out + at * element_size(t.out_dtype);
      p.count = (int32_t)(t.count - at < arcs::kNormPiece ? t.count - at : arcs::kNormPiece);
      p.bf16 = t.dtype == ARCS_DTYPE_BF16;
      p.to_bf16 = t.out_dtype == ARCS_DTYPE_BF16;
      *to++ = p;
    }
  }
  return ARCS_OK;
}

int arcs_gradient_norm(const void* plan, size_t plan_bytes, float* out_norm, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return norm_impl(plan, plan_bytes, 0.0, out_norm, workspace, workspace_bytes, false, stream);
}

int arcs_clip_gradients(const void* plan, size_t plan_bytes, double max_norm, float* out_norm, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0)) return ARCS_ERR_BAD_NORM;
  return norm_impl(plan, plan_bytes, max_norm, out_norm, workspace, workspace_bytes, true, stream);
}

size_t arcs_gradient_workspace_bytes(size_t plan_bytes) { return norm_workspace(plan_bytes); }

size_t arcs_long_history_workspace_bytes(int64_t B, int64_t V) {
  if (B <= 0 || V <= 0) return 0;
  const unsigned __int128 n = (unsigned __int128)B * (unsigned __int128)V * 4u;
  return n > (unsigned __int128)SIZE_MAX ? SIZE_MAX : (size_t)n;
}

size_t arcs_sample_workspace_bytes(int64_t B, int64_t V, int dtype) {
  if (!arcs::split_shape(B, V, dtype)) return 0;
  return (size_t)B * (size_t)arcs::split_slices(B) * sizeof(arcs::SplitPart);
}

const char* arcs_status_string(int code) {
  switch (code) {
    case ARCS_OK: return "ok";
    case ARCS_ERR_NULL_POINTER: return "a required pointer is NULL";
    case ARCS_ERR_BAD_BATCH: return "batch size B must be in [1, 2^31-1]";
    case ARCS_ERR_BAD_VOCAB: return "vocabulary size V must be in [1, 2^31-1]";
    case ARCS_ERR_BAD_STRIDE: return "row_stride must be >= V";
    case ARCS_ERR_BAD_DTYPE: return "dtype must be ARCS_DTYPE_BF16 or ARCS_DTYPE_F32";
    case ARCS_ERR_WORKSPACE_TOO_SMALL: return "workspace smaller than the call's *_workspace_bytes()";
    case ARCS_ERR_BAD_BUDGET: return "budget outside [0, 4096]";
    case ARCS_ERR_BAD_DRY: return "DRY breakers: NULL with n_breakers > 0, or n_breakers outside [0, 64]";
    case ARCS_ERR_SCRATCH_TOO_SMALL:
      return "the shape needs more workspace than arcs_sample_noalloc's scratch (ARCS_NOALLOC_SCRATCH_BYTES)";
    case ARCS_ERR_BAD_HIDDEN: return "hidden size D must be in [1, ARCS_MAX_HIDDEN]";
    case ARCS_ERR_BAD_GROUP: return "group_size must be 32, 64 or 128 and divide D";
    case ARCS_ERR_BAD_ACTIVATION: return "activation must be an arcs_activation, softcap within 2^-100 .. 2^100";
    case ARCS_ERR_BAD_BIAS: return "bias ids, values and offsets must all be NULL or all be set";
    case ARCS_ERR_BAD_MASK: return "mask_rows without a mask, or fewer masks than rows";
    case ARCS_ERR_OVERLAP: return "an output overlaps an input";
    case ARCS_ERR_BAD_NORM: return "max_norm must be >= 0";
    case ARCS_ERR_BAD_PLAN: return "a gradient's count or the plan's size is not valid";
    case ARCS_ERR_LAUNCH: return "kernel launch failed";
    case ARCS_ERR_MISALIGNED: return "an array or its rows are not aligned as the call asks for";
    case ARCS_ERR_BAD_HISTORY: return "hist_ids and hist_offsets must both be NULL or both be set";
    case ARCS_ERR_BAD_TOP_N: return "n must be in [1, ARCS_MAX_TOP_LOGPROBS]";
    case ARCS_ERR_BAD_CAPACITY: return "ring capacity must be >= 1 and capacity * B must fit int64";
    case ARCS_ROW_BAD_TEMPERATURE: return "row: temperature is NaN or negative";
    case ARCS_ROW_BAD_TOP_P: return "row: top_p is NaN or <= 0";
    case ARCS_ROW_BAD_MIN_P: return "row: min_p is NaN or outside [0, 1]";
    case ARCS_ROW_BAD_PENALTY: return "row: a penalty is not finite or repetition < 0";
    case ARCS_ROW_BAD_FLAGS: return "row: flags must be 0";
    case ARCS_ROW_HISTORY_TOO_LONG: return "row: penalties need at most ARCS_MAX_HISTORY distinct history ids";
    case ARCS_ROW_VOCAB_TOO_LARGE: return "row: penalties need V <= ARCS_MAX_PENALTY_VOCAB";
    case ARCS_ROW_BAD_TARGET: return "row: target outside [0, V) and not ignore_index";
    case ARCS_ROW_BAD_MASK: return "row: mask row outside [0, masks) and not -1";
    case ARCS_ROW_NOTHING_ALLOWED: return "row: the mask leaves no token";
    default: return "unknown status";
  }
}

int arcs_version(void) { return 100; }

}  // extern "C"
