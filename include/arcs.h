/*
 * arcs.h -- on-device batched token sampling for AMD Instinct MI355X (gfx950),
 * and the vocabulary head around it: logits from 4-bit weights, linear layers
 * with their gradients, the cross entropy of given tokens with its gradients,
 * adjustments of logits before sampling, and the gradients' norm and clipping.
 *
 * The library turns a [B, V] logits tensor that already lives in GPU memory
 * into one token id per row, without copying the logits to the host.  The
 * pages it follows (the Arc engine's pull requests) price the host path it
 * replaces: Arc PR #222 ("ARC_SAMPLE_ON_DEVICE", section 2) copies the whole
 * [B, 1, vocab] logits tensor to the host every step and samples every row
 * there; Arc PR #217 ("device decode loop", "What this does") keeps the
 * greedy token in an i32[batch] device buffer instead.
 *
 * Conventions shared by every call:
 *  - All array arguments are DEVICE pointers owned by the caller.  The
 *    library allocates nothing, keeps no state between calls, never
 *    synchronises and never reads device memory from the host.  Work is
 *    enqueued on `stream` (a hipStream_t; NULL means the default stream) and
 *    the call returns.
 *  - Logits are row-major: row b starts `b * row_stride` elements after
 *    `logits`, `row_stride >= V`.  dtype ARCS_DTYPE_BF16 (raw bfloat16) or
 *    ARCS_DTYPE_F32.  `logits` must be aligned to its element size; rows
 *    whose start is 16-byte aligned take the vector-load path.
 *  - Host-checkable argument errors are returned as a negative arcs_status
 *    before anything is launched; nothing is written in that case.
 *  - Launch failures are reported as ARCS_ERR_LAUNCH (from hipGetLastError,
 *    without synchronising).
 *  - Calls are reentrant; concurrent calls on different streams are safe.
 */
#ifndef ARCS_H
#define ARCS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum arcs_dtype {
  ARCS_DTYPE_BF16 = 0,
  ARCS_DTYPE_F32 = 1
} arcs_dtype;

typedef enum arcs_status {
  ARCS_OK = 0,
  ARCS_ERR_NULL_POINTER = -1,        /* a required pointer is NULL              */
  ARCS_ERR_BAD_BATCH = -2,           /* B <= 0 or B > 2^31 - 1                  */
  ARCS_ERR_BAD_VOCAB = -3,           /* V <= 0 or V > 2^31 - 1                  */
  ARCS_ERR_BAD_STRIDE = -4,          /* row_stride < V                          */
  ARCS_ERR_BAD_DTYPE = -5,           /* dtype is not an arcs_dtype              */
  ARCS_ERR_WORKSPACE_TOO_SMALL = -6, /* workspace_bytes below the call's *_workspace_bytes() */
  ARCS_ERR_LAUNCH = -7,              /* the HIP runtime rejected a launch       */
  ARCS_ERR_MISALIGNED = -8,          /* an array not aligned as its call asks for */
  ARCS_ERR_BAD_HISTORY = -9,         /* exactly one of hist_ids/hist_offsets is NULL */
  ARCS_ERR_BAD_TOP_N = -10,          /* arcs_top_logprobs: n outside [1, ARCS_MAX_TOP_LOGPROBS] */
  ARCS_ERR_BAD_CAPACITY = -11,       /* arcs_commit_tokens: capacity 0, or capacity * B too large */
  ARCS_ERR_SCRATCH_TOO_SMALL = -12,  /* arcs_sample_noalloc: the shape needs more than its scratch */
  ARCS_ERR_BAD_BUDGET = -13,         /* arcs_sample_hybrid_nucleus: budget outside [0, 4096] */
  ARCS_ERR_BAD_DRY = -14,            /* arcs_sample_dry: breakers NULL or n_breakers outside [0, 64] */
  ARCS_ERR_BAD_HIDDEN = -15,         /* hidden size D outside [1, ARCS_MAX_HIDDEN] */
  ARCS_ERR_BAD_GROUP = -16,          /* arcs_w4_logits: group_size not 32, 64 or 128, or no divisor of D */
  ARCS_ERR_BAD_ACTIVATION = -17,     /* arcs_linear: no arcs_activation, or softcap outside 2^-100 .. 2^100 */
  ARCS_ERR_BAD_BIAS = -18,           /* arcs_adjust_logits: some of the three bias arrays are NULL, not all */
  ARCS_ERR_BAD_MASK = -19,           /* arcs_adjust_logits: mask_rows without a mask, or fewer masks than rows */
  ARCS_ERR_OVERLAP = -20,            /* an output overlaps an input and is not that input in place */
  ARCS_ERR_BAD_NORM = -21,           /* arcs_clip_gradients: max_norm is NaN or negative */
  ARCS_ERR_BAD_PLAN = -22            /* gradients: a tensor's count or the plan's size is not valid */
} arcs_status;

/* Per-row status codes written to out_status[b] (out_ids[b] = -1 when != 0). */
enum {
  ARCS_ROW_OK = 0,
  ARCS_ROW_BAD_TEMPERATURE = 1,      /* temperature NaN or < 0                  */
  ARCS_ROW_BAD_TOP_P = 2,            /* top_p NaN or <= 0                       */
  ARCS_ROW_BAD_MIN_P = 3,            /* min_p NaN, < 0 or > 1                   */
  ARCS_ROW_BAD_PENALTY = 4,          /* non-finite penalty, or repetition < 0   */
  ARCS_ROW_BAD_FLAGS = 5,            /* flags has a bit other than ARCS_ROW_TIES_WIDE */
  ARCS_ROW_HISTORY_TOO_LONG = 6,     /* penalties active, > ARCS_MAX_HISTORY distinct ids,
                                        and no long-history workspace */
  ARCS_ROW_VOCAB_TOO_LARGE = 7,      /* penalties active, V > ARCS_MAX_PENALTY_VOCAB,
                                        and no long-history workspace */
  ARCS_ROW_BAD_TARGET = 8,           /* arcs_linear_cross_entropy: target outside [0, V) and not ignore_index */
  ARCS_ROW_BAD_MASK = 9,             /* arcs_adjust_logits: mask row outside [0, masks) and not -1 */
  ARCS_ROW_NOTHING_ALLOWED = 10      /* arcs_adjust_logits: the mask leaves no token */
};

/* Limits of the penalty tables kept in LDS (per row): distinct history ids
 * in [0, V) (the number of history entries itself is not limited) and V.
 * Beyond them a penalised call needs a long-history workspace (see
 * arcs_long_history_workspace_bytes); without one such rows get the status
 * codes above. */
#define ARCS_MAX_HISTORY 4096
#define ARCS_MAX_PENALTY_VOCAB 262144

/* Codes arcs_commit_tokens latches into its fault word (the first one stays). */
enum {
  ARCS_FAULT_NONE = 0,
  ARCS_FAULT_TOKEN_RANGE = 1,        /* a token outside [0, V) other than -1            */
  ARCS_FAULT_RING_OVERRUN = 2        /* the ring slot still holds a step not drained yet */
};

/* Largest hidden size of arcs_w4_logits, arcs_linear and arcs_linear_cross_entropy. */
#define ARCS_MAX_HIDDEN 65536

/* Limits of arcs_top_logprobs: entries per row, and V. */
#define ARCS_MAX_TOP_LOGPROBS 64
#define ARCS_TOP_LOGPROBS_MAX_VOCAB 262144

/*
 * Per-row sampling parameters, 32 bytes, device array of B records.
 * Filters follow Arc PR #222 section 3(b): the host sampler's sorted list
 * feeds zero-the-rest (top-k), the top-p walk and the min-p scan, all three
 * inert under top_k = -1, top_p = 1, min_p = 0, in which case no cutoff is
 * computed at all.
 *   temperature  0 => greedy (argmax); > 0 => q ~ exp(z'/T)
 *   top_k        <= 0 or >= V => off; 1 => greedy; else keep the k first ids
 *                of the order (value desc, id asc)
 *   top_p        >= 1 => off; else keep the shortest prefix of that order
 *                whose mass reaches top_p of the FULL mass
 *   min_p        0 => off; keep ids with q_v >= min_p * q_max
 *   presence     0 => off; z -= presence for ids in the history
 *   frequency    0 => off; z -= frequency * count for ids in the history
 *   repetition   1 (or 0) => off; z = z > 0 ? z / r : z * r for history ids
 *                (applied first, then frequency, then presence; each an
 *                IEEE binary32 operation without fused multiply-add)
 *   flags        0, or ARCS_ROW_TIES_WIDE: the kept prefix grows to every id
 *                whose value equals that of its last id (the wider tie rule
 *                the pages report for their fallback device selector, Arc PR
 *                #194, squashed commit #130); other bits are a row error
 * The kept set is the shortest of the three prefixes (no renormalisation
 * between filters).
 */
#define ARCS_ROW_TIES_WIDE 1
typedef struct arcs_row_params {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  float presence;
  float frequency;
  float repetition;
  int32_t flags;
} arcs_row_params;

/*
 * Per-row DRY ("don't repeat yourself") penalty, 16 bytes, device array of B
 * records (arcs_sample_dry).  The pages name the penalty and fix one fact:
 * at its disabled default, multiplier 0.0, it touches no logit (Arc PR #222,
 * section 3(a)), so such rows keep the fast path.  Otherwise, over the last
 * min(range, ARCS_DRY_MAX_WINDOW) history ids (range 0: all, up to the
 * window), a token t gets n = the length of the longest tail of that window
 * which also ends right before an earlier occurrence of t (no sequence
 * breaker, and no id outside [0, V), inside the match or as t), and when
 * n >= allowed_length its logit loses multiplier * base^(n - allowed_length),
 * after the presence / frequency / repetition penalties (binary32: the power
 * by repeated multiplication, the product, the subtraction).
 *   multiplier      >= 0, finite (0: off)
 *   base            > 0, finite
 *   allowed_length  >= 1
 *   range           >= 0 (0: the whole window)
 * Invalid records give the row ARCS_ROW_BAD_PENALTY.  DRY needs the row's
 * history: rows without history arrays ignore the record.
 */
typedef struct arcs_dry_params {
  float multiplier;
  float base;
  int32_t allowed_length;
  int32_t range;
} arcs_dry_params;
#define ARCS_DRY_MAX_WINDOW 2048
#define ARCS_DRY_MAX_BREAKERS 64

/* Per-row diagnostics written by arcs_sample_debug only. */
typedef struct arcs_row_stats {
  int32_t id;          /* the sampled token (or -1)                         */
  int32_t argmax;      /* argmax of the penalised logits, lowest index      */
  int32_t kept;        /* size L of the kept set (0 for greedy rows)        */
  int32_t cut_index;   /* last kept id in (value desc, id asc) order        */
  float cut_value;     /* its penalised logit                               */
  float max_logit;     /* max of the penalised logits                       */
  int32_t status;      /* per-row status code                               */
  uint32_t path;       /* ARCS_PATH_* bits: which stages ran                */
  double mass_total;   /* S   = sum of weights exp((z' - max)/T), as used   */
  double mass_kept;    /* S_K = sum over the kept set, as used              */
  double uniform;      /* the uniform u that drove the draw                 */
  uint64_t reserved;
} arcs_row_stats;

enum {
  ARCS_PATH_GREEDY = 1u,      /* argmax only                                   */
  ARCS_PATH_SORT_SKIP = 2u,   /* no filter active: no cutoff computed          */
  ARCS_PATH_CUTOFF = 4u,      /* radix-select cutoff ran                       */
  ARCS_PATH_MINP_FLOOR = 8u,  /* the min-p threshold bounded the kept set      */
  ARCS_PATH_TIE_SPLIT = 16u,  /* the boundary value's ties were split by id    */
  ARCS_PATH_PENALTY = 32u,    /* penalties applied                             */
  ARCS_PATH_SPECIAL = 64u,    /* special values (all -inf, +inf or NaN) seen   */
  ARCS_PATH_RESIDENT = 128u,  /* the row was kept in registers (single HBM read) */
  ARCS_PATH_REREAD = 256u     /* fp32 row: one HBM read, then one re-read from cache */
};

/*
 * arcs_argmax: out_ids[b] = argmax_v logits[b, v], lowest index among equal
 * values (bit-exact with a host argmax; Arc PR #217, "What this does", step 2).
 * NaN counts as -inf and -0 equals +0; a row of all -inf/NaN gives 0.
 *   logits     device, [B, row_stride] of dtype
 *   out_ids    device, int32[B]
 * Returns ARCS_OK or a negative arcs_status.
 */
int arcs_argmax(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                int32_t* out_ids, void* stream);

/*
 * arcs_sample: one token per row (Arc PR #222, sections 2 and 3; penalties
 * per the parameter record above).  Per row b:
 *   z'   = logits widened to float32 (NaN -> -inf), penalties applied to the
 *          ids in hist_ids[hist_offsets[b] .. hist_offsets[b+1]) (ids outside
 *          [0, V) are skipped; duplicates count);
 *   greedy rows (T == 0 or top_k == 1): argmax of z';
 *   else K = the kept prefix, and the token is the first id of K, in id
 *   order, whose running weight exceeds u * S_K, with u the SplitMix64
 *   uniform of counter step * 2^32 + b under `seed` (Arc PR #217, "Default
 *   OFF", names SplitMix64 for the device sampler).
 *   params         device, arcs_row_params[B]
 *   hist_ids       device int32 ids, or NULL (no penalties anywhere)
 *   hist_offsets   device int64[B + 1] CSR offsets into hist_ids, or NULL
 *   seed, step     RNG key, by value
 *   out_ids        device int32[B]; -1 for rows with invalid parameters
 *   out_status     device int32[B] per-row codes, or NULL
 *   workspace      device scratch of workspace_bytes, 16-byte aligned, owned by
 *                  the caller and not read before it is written; may be NULL
 *                  when arcs_sample_workspace_bytes() returns 0.  Batches of
 *                  at most 64 bf16 rows with 8192 <= V <= 131072, V % 8 == 0
 *                  use it: their greedy rows and rows without filters are read
 *                  by P = clamp(512 / B, 8, 128) workgroups per row, which
 *                  leave per-slice partials (16 bytes each) there for the
 *                  row's own workgroup.  Calls that share a workspace must be
 *                  ordered on one stream.
 * Returns ARCS_OK or a negative arcs_status (ARCS_ERR_WORKSPACE_TOO_SMALL
 * when workspace_bytes is below arcs_sample_workspace_bytes(),
 * ARCS_ERR_NULL_POINTER for a NULL workspace the shape needs,
 * ARCS_ERR_MISALIGNED for a workspace not 16-byte aligned).
 */
int arcs_sample(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                const arcs_row_params* params, const int32_t* hist_ids,
                const int64_t* hist_offsets, uint64_t seed, uint64_t step, int32_t* out_ids,
                int32_t* out_status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * arcs_sample_keyed: arcs_sample with the RNG key in device memory, for
 * decode loops captured in a HIP graph.  Arc PR #217 ("device decode loop",
 * "What this does", step 3) keeps the per-step state on the device and moves
 * it on with a device kernel, so that a captured step needs no host work
 * between launches; a key passed by value would instead be frozen into the
 * graph at capture time.
 *   key       device uint64[2] = {seed, step}, 8-byte aligned, read when the
 *             kernels run (the uniform of row b uses counter step * 2^32 + b
 *             under seed, exactly as arcs_sample)
 *   advance   nonzero: a one-thread kernel enqueued after the sampling kernel
 *             on the same stream adds 1 to key[1] (each graph replay then
 *             samples the next step); 0: key is only read
 * Other arguments, errors and outputs as arcs_sample; a NULL or misaligned
 * key is rejected before any launch.  Calls that share one key must be
 * ordered on one stream.
 */
int arcs_sample_keyed(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const arcs_row_params* params, const int32_t* hist_ids,
                      const int64_t* hist_offsets, uint64_t* key, int advance, int32_t* out_ids,
                      int32_t* out_status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * arcs_sample_noalloc: arcs_sample for callers that cannot allocate device
 * memory (code under HIP graph capture, serving loops that forbid
 * allocation).  It takes no workspace: shapes that need one use a device
 * array inside the library, ARCS_NOALLOC_SCRATCH_BYTES per GPU, allocated
 * with the library's code object and held until the process ends.  The call
 * allocates nothing (no hipMalloc, no library routine that allocates); the
 * first call on a device looks up that device's copy of the array.
 * Every call on one GPU shares that GPU's array: calls on one GPU that may
 * overlap (other streams, other host threads) race and must be ordered by
 * the caller.  Shapes needing more than the array (none today: the largest
 * split workspace is 567 * 16 = 9,072 bytes) get ARCS_ERR_SCRATCH_TOO_SMALL before
 * any launch.  Arguments, outputs and other errors as arcs_sample.
 */
#define ARCS_NOALLOC_SCRATCH_BYTES 16384
int arcs_sample_noalloc(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                        const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                        uint64_t seed, uint64_t step, int32_t* out_ids, int32_t* out_status, void* stream);

/*
 * arcs_sample_dry: arcs_sample with a DRY penalty record per row (see
 * arcs_dry_params) and the call's sequence breakers.
 *   dry          device arcs_dry_params[B], or NULL (= arcs_sample)
 *   breakers     device int32 ids that break repeats, n_breakers of them
 *                (0 .. ARCS_DRY_MAX_BREAKERS; NULL when 0)
 * Rows whose DRY record is active (multiplier != 0, with history) run on the
 * general pipeline.  Other arguments, outputs and errors as arcs_sample, plus
 * ARCS_ERR_BAD_DRY.
 */
int arcs_sample_dry(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                    const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                    const arcs_dry_params* dry, const int32_t* breakers, int n_breakers, uint64_t seed,
                    uint64_t step, int32_t* out_ids, int32_t* out_status, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * arcs_sample_hybrid_nucleus: a baseline nucleus (top-p) sampler, for A/B
 * timing against arcs_sample.  It is the selector the pages report for their
 * device sampler (Arc PR #194, squashed commit #130, "hybrid nucleus
 * selector"): per row, the ids of the order (value desc, id asc) are
 * enumerated one at a time, for at most `budget` ids, until their mass
 * reaches top_p of the row's mass, and the kept set is that prefix; past the
 * budget, 32 halvings of the value key find the largest threshold whose mass
 * reaches top_p, and every id at or above it is kept (ties at the boundary
 * value all kept: the wider rule).  top_p >= 1 keeps every id.  No penalties,
 * top-k or min-p.  The draw is arcs_sample's: the first kept id in id order
 * whose running weight exceeds u * S_K, u the SplitMix64 uniform of counter
 * step * 2^32 + b under seed.  fp32 weights, fp64 sums.
 *   logits       device bf16 [B, row_stride], rows 16-byte aligned,
 *                V % 8 == 0, V <= 131072
 *   temperature  device float[B], > 0 and finite (else row status 1)
 *   top_p        device float[B], > 0 (else row status 2)
 *   budget       ids enumerated before bisection takes over, 0 .. 4096
 *   out_ids      device int32[B]; out_kept device int32[B] (kept set size) or
 *                NULL; out_status device int32[B] or NULL
 * Returns ARCS_OK, ARCS_ERR_BAD_DTYPE (not bf16), ARCS_ERR_BAD_VOCAB,
 * ARCS_ERR_MISALIGNED, ARCS_ERR_BAD_BUDGET or another negative arcs_status.
 */
int arcs_sample_hybrid_nucleus(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                               const float* temperature, const float* top_p, int budget, uint64_t seed,
                               uint64_t step, int32_t* out_ids, int32_t* out_kept, int32_t* out_status,
                               void* stream);

/* Bytes of device workspace arcs_sample, arcs_sample_keyed and
 * arcs_sample_debug need for this shape: B * P * 16 for the split batches
 * described under arcs_sample, else 0. */
size_t arcs_sample_workspace_bytes(int64_t B, int64_t V, int dtype);

/*
 * arcs_long_history_workspace_bytes: B * V * 4 (saturating).  A call with
 * history arrays (arcs_sample, arcs_sample_keyed, arcs_sample_debug,
 * arcs_sample_dry) whose workspace is at least this large and 16-byte aligned
 * samples rows whose active penalties the LDS tables cannot hold (more than
 * ARCS_MAX_HISTORY distinct history ids, or V > ARCS_MAX_PENALTY_VOCAB)
 * instead of failing them: such a row's penalised logits (repetition,
 * frequency and presence, Arc PR #222 page, section 3(a); and the
 * DRY record if active) are written in binary32 to the row's slice of the
 * workspace (offset row * V * 4) and the general pipeline samples that copy,
 * in two more launches on the same stream that other rows leave at once.
 * The results equal the table path's.  The workspace is owned by the caller,
 * not read before it is written, and shared only by calls ordered on one
 * stream; smaller workspaces (or none) keep the status codes
 * ARCS_ROW_HISTORY_TOO_LONG / ARCS_ROW_VOCAB_TOO_LARGE.
 */
size_t arcs_long_history_workspace_bytes(int64_t B, int64_t V);

/* Human-readable text for an arcs_status or ARCS_ROW_* code. */
const char* arcs_status_string(int code);

/*
 * arcs_sample_debug: arcs_sample plus test hooks, kept off the hot path.
 *   uniforms    device double[B] in [0, 1) replacing the SplitMix64 draw, or NULL
 *   out_probs   device float[B, V]: the filtered distribution q (0 outside
 *               the kept set; greedy rows get a one-hot), or NULL
 *   out_stats   device arcs_row_stats[B], or NULL
 */
int arcs_sample_debug(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const arcs_row_params* params, const int32_t* hist_ids,
                      const int64_t* hist_offsets, uint64_t seed, uint64_t step,
                      int32_t* out_ids, int32_t* out_status, void* workspace,
                      size_t workspace_bytes, const double* uniforms, float* out_probs,
                      arcs_row_stats* out_stats, void* stream);

/*
 * arcs_top_logprobs: the n most probable tokens of each row with their
 * log-probabilities, next to the draw (Arc PR #222, section 3(c): the host
 * sampler finds them by a partial sort of the probabilities).  Per row b, at
 * temperature T = temperature[b] (1 when `temperature` is NULL):
 *   z = logits widened to float32 (NaN -> -inf, -0 -> +0), m = max z,
 *   w_v = exp((z_v - m) / T), w_v = 1 where z_v == m (so +inf logits share
 *   the mass and a row of -inf is uniform), S = sum of w,
 *   out_ids[b, r], r < n: the r-th id of the order (z desc, id asc);
 *   out_logprobs[b, r] = ln(w / S) of that id, computed in binary64 and
 *   rounded to binary32.
 * No penalties or filters are applied: this is the distribution of the
 * logits at temperature T.  Rows with V < n end with id -1 and -inf.
 *   logits        device, [B, row_stride] of dtype
 *   temperature   device, float[B], or NULL; a row whose T is NaN, <= 0 or
 *                 +inf gets ids -1, logprobs NaN, status ARCS_ROW_BAD_TEMPERATURE
 *   n             1 .. ARCS_MAX_TOP_LOGPROBS (else ARCS_ERR_BAD_TOP_N)
 *   out_ids       device, int32[B * n] (row-major)
 *   out_logprobs  device, float[B * n] (row-major)
 *   out_status    device, int32[B], or NULL
 * V must not exceed ARCS_TOP_LOGPROBS_MAX_VOCAB (else ARCS_ERR_BAD_VOCAB).
 * Returns ARCS_OK or a negative arcs_status (nothing launched then).
 */
int arcs_top_logprobs(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                      const float* temperature, int n, int32_t* out_ids, float* out_logprobs,
                      int32_t* out_status, void* stream);

/*
 * arcs_commit_tokens: publish the tokens of one decode step to the host
 * without a synchronisation (Arc PR #217, "What this does", step 3: the
 * token goes into the next step's input buffer, the device position moves on
 * and the token is published into a pinned, mapped host ring; the fault
 * handling there: the commit range-checks token and position before writing
 * anything and latches a code into a pinned fault word).  One launch:
 *   p = *position;
 *   refused, with *fault set to the code if it was ARCS_FAULT_NONE, when a
 *   token is outside [0, V) and is not -1 (ARCS_FAULT_TOKEN_RANGE; -1 is the
 *   sampler's mark for a row it refused, published as it is so that one
 *   request's invalid parameters do not stop the batch), or the slot p % capacity
 *   still holds a step the host has not drained, p - *drained >= capacity
 *   (ARCS_FAULT_RING_OVERRUN); also refused, silently, while *fault is set
 *   (a latched fault stops publication until the host clears it); nothing
 *   else is written then;
 *   otherwise next_input[b] = ids[b] (if next_input is not NULL),
 *   ring[(p % capacity) * B + b] = ids[b], then, after a system-scope fence,
 *   *published = p + 1 and *position = p + 1.
 *   ids          device, int32[B] (e.g. out_ids of arcs_sample)
 *   next_input   device, int32[B], or NULL
 *   position     device, uint64: the step counter
 *   ring         pinned host memory (hipHostMalloc), int32[capacity * B]
 *   published    pinned host memory, uint64: steps whose tokens are in the ring
 *   drained      pinned host memory, uint64, written by the host: steps consumed
 *   fault        pinned host memory, uint32, sticky; the host clears it
 * The host polls *published and *fault with plain volatile loads.  Calls on
 * one stream run in order; the ring and words belong to that stream.
 * Returns ARCS_OK or a negative arcs_status (nothing launched then).
 */
int arcs_commit_tokens(const int32_t* ids, int64_t B, int64_t V, int32_t* next_input, uint64_t* position,
                       int32_t* ring, uint64_t capacity, uint64_t* published, const uint64_t* drained,
                       uint32_t* fault, void* stream);

/*
 * arcs_w4_logits: the logits arcs_argmax, arcs_sample and arcs_top_logprobs
 * read, from the last hidden states and a vocabulary head whose weights are
 * held in 4 bits with a scale for each group of group_size of them:
 *   logits[b, v] = sum over groups g of
 *       scales[v, g] * sum over d in g of (q[v, d] - zeros[v, g]) * hidden[b, d]
 * with q in 0 .. 15 and zeros 8 where `zeros` is NULL.  Products and sums are
 * held in binary32 (levels q - z and hidden states enter exactly, hidden states
 * below 2^-107 in magnitude may count as 0) and each logit is rounded once to
 * its type.  An infinity in a hidden state gives its row the infinities of the
 * levels' signs, NaN at a level of 0; NaN and infinities in a scale reach its
 * column.
 *   hidden         device bfloat16 [B, hidden_stride], rows 16-byte aligned
 *   D              hidden size, 1 .. ARCS_MAX_HIDDEN, a multiple of group_size
 *   qweight        device bytes [V, qweight_stride], rows 16-byte aligned: byte d / 2
 *                  holds weight d in its low nibble and weight d + 1 in its high
 *                  nibble (d even); qweight_stride >= D / 2
 *   scales         device [V, scale_stride] of scale_dtype (ARCS_DTYPE_BF16 or
 *                  ARCS_DTYPE_F32), scale_stride >= D / group_size elements
 *   zeros          device bytes [V, zero_stride], 0 .. 15 each (the upper four
 *                  bits are ignored), or NULL
 *   group_size     32, 64 or 128
 *   logits         device [B, row_stride] of logits_dtype, row_stride >= V
 *   workspace      device scratch of at least arcs_w4_logits_workspace_bytes(),
 *                  256-byte aligned, not read before it is written; calls that
 *                  share one must be ordered on one stream; may be NULL when
 *                  none is needed
 * The logits must not overlap an input.
 * Returns ARCS_OK or a negative arcs_status (nothing launched then):
 * ARCS_ERR_BAD_STRIDE for any stride below its row, or a stride of qweight,
 * scales or zeros above 2^21, ARCS_ERR_MISALIGNED for `hidden` or `qweight`
 * rows that are not 16-byte aligned or another array not aligned to its
 * element, ARCS_ERR_BAD_BATCH also for B above 2^19 or B * V above 2^36,
 * ARCS_ERR_BAD_VOCAB also for V above 2^28.
 */
int arcs_w4_logits(const void* hidden, int64_t B, int64_t D, int64_t hidden_stride, const uint8_t* qweight,
                   int64_t V, int64_t qweight_stride, const void* scales, int scale_dtype,
                   int64_t scale_stride, const uint8_t* zeros, int64_t zero_stride, int group_size,
                   void* logits, int logits_dtype, int64_t row_stride, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Bytes of workspace arcs_w4_logits needs: 0 for batches of at most 16 rows. */
size_t arcs_w4_logits_workspace_bytes(int64_t B, int64_t D, int group_size);

/*
 * arcs_linear_cross_entropy: the log-probabilities of given tokens, or the
 * training loss, straight from the hidden states and the vocabulary head; the
 * [N, V] logits are never kept.  Per row n, at temperature T = temperature[n]
 * (1 when `temperature` is NULL):
 *   z_v = dot(hidden[n], weight[v]) / T,
 *   out_lse[n] = ln sum_v exp(z_v),   out_loss[n] = out_lse[n] - z_target[n],
 * so -out_loss is the target's log-probability, as arcs_top_logprobs reports
 * it for the logits' distribution.  Rows whose target is ignore_index (which
 * may be any value) are left out: loss and lse 0, and what their hidden states
 * hold (NaN, say) reaches nothing.  Rows whose target is outside [0, V), or
 * whose T is NaN, <= 0 or +inf, get loss and lse NaN and a row status.  Other NaN
 * and infinities propagate: a row with a NaN or +inf logit has a NaN loss.
 *   hidden      device [N, hidden_stride] of dtype (ARCS_DTYPE_BF16 or
 *               ARCS_DTYPE_F32), hidden_stride >= D, D in 1 .. ARCS_MAX_HIDDEN
 *   weight      device [V, weight_stride] of the same dtype, weight_stride >= D
 *   targets     device int32[N]
 *   temperature device float[N], or NULL
 *   out_loss    device float[N]
 *   out_lse     device float[N] (arcs_linear_cross_entropy_backward reads it)
 *   out_status  device int32[N]: ARCS_ROW_OK, ARCS_ROW_BAD_TARGET or
 *               ARCS_ROW_BAD_TEMPERATURE; or NULL
 *   workspace   device scratch of at least
 *               arcs_linear_cross_entropy_workspace_bytes(N, V, D, dtype, 0),
 *               256-byte aligned, not read before it is written; calls that share
 *               one must be ordered on one stream
 * Products and sums are held in binary32.  The same call gives the same bits.
 * Outputs must not overlap inputs or each other.
 * Rows on the 16-byte grid (pointers, strides and D, in each array and output;
 * weight_stride below 2^23 bytes) take the matrix kernels, others a general
 * kernel that takes 8 to 14 times as long in bfloat16 and 2 to 4 times in float32.
 * Returns ARCS_OK or a negative arcs_status (nothing launched then);
 * ARCS_ERR_BAD_BATCH also for more than 65,535 tiles of 128 rows, or more than
 * 2^23 tiles of 128 x 128 in [N, the larger of V and D].
 */
int arcs_linear_cross_entropy(const void* hidden, int64_t hidden_stride, const void* weight,
                              int64_t weight_stride, int dtype, int64_t N, int64_t V, int64_t D,
                              const int32_t* targets, int32_t ignore_index, const float* temperature,
                              float* out_loss, float* out_lse, int32_t* out_status, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * arcs_linear_cross_entropy_backward: the gradients of
 * sum_n grad_loss[n] * out_loss[n] of the call above.  With p = softmax(z_n)
 * computed again from out_lse, in pieces of the vocabulary:
 *   dz[n, v] = (p_v - [v == target]) * grad_loss[n] / T,
 *   out_dhidden[n] = sum_v dz[n, v] * weight[v],
 *   out_dweight[v] = sum_n dz[n, v] * hidden[n].
 * Rows that are ignored or refused have a zero gradient and add nothing.
 *   lse          device float[N], out_lse of the forward call on the same inputs
 *                (its rounding to binary32, up to 2^-24 |lse|, is a relative error
 *                of every p_v)
 *   grad_loss    device float[N]
 *   out_dhidden  device [N, D] of dtype, dense, or NULL (not wanted)
 *   out_dweight  device [V, D] of dtype, dense, or NULL (not wanted); written
 *                whole, not added to.  One of the two must be given.
 *   workspace    arcs_linear_cross_entropy_workspace_bytes(N, V, D, dtype, 1)
 * Sums are held in binary32.  For bfloat16 the matrix kernels hold dz of a
 * piece in bfloat16, in units of the largest |grad_loss / T| of the call (so
 * that equal weights are not rounded); rows whose |grad_loss / T| is 2^-100 of
 * the largest or less may have a gradient of 0, for float32 too.  Other
 * arguments and errors as the forward call; outputs must not overlap inputs.
 */
int arcs_linear_cross_entropy_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                       int64_t weight_stride, int dtype, int64_t N, int64_t V, int64_t D,
                                       const int32_t* targets, int32_t ignore_index, const float* temperature,
                                       const float* lse, const float* grad_loss, void* out_dhidden,
                                       void* out_dweight, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace the two calls above need (0 for sizes they refuse). */
size_t arcs_linear_cross_entropy_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int backward);

/* Activations of arcs_linear. */
typedef enum arcs_activation {
  ARCS_ACT_NONE = 0,
  ARCS_ACT_RELU = 1,
  ARCS_ACT_GELU = 2,       /* z (1 + erf(z / sqrt 2)) / 2 */
  ARCS_ACT_GELU_TANH = 3,  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
  ARCS_ACT_SILU = 4,       /* z / (1 + exp(-z)) */
  ARCS_ACT_SOFTCAP = 5     /* c tanh(z / c), c = softcap */
} arcs_activation;

/*
 * arcs_linear: a linear layer with bias, activation and residual, in one pass:
 * the logits of a head whose weights are not quantised, for arcs_argmax,
 * arcs_sample and arcs_top_logprobs, or the blocks in front of it, such as a
 * draft head's hidden + silu(weight hidden + bias).  Per row n:
 *   z = hidden[n] weight^T + bias,   out[n] = residual[n] + act(z).
 * Products, sums and the activation are held in binary32 and each result is
 * rounded once to its type: act(z) is within 20 2^-24 of itself where it is a
 * normal number.  NaN and infinities propagate.
 *   hidden      device [N, hidden_stride] of dtype (ARCS_DTYPE_BF16 or
 *               ARCS_DTYPE_F32), hidden_stride >= D, D in 1 .. ARCS_MAX_HIDDEN
 *   weight      device [V, weight_stride] of dtype, weight_stride >= D
 *   bias        device [V] of dtype, or NULL
 *   activation  an arcs_activation; softcap is read for ARCS_ACT_SOFTCAP only,
 *               and has to be within 2^-100 .. 2^100 there
 *   residual    device [N, residual_stride] of dtype, residual_stride >= V, or NULL
 *   out         device [N, out_stride] of out_dtype, out_stride >= V; may be
 *               the residual itself where type and stride are the same
 *   out_pre     device [N, V] of dtype, dense: z, which the backward pass of an
 *               activation needs; or NULL
 *   workspace   device scratch of at least arcs_linear_workspace_bytes(),
 *               256-byte aligned, not read before it is written; calls that share
 *               one must be ordered on one stream; may be NULL when none is needed
 * The same call gives the same bits.  Outputs must not overlap inputs (but for
 * the residual, where that is not the hidden states) or each other
 * (ARCS_ERR_OVERLAP).  Rows of hidden and weight that are not on the
 * 16-byte grid (pointer, stride and D; strides of 2^23 bytes or more count as such)
 * are copied to the workspace first, unless N is at most 16.
 * Returns ARCS_OK or a negative arcs_status (nothing launched then);
 * ARCS_ERR_BAD_BATCH also for N above 2^22 or N * V above 2^40,
 * ARCS_ERR_BAD_VOCAB also for V above 2^24.
 */
int arcs_linear(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride, int dtype,
                int64_t N, int64_t V, int64_t D, const void* bias, int activation, float softcap,
                const void* residual, int64_t residual_stride, void* out, int out_dtype, int64_t out_stride,
                void* out_pre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * arcs_linear_backward: the gradients of sum(grad_out * out) of the call above:
 *   dz = grad_out * act'(z),   out_dhidden = dz weight,
 *   out_dweight = dz^T hidden,   out_dbias = the sums of dz over n.
 * (The residual's gradient is grad_out itself.)
 *   pre          out_pre of the forward call, [N, V] of dtype, dense; may be NULL
 *                for ARCS_ACT_NONE
 *   grad_out     device [N, grad_stride] of grad_dtype, grad_stride >= V
 *   out_dhidden  device [N, D] of dtype, dense, or NULL (not wanted)
 *   out_dweight  device [V, D] of dtype, dense, or NULL (not wanted)
 *   out_dbias    device [V] of dtype, or NULL (not wanted); one of the three
 *                must be given; each is written whole, not added to
 *   workspace    arcs_linear_backward_workspace_bytes()
 * dz is rounded to dtype before the products (as z was), and summed for out_dbias
 * before that; sums are held in binary32 or more.  act'(z) is within 32 2^-24 of the
 * sum of its terms' sizes (for the softcap, 16 (1 + |z / softcap|) 2^-24 of itself).
 * Other arguments and errors as the forward call; ARCS_ERR_BAD_VOCAB also for V above 2^21 - 8.
 */
int arcs_linear_backward(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride,
                         int dtype, int64_t N, int64_t V, int64_t D, int activation, float softcap,
                         const void* pre, const void* grad_out, int grad_dtype, int64_t grad_stride,
                         void* out_dhidden, void* out_dweight, void* out_dbias, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace the two calls need (0 for sizes they refuse).
 * rows_aligned: whether all rows of hidden and weight are on the 16-byte grid
 * (pointers, strides and D, and strides below 2^23 bytes); 0 is enough for either.
 */
size_t arcs_linear_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int rows_aligned);
size_t arcs_linear_backward_workspace_bytes(int64_t N, int64_t V, int64_t D, int dtype, int rows_aligned);

/*
 * arcs_adjust_logits: logits as the sampler is to see them: penalties for what a
 * row's history holds, biases, and the tokens its grammar allows.  Per row b,
 * in binary32 and in this order:
 *   1. ids in the history: the presence, frequency and repetition penalties of
 *      params[b], the same operations as arcs_sample's (ids outside [0, V) are
 *      skipped; duplicates count).  The rows then go to arcs_sample with the same
 *      records and without a history;
 *   2. ids in the bias list: their bias is added (the sum in list order
 *      of those of an id listed more than once; ids outside [0, V) are skipped);
 *   3. tokens whose mask bit is 0 become -inf, whatever they held;
 * then each value is rounded once to out_dtype.  Other tokens keep their value,
 * NaN and infinities too.
 *   params        device, arcs_row_params[B] (its other fields are not read), or
 *                 NULL: no penalties (the history must be NULL then)
 *   hist_ids, hist_offsets   as in arcs_sample, or both NULL
 *   bias_ids      device int32, bias_values device float, bias_offsets device
 *                 int64[B + 1] CSR offsets into both; or all three NULL
 *   mask          device uint32 [masks, mask_stride], mask_stride >= ceil(V / 32):
 *                 bit v % 32 of word v / 32 is 1 where token v is allowed; or NULL
 *   mask_rows     device int32[B]: the mask of each row, -1 for a row without
 *                 one; or NULL: row b has mask b (masks >= B then)
 *   out           device [B, out_stride] of out_dtype, out_stride >= V; may be
 *                 `logits` itself with the same type and stride: then only
 *                 16-byte groups that change are written
 *   out_status    device int32[B]: ARCS_ROW_OK; ARCS_ROW_BAD_PENALTY (a penalty
 *                 is not finite, or repetition < 0) or ARCS_ROW_BAD_MASK: the row
 *                 is filled with NaN; ARCS_ROW_NOTHING_ALLOWED: the mask leaves
 *                 no token, the row is -inf.  Or NULL
 * Outputs must not overlap inputs otherwise (ARCS_ERR_OVERLAP where logits and
 * out do).  Returns ARCS_OK or a negative arcs_status (nothing launched then);
 * ARCS_ERR_BAD_BATCH also for B * (ceil(V / 4096) + 1) above 2^31 - 1.
 */
int arcs_adjust_logits(const void* logits, int dtype, int64_t B, int64_t V, int64_t row_stride,
                       const arcs_row_params* params, const int32_t* hist_ids, const int64_t* hist_offsets,
                       const int32_t* bias_ids, const float* bias_values, const int64_t* bias_offsets,
                       const uint32_t* mask, int64_t masks, int64_t mask_stride, const int32_t* mask_rows,
                       void* out, int out_dtype, int64_t out_stride, int32_t* out_status, void* stream);

/* One tensor of a list of gradients: `count` elements, dense. */
typedef struct arcs_tensor {
  const void* data;  /* device, aligned to its element; may be NULL when count is 0 */
  void* out;         /* where arcs_clip_gradients writes: `data` (in place, of the same type)
                        or memory that overlaps no tensor; NULL: it writes nothing for this one */
  int64_t count;     /* >= 0 */
  int32_t dtype;
  int32_t out_dtype;
} arcs_tensor;

/*
 * arcs_gradient_plan: lists the pieces of n tensors (a host array) in `plan`, host
 * memory of arcs_gradient_plan_bytes().  The caller copies the plan to the device once
 * and uses it as long as the tensors stay where they are.  Tensors must not
 * overlap each other.  Nothing is launched.  ARCS_ERR_BAD_BATCH for n < 0,
 * ARCS_ERR_BAD_PLAN for a count below 0 or a total above 2^40 elements,
 * ARCS_ERR_OVERLAP for an `out` that is `data` of another type.
 */
int arcs_gradient_plan(const arcs_tensor* tensors, int64_t n, void* plan, size_t plan_bytes);
/* Bytes of the plan of n tensors (0 for a list that is refused, and for one without elements). */
size_t arcs_gradient_plan_bytes(const arcs_tensor* tensors, int64_t n);

/*
 * arcs_gradient_norm: out_norm[0] = sqrt(sum of x^2 over all elements of the plan's
 * tensors), summed in binary64 in an order that does not depend on timing and
 * rounded once to binary32 (0 for an empty plan).
 *   plan        device copy of arcs_gradient_plan's, 8-byte aligned; may be
 *               NULL when plan_bytes is 0
 *   out_norm    device float[1]
 *   workspace   device scratch of at least arcs_gradient_workspace_bytes(plan_bytes),
 *               256-byte aligned; calls that share one must be ordered on one stream
 */
int arcs_gradient_norm(const void* plan, size_t plan_bytes, float* out_norm, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * arcs_clip_gradients: the norm as above and, where it is above max_norm and
 * finite, every element times max_norm / norm (taken in binary64, rounded to
 * binary32 and then to its output's type).  Otherwise the elements keep their
 * values: tensors in place are not touched, others are copied to their outputs.
 * The norm is compared and divided by in binary64: gradients whose norm is past
 * binary32's range are scaled too, and out_norm[0] is infinity then.
 *   max_norm    >= 0 (ARCS_ERR_BAD_NORM for NaN and negative values)
 * Tensors of the plan without an `out` count in the norm and are not written.
 */
int arcs_clip_gradients(const void* plan, size_t plan_bytes, double max_norm, float* out_norm, void* workspace,
                        size_t workspace_bytes, void* stream);

size_t arcs_gradient_workspace_bytes(size_t plan_bytes);

/* Library version, major * 10000 + minor * 100 + patch. */
int arcs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ARCS_H */
