/*
 * llp.h -- C ABI of the fused linear log-prob operator for AMD Instinct MI355X (gfx950).
 *
 * The operator turns a language model's final hidden states and its (vocabulary-partitioned)
 * output projection into per-token log-probabilities of given target ids, optional entropy,
 * their gradients, the rank-ordered merge of per-shard partials, and compact top-p replay
 * scores. Sources (three pull-request pages; cited by title and section):
 *   [CUDA provider] "feat(rl-kernel): add CUDA linear logp provider integration"
 *   [ROCm provider] "feat(rl-kernel): add ROCm linear logp provider integration"
 *   [top-p replay]  "Perf/cuda compact top p replay"
 *
 * The request structs mirror the provider contract of [CUDA provider, "Changes" /
 * "Linear-logp provider contract"]: a request (LinearLogpRequest) carrying a projection
 * (LinearProjection: output-layer hidden states, local projection weight and bias), a
 * vocabulary partition (VocabPartition: tensor-parallel vocabulary range, real and padded
 * vocabulary sizes) and a token layout (TokenLayout: packing and loss masks), plus target
 * ids and the temperature.
 *
 * Conventions for every call:
 *   - Tensor pointers are DEVICE pointers unless stated otherwise; the caller owns all memory
 *     and keeps it valid until the work enqueued on `stream` completes.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *   - Execution calls (every call but llp_open and the workspace sizes) never allocate, never
 *     synchronize and never read device memory on the host, so they can be captured into a
 *     HIP graph. Results are bitwise reproducible run to run. What is computed per row (scores
 *     and their partials, dhidden, quantised and embedded rows) is a function of that row's
 *     inputs and the fixed kernel configuration only and does not depend on how rows are
 *     batched or ordered; nor do a preference pair's own loss and rewards. Sums over a batch
 *     (dweight, dbias, the embedding gradient, the losses' totals and statistics) are
 *     reproducible for a fixed batch.
 *   - Errors are returned as llp_status; no exception crosses the ABI and the library never
 *     aborts. llp_last_error() describes the last non-OK status of the calling thread.
 *   - Host-detectable problems (shapes, strides, alignment, partition, temperature, limits)
 *     return LLP_ERR_INVALID_ARGUMENT before anything is enqueued. Data-dependent problems
 *     found on the device (a bad target or replay id, a malformed cu_seqlens) are OR-ed into
 *     the optional device `status_word` (LLP_STATUS_* bits) and the affected rows get -inf
 *     log-probabilities; nothing becomes NaN. (What the losses and the embedding do with such
 *     rows stands at their requests.)
 */
#ifndef LLP_H
#define LLP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLP_API __attribute__((visibility("default")))

#define LLP_VERSION "0.1.0"
/* Most replay candidate ids per row ([top-p replay, "Changes" table]: up to 64 ids). */
#define LLP_MAX_REPLAY_IDS 64
/* Most vocabulary shards llp_merge combines in one call. */
#define LLP_MAX_WORLD 64

/* Return codes. Only llp_open returns LLP_ERR_UNAVAILABLE: that is the one status a caller
 * may treat as "provider unavailable, use another path" ([CUDA provider, "Motivation"]:
 * auto mode falls back only on an explicit unavailable report; strict mode fails closed).
 * Loading (llp_open) is kept apart from execution so that an execution failure is never
 * mistaken for unavailability ([CUDA provider], review discussion). */
typedef enum {
  LLP_OK = 0,
  LLP_ERR_UNAVAILABLE = 1,      /* no gfx950 device / kernels cannot be loaded (llp_open) */
  LLP_ERR_INVALID_ARGUMENT = 2, /* malformed request; nothing was enqueued */
  LLP_ERR_UNSUPPORTED = 3,      /* well formed but outside the compiled envelope */
  LLP_ERR_HIP = 4,              /* a HIP runtime call or kernel launch failed */
  LLP_ERR_INTERNAL = 5
} llp_status;

/* Device status-word bits (OR-ed with integer atomics). */
enum {
  LLP_STATUS_TARGET_OUT_OF_RANGE = 1, /* a scored row's target is outside [0, real_vocab) */
  LLP_STATUS_TARGET_NOT_FOUND = 2,    /* no shard (or no replay candidate) holds the target */
  LLP_STATUS_REPLAY_ID_INVALID = 4,   /* a replay id outside [-1, real_vocab) (slot ignored) */
  LLP_STATUS_LAYOUT_INVALID = 8,      /* cu_seqlens not 0 = c0 <= c1 <= ... <= cS = T */
  LLP_STATUS_TOKEN_OUT_OF_RANGE = 16, /* an embedded token id outside [0, real_vocab) */
  LLP_STATUS_VALUE_NOT_FINITE = 32,   /* a scored row of a loss, a beam's logits or its score
                                         hold a NaN or an infinity that has no meaning there */
  LLP_STATUS_PARENT_INVALID = 64      /* a parent outside [-1, number of source beams) */
};

enum { LLP_DTYPE_BF16 = 1, LLP_DTYPE_F32 = 2 };
enum { LLP_OP_FORWARD = 1, LLP_OP_BACKWARD = 2 };
/* Request flags.
 *   LLP_FLAG_WANT_ENTROPY     the forward also computes the entropy.
 *   LLP_FLAG_OVERWRITE_GRADS  llp_backward writes dweight and dbias (= this call's gradient,
 *                             padding rows 0) instead of adding to them: the first chunk of a
 *                             step needs no zeroed buffer and no read of one. Ignored by
 *                             llp_forward.
 *   LLP_FLAG_G_SLABS          llp_backward never holds the whole G: it computes G, its
 *                             dhidden and dweight products one vocabulary slab of
 *                             LLP_G_SLAB_COLUMNS local columns at a time, in slab order, and
 *                             adds each slab's dhidden into fp32 partials in the workspace.
 *                             The workspace holds one slab of G instead of all of it
 *                             (llp_workspace_bytes sizes it from this flag). dweight and dbias
 *                             are bitwise those of the default mode; dhidden agrees to rounding
 *                             (its vocabulary sum runs slab by slab) and is still bitwise
 *                             reproducible and independent of the batch. Ignored by
 *                             llp_forward. */
enum { LLP_FLAG_WANT_ENTROPY = 1, LLP_FLAG_OVERWRITE_GRADS = 2, LLP_FLAG_G_SLABS = 4 };
#define LLP_G_SLAB_COLUMNS 32768

/* Library identity and route evidence ([CUDA provider, "Changes"]: validation of identity;
 * native/provider route evidence). */
typedef struct {
  char name[32];       /* "lm_head_linear_logp_amd" */
  char version[16];    /* LLP_VERSION */
  char arch[32];       /* device architecture the kernels run on, e.g. "gfx950" */
  char route[128];     /* kernel variant and tile configuration */
  int32_t max_replay_ids;
  int32_t num_cus;
  int32_t device;
  int32_t reserved;
} llp_info;

/* LinearProjection ([CUDA provider, "Megatron integration"]: output-layer hidden states, local
 * projection weight and bias).
 *   hidden  [T, H] bf16, row stride hidden_stride (elements, >= H, multiple of 8), 16-byte
 *           aligned base.
 *   weight  [local_size, H] bf16 -- this shard's rows of the LM-head weight, row stride
 *           weight_stride (elements, >= H, multiple of 8), 16-byte aligned base. Rows past the
 *           shard's real columns (padding) are never read into a result.
 *   bias    [local_size] of bias_dtype (LLP_DTYPE_BF16 or LLP_DTYPE_F32), or NULL; 16-byte
 *           aligned base for F32, 8-byte for BF16.
 *   H must be a positive multiple of 64, at most 2^20 (else LLP_ERR_UNSUPPORTED). Operand
 *   rows are addressed with 32-bit byte offsets, which bounds the envelope (else
 *   LLP_ERR_UNSUPPORTED): hidden_stride and weight_stride < 2^23, T * hidden_stride * 2 < 2^31
 *   (the bytes the T hidden rows span), T <= 2^23 - 256 and local_size <= 2^23 - 256. */
typedef struct {
  const void* hidden;
  int64_t hidden_stride;
  const void* weight;
  int64_t weight_stride;
  const void* bias;
  int32_t bias_dtype;
  int32_t reserved;
  int64_t hidden_size; /* H */
} llp_projection;

/* VocabPartition ([CUDA provider, "Megatron integration"]: tensor-parallel vocabulary range
 * and real/padded vocabulary sizes; [CUDA provider, "CUDA compatibility and launch support"]:
 * tensor parallelism is the vocabulary reduction group). The shard owns global ids
 * [offset, offset + local_size); its real columns are the first
 * clamp(real_vocab - offset, 0, local_size). Requires 0 <= offset, offset + local_size <=
 * padded_vocab, 0 < real_vocab <= padded_vocab, 0 <= rank < world <= LLP_MAX_WORLD, and for
 * world == 1: offset == 0 and local_size == padded_vocab. local_size == 0 is an empty shard. */
typedef struct {
  int64_t offset;
  int64_t local_size;
  int64_t real_vocab;
  int64_t padded_vocab;
  int32_t rank;
  int32_t world;
} llp_vocab_partition;

/* TokenLayout ([CUDA provider, "Summary"]: the framework keeps token layout and masking;
 * [CUDA provider, "CUDA compatibility and launch support"]: context parallelism is row
 * ownership). Rows are independent: num_seqs/cu_seqlens describe packing and are validated
 * on the device (LLP_STATUS_LAYOUT_INVALID) but do not change any row's arithmetic.
 *   num_tokens  T >= 0 rows (llp_forward / llp_backward: at most 2^23 - 256, else
 *               LLP_ERR_UNSUPPORTED; llp_forward_logits: below 2^31, else INVALID_ARGUMENT).
 *   cu_seqlens  int32 [num_seqs + 1] device array or NULL (num_seqs ignored when NULL).
 *   loss_mask   uint8 [T] device array (non-zero = scored) or NULL (every row scored).
 * Unscored rows are not computed; all their outputs are written as 0 and they get no
 * gradient. Targets are row-aligned: the operator never shifts them. */
typedef struct {
  int64_t num_tokens;
  int32_t num_seqs;
  int32_t reserved;
  const int32_t* cu_seqlens;
  const uint8_t* loss_mask;
} llp_token_layout;

/* LinearLogpRequest ([CUDA provider, "Motivation"]: logits or projection, target ids,
 * tensor-parallel group, token layout and masks).
 *   target_ids   int64 [T] device array (global vocabulary ids).
 *   temperature  finite, > 0. Logits are z = (hidden . weight^T + bias) * fl32(1/temperature):
 *                temperature is applied exactly once ([ROCm provider, "Megatron
 *                integration"]; [top-p replay, "Summary"]).
 *   flags        LLP_FLAG_WANT_ENTROPY, LLP_FLAG_OVERWRITE_GRADS, LLP_FLAG_G_SLABS.
 *   status_word  int32 device word OR-ed with LLP_STATUS_* bits, or NULL. */
typedef struct {
  llp_projection proj;
  llp_vocab_partition vocab;
  llp_token_layout layout;
  const int64_t* target_ids;
  float temperature;
  uint32_t flags;
  int32_t* status_word;
} llp_request;

/* Per-shard partials, one value per row, all device arrays of length T.
 * Written by llp_forward and llp_top_p_replay, read by llp_merge.
 *   target_logit  z[target] if the target lies in this shard's real columns, else 0
 *   in_range      1 if it does, else 0
 *   lse           log-sum-exp of z over the shard's real columns (-inf for no columns)
 *   entropy       entropy of the shard-local softmax (0 for no columns); NULL = not wanted
 *   logp          target_logit - lse if in_range, else -inf; NULL = not wanted.
 *                 For an unsharded call (world == 1) this is the final log-probability.
 * Unscored rows: every field 0. */
typedef struct {
  float* target_logit;
  uint8_t* in_range;
  float* lse;
  float* entropy;
  float* logp;
} llp_partials;

/* Merged per-row results of llp_merge (device arrays of length T; entropy may be NULL). */
typedef struct {
  float* logp;
  float* lse;
  float* entropy;
} llp_final_out;

/* Inputs of llp_backward (device arrays of length T).
 *   lse       the merged (global) log-sum-exp of every row (llp_merge / llp_forward at world 1)
 *   dlogp     upstream gradient of each row's logp
 *   dentropy  upstream gradient of each row's entropy, or NULL
 *   entropy   the merged entropy (required when dentropy is given) */
typedef struct {
  const float* lse;
  const float* dlogp;
  const float* dentropy;
  const float* entropy;
} llp_bwd_in;

/* Outputs of llp_backward.
 *   dhidden  bf16 [T, H], row stride dhidden_stride (>= H, multiple of 8): OVERWRITTEN with
 *            this shard's contribution G . weight (unscored rows 0). With world > 1 the caller
 *            sums the shards' dhidden.
 *   dweight  fp32 [local_size, H], row stride dweight_stride (>= H, multiple of 4, < 2^21,
 *            else INVALID_ARGUMENT / UNSUPPORTED), 16-byte aligned base: ACCUMULATED (+=) with
 *            G^T . hidden over this call's rows; padding rows untouched. With
 *            LLP_FLAG_OVERWRITE_GRADS: OVERWRITTEN with G^T . hidden, padding rows (and every
 *            row of a call with no rows) written as 0; bitwise the accumulate form applied
 *            to a zeroed buffer.
 *   dbias    fp32 [local_size] ACCUMULATED (OVERWRITTEN with LLP_FLAG_OVERWRITE_GRADS), or
 *            NULL.
 * G[t, v] = (dlogp_t (1[v = target_t] - p_tv) - dentropy_t p_tv (z_tv - E_p z_t)) / temperature
 * with p = exp(z - lse), is rounded to bf16 once and feeds all three products. */
typedef struct {
  void* dhidden;
  int64_t dhidden_stride;
  float* dweight;
  int64_t dweight_stride;
  float* dbias;
} llp_bwd_out;

/* Compact top-p replay request ([top-p replay, "Summary"]: replay the native finite nucleus,
 * scoring the compact replay ids directly instead of a full-vocabulary keep mask;
 * [top-p replay, "Changes" table]: validate replay inputs, sort and deduplicate up to 64 ids,
 * apply temperature, return local reductions).
 *   logits        [T, local_size] this shard's local logits (logits_dtype: LLP_DTYPE_F32 or
 *                 LLP_DTYPE_BF16), row stride logits_stride elements.
 *   num_tokens    T rows, 0 <= T < 2^31 (else LLP_ERR_INVALID_ARGUMENT).
 *   replay_ids    int64 [T, num_replay] global ids, row stride replay_stride; -1 = empty slot;
 *                 num_replay in [1, LLP_MAX_REPLAY_IDS]. Duplicates count once.
 *   processed_logprobs must be 1: replay scores processed (temperature/top-p) log-probs
 *                 only; raw mode is rejected ([top-p replay], review: replay only for
 *                 processed logprobs).
 * Writes target_logit, in_range, lse and logp of `out` (entropy must be NULL). */
typedef struct {
  const void* logits;
  int32_t logits_dtype;
  int32_t num_replay;
  int64_t logits_stride;
  int64_t num_tokens;
  llp_vocab_partition vocab;
  const int64_t* replay_ids;
  int64_t replay_stride;
  const int64_t* target_ids;
  const uint8_t* loss_mask;
  float temperature;
  int32_t processed_logprobs;
  int32_t* status_word;
} llp_topp_request;

/* Logits-input forward request ([CUDA provider, "Megatron integration"]: strict LM-head local
 * logits are reused when available, avoiding a second projection; [top-p replay, "Summary"]:
 * temperature is applied exactly once).
 *   logits        [T, local_size] of logits_dtype (LLP_DTYPE_F32 or LLP_DTYPE_BF16), the
 *                 shard's unscaled local logits h . W^T + b; row stride logits_stride
 *                 (elements, >= local_size; the rows must be 16-byte aligned: base aligned and
 *                 stride * element size a multiple of 16). Padded columns are never read.
 *   vocab, layout, target_ids, temperature, flags, status_word: as in llp_request (z = x *
 *                 fl32(1/temperature); flags: LLP_FLAG_WANT_ENTROPY). */
typedef struct {
  const void* logits;
  int32_t logits_dtype;
  int32_t reserved;
  int64_t logits_stride;
  llp_vocab_partition vocab;
  llp_token_layout layout;
  const int64_t* target_ids;
  float temperature;
  uint32_t flags;
  int32_t* status_word;
} llp_logits_request;

/* Dense keep-mask replay request ([top-p replay, "Changes" table]: the local logits are
 * reused with a keep mask and excluded entries are -inf; [top-p replay, "Validation"]: the
 * dense-mask and compact forms agree bitwise across shard offsets and empty shards).
 *   logits        as in llp_topp_request, with 16-byte aligned rows (see llp_logits_request).
 *   keep_mask     uint8 [num_tokens, local_size], row stride keep_stride (bytes, >= local_size,
 *                 multiple of 16), 16-byte aligned base; nonzero = the column is in the row's
 *                 nucleus. Columns past the shard's real ones are ignored.
 *   num_tokens, vocab, target_ids, loss_mask, temperature, processed_logprobs, status_word:
 *                 as in llp_topp_request. */
typedef struct {
  const void* logits;
  int32_t logits_dtype;
  int32_t processed_logprobs;
  int64_t logits_stride;
  const uint8_t* keep_mask;
  int64_t keep_stride;
  int64_t num_tokens;
  llp_vocab_partition vocab;
  const int64_t* target_ids;
  const uint8_t* loss_mask;
  float temperature;
  int32_t reserved;
  int32_t* status_word;
} llp_keep_mask_request;

/* ---- Scoring with a head in 8-bit integers -------------------------------------------------
 * A frozen policy (the reference of a KL term or of a preference loss) needs log-probabilities
 * and no gradient. Its head may then be held as int8 rows with one fp32 scale per vocabulary
 * column, and the hidden states be quantised per token: half the bytes and twice the MFMA rate
 * of bf16. */
#define LLP_INT8_COLUMNS 128 /* int8 rows hold a multiple of this many columns */

/* Symmetric 8-bit quantisation of rows.
 *   x      [rows, cols] bf16 or fp32 (x_dtype), row stride x_stride elements (>= cols), any
 *          alignment of its element type.
 *   q      int8 [rows, cols_padded], cols_padded = cols rounded up to LLP_INT8_COLUMNS; row
 *          stride q_stride bytes (>= cols_padded, multiple of 16), 16-byte aligned base.
 *          Columns cols .. cols_padded - 1 are written as 0.
 *   scale  fp32 [rows].
 * With a = max_k |x[r][k]|: scale[r] = max(a, 1e-30) * fl32(1/127) and q[r][k] = x[r][k] /
 * scale[r] (fp32, correctly rounded) to the nearest integer, ties to even. A row of zeros
 * gives q = 0. A row holding an infinity or NaN gives q = 0 and scale = NaN. */
typedef struct {
  const void* x;
  int32_t x_dtype;
  int32_t reserved;
  int64_t x_stride;
  int64_t rows; /* 0 <= rows < 2^31 */
  int64_t cols; /* 1 <= cols <= 2^20 */
  int8_t* q;
  int64_t q_stride;
  float* scale;
} llp_quant_request;

/* llp_request with the projection in 8-bit integers: z = (sum_k hidden[t][k] weight[v][k] *
 * hidden_scale[t] * weight_scale[v] + bias[v]) * fl32(1/temperature), the sum exact in int32.
 *   hidden        int8 [T, hidden_size], row stride hidden_stride bytes; weight int8
 *                 [local_size, hidden_size], row stride weight_stride bytes: strides >=
 *                 hidden_size and multiples of 16, 16-byte aligned bases. As
 *                 llp_quantize_rows writes them (values in [-127, 127]; -128 is read as such).
 *   hidden_scale  fp32 [T]; weight_scale fp32 [local_size]; bias as in llp_projection, aligned
 *                 to its element type.
 *   hidden_size   the padded width: a positive multiple of LLP_INT8_COLUMNS, at most 2^17 - 128
 *                 (the int32 sums cannot overflow; else LLP_ERR_UNSUPPORTED).
 *   hidden_stride and weight_stride < 2^24, T * hidden_stride < 2^31 and the row limits of
 *   llp_projection (else LLP_ERR_UNSUPPORTED). Where hidden_size / LLP_INT8_COLUMNS is odd,
 *   ceil(T / 256) * ceil(real columns / 256) < 2^23 (else LLP_ERR_UNSUPPORTED).
 * The other fields are those of llp_request (flags: LLP_FLAG_WANT_ENTROPY). Values that are not
 * finite (scales of rows that were not) spread as they do in llp_forward. */
typedef struct {
  const int8_t* hidden;
  int64_t hidden_stride;
  const float* hidden_scale;
  const int8_t* weight;
  int64_t weight_stride;
  const float* weight_scale;
  const void* bias;
  int32_t bias_dtype;
  uint32_t flags;
  int64_t hidden_size;
  llp_vocab_partition vocab;
  llp_token_layout layout;
  const int64_t* target_ids;
  float temperature;
  int32_t reserved;
  int32_t* status_word;
} llp_int8_request;

/* ---- Losses on the scored log-probabilities ------------------------------------------------
 * Both read what llp_forward / llp_merge write (logp, entropy) and write what llp_backward takes
 * (dlogp, dentropy). Rows whose loss_mask is 0 are never read into a result (they may hold
 * anything) and get gradient 0. */
enum { LLP_KL_K1 = 1, LLP_KL_K2 = 2, LLP_KL_K3 = 3 };
enum { LLP_REDUCE_TOKEN_MEAN = 1, LLP_REDUCE_SEQ_MEAN = 2, LLP_REDUCE_SUM = 3 };
/* Log ratios are clamped to [-20, 20] before their exponential; outside, it passes no gradient. */
#define LLP_LOG_RATIO_MAX 20
#define LLP_POLICY_STATS 8

/* Clipped policy loss with a KL term and an entropy bonus. For a scored row with
 * d = logp - old_logp, r = exp(clamp(d)), A = advantages:
 *   policy  = -min(A r, A clip(r, 1 - clip_low, 1 + clip_high)); with dual_clip = c > 0 and A < 0
 *             at most -A c. Where the clip holds (r > 1 + clip_high for A > 0; r < 1 - clip_low
 *             or r > c for A < 0) it passes no gradient, else d policy / d logp = -A r. The
 *             borders, the clamps' too, are compared in 64 bits: d > log(1 + clip_high) and so on.
 *   kl      = with x = ref_logp - logp: k1 = -x, k2 = x^2 / 2, k3 = exp(clamp(x)) - clamp(x) - 1.
 *   loss    = sum_t w_t (policy + kl_coef kl - entropy_coef entropy)
 * and w_t by `reduction`: TOKEN_MEAN 1 / (scored rows); SEQ_MEAN 1 / (scored rows of t's
 * sequence * sequences that have any); SUM 1. `denominator` (a device float, or NULL) takes the
 * place of the number of rows (TOKEN_MEAN) or sequences (SEQ_MEAN), for a batch spread over
 * several processes; a value that is not finite and > 0 gives w = 0, as a batch without scored
 * rows does.
 *   logp, old_logp, advantages   fp32 [T]
 *   ref_logp   fp32 [T], or NULL (then no KL term; kl_coef must be 0)
 *   entropy    fp32 [T], or NULL (then no bonus; entropy_coef must be 0)
 *   layout     T < 2^31; num_seqs <= 2^23 (else LLP_ERR_UNSUPPORTED); cu_seqlens is required
 *              for SEQ_MEAN. A malformed cu_seqlens sets
 *              LLP_STATUS_LAYOUT_INVALID, and with SEQ_MEAN every output is 0 then.
 *   0 <= clip_low <= 1, clip_high >= 0, dual_clip 0 (none) or > 1, all coefficients finite.
 * A scored row holding a value that is not finite (of the arrays that are used) sets
 * LLP_STATUS_VALUE_NOT_FINITE, adds nothing and gets gradient 0; it still counts as scored. */
typedef struct {
  const float* logp;
  const float* old_logp;
  const float* advantages;
  const float* ref_logp;
  const float* entropy;
  llp_token_layout layout;
  double clip_low;
  double clip_high;
  double dual_clip;
  double kl_coef;
  double entropy_coef;
  int32_t kl_kind;
  int32_t reduction;
  const float* denominator;
  int32_t* status_word;
} llp_policy_request;

/*   loss      fp32 [1]
 *   stats     fp32 [LLP_POLICY_STATS], or NULL: loss, then the w-weighted sums of policy, kl,
 *             entropy, clipped (0/1), r and -d, then the number of scored rows
 *   dloss     fp32 [1] upstream gradient of the loss (device), or NULL for 1
 *   dlogp     fp32 [T] d loss / d logp * dloss, or NULL
 *   dentropy  fp32 [T], or NULL (needs entropy when given) */
typedef struct {
  float* loss;
  float* stats;
  const float* dloss;
  float* dlogp;
  float* dentropy;
} llp_policy_out;

enum { LLP_PREF_SIGMOID = 1, LLP_PREF_HINGE = 2, LLP_PREF_IPO = 3 };

/* Preference loss of P pairs of packed sequences: sequence 2i is pair i's chosen response, 2i + 1
 * the rejected one (layout.num_seqs = 2 P <= 2^23, cu_seqlens required). For each sequence R = the sum,
 * or with `average` the mean, of logp - ref_logp over its scored rows (0 when it has none), and
 * h = R_chosen - R_rejected:
 *   SIGMOID  (1 - e) softplus(-m) + e softplus(m), m = beta h - gamma, e = label_smoothing
 *   HINGE    max(0, 1 - m)
 *   IPO      (h - 1 / (2 beta))^2
 * loss = sum_i pair_weight_i l_i / P, or without the 1 / P for LLP_REDUCE_SUM.
 *   logp         fp32 [T];  ref_logp fp32 [T] or NULL
 *   pair_weight  fp32 [P] or NULL (1). A pair of weight 0 adds nothing whatever its rows hold; its
 *                own outputs (l_i, beta R) are written as any pair's, or as 0 where a scored row is
 *                not finite, without a status.
 *   beta > 0, 0 <= label_smoothing < 1 (0 unless SIGMOID), gamma finite (0 for IPO)
 *   reduction    LLP_REDUCE_SUM, or LLP_REDUCE_TOKEN_MEAN for the mean over pairs
 * Another pair with a scored row (or a weight) that is not finite sets
 * LLP_STATUS_VALUE_NOT_FINITE, adds nothing, and its outputs and gradients are 0. A malformed cu_seqlens sets
 * LLP_STATUS_LAYOUT_INVALID and every output is 0. */
typedef struct {
  const float* logp;
  const float* ref_logp;
  const float* pair_weight;
  llp_token_layout layout;
  double beta;
  double gamma;
  double label_smoothing;
  int32_t kind;
  int32_t average;
  int32_t reduction;
  int32_t reserved;
  int32_t* status_word;
} llp_pref_request;

/*   loss                       fp32 [1]
 *   pair_loss                  fp32 [P] (l_i), or NULL
 *   chosen, rejected           fp32 [P] (beta R), or NULL
 *   dloss, dlogp               as in llp_policy_out */
typedef struct {
  float* loss;
  float* pair_loss;
  float* chosen;
  float* rejected;
  const float* dloss;
  float* dlogp;
} llp_pref_out;

/* ---- Token embedding -----------------------------------------------------------------------
 * The input side of a vocabulary-partitioned table (the LM head's own weight in a model that
 * ties the two): out[t] = scale * weight[id_t - offset], and its gradient, which adds into the
 * same fp32 dweight that llp_backward writes.
 *   token_ids    int64 [T]; a row whose token_mask (uint8 [T], or NULL) is 0, or whose id is
 *                another shard's, gives a row of zeros and no gradient (the caller sums the
 *                shards); so does an id outside [0, real_vocab), with
 *                LLP_STATUS_TOKEN_OUT_OF_RANGE.
 *   weight       [local_size, hidden_size] of weight_dtype (bf16 or fp32); llp_embedding only
 *   hidden_size  a positive multiple of 8, at most 2^20. Every row operand has a stride in
 *                elements >= hidden_size that is a multiple of 8, and a 16-byte aligned base.
 *   num_tokens   0 <= T <= 2^23 - 256; local_size <= 2^23 - 256 (else LLP_ERR_UNSUPPORTED)
 *   scale        finite */
typedef struct {
  const int64_t* token_ids;
  const uint8_t* token_mask;
  int64_t num_tokens;
  llp_vocab_partition vocab;
  int64_t hidden_size;
  float scale;
  uint32_t flags; /* llp_embedding_backward: LLP_FLAG_OVERWRITE_GRADS */
  int32_t* status_word;
} llp_embedding_request;

/* ---- Products of operands in 8-bit floating point -------------------------------------------
 * A head (or another projection) held as e4m3 bytes with an fp32 scale for each block of
 * 128 x 128, multiplied with activations quantised in groups of 128 columns: logits for decoding,
 * and, with the operands quantised along the other dimension, both gradients. An operand is a
 * matrix [rows, depth] whose depth is the summed dimension, padded with zero bytes to a multiple
 * of LLP_FP8_BLOCK. Its scales come in one of two layouts, G = depth / LLP_FP8_BLOCK:
 *   by group  (block_rows 1): scale[g * scale_stride + r], scale_stride >= rows
 *   by block  (block_rows 128): scale[(r / 128) * scale_stride + g], scale_stride >= G */
#define LLP_FP8_BLOCK 128

/* Quantisation of x, or with `transpose` of its transpose: the operand Y [M, K] is x [rows, cols]
 * or its transpose.
 *   x      [rows, cols] bf16 or fp32 (x_dtype), row stride x_stride elements (>= cols), any
 *          alignment of its element type.
 *   q      e4m3 (finite, no infinities) [M, K rounded up to LLP_FP8_BLOCK], row stride q_stride
 *          bytes (>= the padded K, multiple of 16), 16-byte aligned base. Columns past K are
 *          written as 0.
 *   scale  fp32, as above for `block_rows` (1 or LLP_FP8_BLOCK).
 * With a = max |Y| over a block: its scale is max(a, 1e-30) * fl32(1/448) and q = Y / scale (fp32,
 * correctly rounded) to the nearest e4m3 value, ties to even. A block holding an infinity or NaN
 * gives q = 0 and scale = NaN. rows and cols >= 0, below 2^31; ceil(rows / 128) * ceil(cols / 128)
 * < 2^23 (else LLP_ERR_UNSUPPORTED). */
typedef struct {
  const void* x;
  int32_t x_dtype;
  int32_t block_rows;
  int64_t x_stride;
  int64_t rows;
  int64_t cols;
  int32_t transpose;
  int32_t reserved;
  uint8_t* q;
  int64_t q_stride;
  float* scale;
  int64_t scale_stride;
} llp_fp8_quant_request;

/* A product of two such operands over their common depth:
 *   p[t][v] = sum_g x_scale[g][t] weight_scale[v / 128][g] sum_{k in g} x[t][k] weight[v][k]
 *   x       [rows, depth] e4m3, scales by group; weight [cols, depth] e4m3, scales by block. Row
 *           strides in bytes, >= depth and multiples of 16, at most 2^23; 16-byte aligned bases.
 *   depth   a multiple of LLP_FP8_BLOCK, 0 <= depth <= 2^23 (0: the sums are 0).
 *   rows, cols  0 .. 2^23 - 256; ceil(rows / 32) * ceil(cols / 128) < 2^23 (else
 *           LLP_ERR_UNSUPPORTED).
 * The groups are added in fp32 in ascending order from group (v / 1280) mod the number of groups on, then
 * from 0, so an element depends on its two rows and v alone, whatever the call's other rows. v is counted in
 * the call: a weight row that is another column of another call, as in a shard and in the whole weight,
 * gives a sum in another order, equal to rounding. A
 * group's 128 products are summed in fp32 where out is fp32; where it
 * is bf16 they are summed by the 8-bit matrix instructions, which cut 8 products at a time about 14
 * bits below the largest of them. That is a hundredth of the rounding to bf16 of a result as large as its products
 * make it, and more than it where they nearly cancel (operands drawn as activations and weights are: 1.7 % of the
 * results not the nearest bf16 value, 0.3 % a step or more off). fp32 results, rounded, have none of it.
 * llp_linear_fp8: out[t][v] = p + bias[v], [rows, cols] of out_dtype, row stride out_stride
 *   elements (>= cols), any alignment of its element type, rounded once. bias [cols] of bias_dtype
 *   or NULL. flags must be 0.
 * llp_dweight_fp8: the gradient of a weight, with `weight` the transposed upstream gradient [V, T]
 *   and `x` the transposed input [H, T]: out[v][t] += p (fp32), [cols, rows], row stride
 *   out_stride >= rows, below 2^24 in fp32 (else LLP_ERR_UNSUPPORTED). With LLP_FLAG_OVERWRITE_GRADS
 *   it is written, and out_dtype may be bf16.
 *   bias must be NULL. */
typedef struct {
  const uint8_t* x;
  int64_t x_stride;
  const float* x_scale;
  int64_t x_scale_stride;
  const uint8_t* weight;
  int64_t weight_stride;
  const float* weight_scale;
  int64_t weight_scale_stride;
  const void* bias;
  int32_t bias_dtype;
  int32_t out_dtype;
  void* out;
  int64_t out_stride;
  int64_t rows;
  int64_t cols;
  int64_t depth;
  uint32_t flags;
  int32_t reserved;
} llp_fp8_linear_request;

/* ---- Beam search ----------------------------------------------------------------------------
 * One step over B sequences of K beams each: every beam's most likely tokens from its logits (per
 * vocabulary shard), the selection over a sequence's beams, shards and vocabulary, and the
 * reordering of whatever is kept per beam. */
#define LLP_MAX_BEAMS 64      /* beams of a sequence, and candidates selected for it */

/* Candidates of each row of logits: the `num` largest real columns (1 <= num <= LLP_MAX_BEAMS), by
 * logit descending and token ascending, and what normalises the row.
 *   logits   as in llp_logits_request; num_rows rows, below 2^22.
 *   vocab    as in llp_request; local_size at most 2^21 and padded_vocab < 2^40 (else
 *            LLP_ERR_UNSUPPORTED).
 *   temperature  in [2^-64, 2^64]; z = x * fl32(1/temperature).
 * -inf logits are no candidates. A row that holds a NaN or +inf among its real columns sets
 * LLP_STATUS_VALUE_NOT_FINITE and gets no candidates and sum = -1. */
typedef struct {
  const void* logits;
  int32_t logits_dtype;
  int32_t num;
  int64_t logits_stride;
  int64_t num_rows;
  llp_vocab_partition vocab;
  float temperature;
  int32_t reserved;
  int32_t* status_word;
} llp_beam_request;

/* What llp_beam_candidates writes and llp_beam_select reads, device arrays:
 *   value   fp32 [num_rows, num], the logits x in descending order (-inf past the last candidate)
 *   token   int64 [num_rows, num] global ids (-1 past the last candidate)
 *   max     fp32 [num_rows], the largest logit (-inf for a row without one)
 *   sum     fp64 [num_rows], sum exp((x - max) c), c = fl32(1/temperature), over the real columns; 0 for a
 *           row without a finite logit. A term below 1 is within 2^-23 (1 + (max - x) c) of itself, and
 *           terms are added in fp64. */
typedef struct {
  float* value;
  int64_t* token;
  float* max;
  double* sum;
} llp_beam_parts;

/* Selection over `world` shards' candidates (rank order) of num_seqs x num_beams rows.
 *   scores     fp32 [num_seqs, num_beams], a beam's score so far
 *   finished   uint8 [num_seqs, num_beams] or NULL: a finished beam has one candidate, end_id, with
 *              its own score
 *   num        candidates in each row of the parts; num_out chosen, 1 <= num_out <= num <=
 *              LLP_MAX_BEAMS (so the choice is one over the whole vocabulary); num_seqs < 2^22
 * A candidate's total is score + ((x - M) c - log(sum_r sum[r] e^{(max[r] - M) c})) with M =
 * max_r max[r] and c = fl32(1/temperature), in fp64; one whose token is outside [0, 2^40) is none. Chosen are the num_out largest totals above -inf, by total
 * descending, then beam, then token ascending.
 * A beam whose score is -inf has no candidates; nor has one whose score is NaN or +inf or whose
 * row has sum < 0 in a shard, which sets LLP_STATUS_VALUE_NOT_FINITE. */
typedef struct {
  int32_t world;
  int32_t num;
  const llp_beam_parts* parts; /* HOST array of `world` structs */
  int64_t num_seqs;
  int32_t num_beams;
  int32_t num_out;
  const float* scores;
  const uint8_t* finished;
  int64_t end_id;
  float temperature;
  int32_t reserved;
  int32_t* status_word;
} llp_beam_select_request;

/*   token   int64 [num_seqs, num_out], -1 where fewer candidates than num_out have a total
 *   parent  int32 [num_seqs, num_out], the beam it continues (-1 there)
 *   score   fp32 [num_seqs, num_out], the total (-inf there) */
typedef struct {
  int64_t* token;
  int32_t* parent;
  float* score;
} llp_beam_out;

/* Reordering of what is kept per beam: for every sequence b and slot j, row b * num_out + j of dst
 * takes row b * num_src + parents[b][j] of src. A parent of -1 leaves the slot as it is; one
 * outside [-1, num_src) does too and sets LLP_STATUS_PARENT_INVALID.
 * A state is `rows` of `outer` pieces of `inner` contiguous bytes: row r's piece o begins at
 * base + r * row_stride + o * outer_stride (bytes). Pieces of one state do not overlap.
 *   src, dst  HOST arrays of num_states device pointers, all of the one shape; dst[i] == src[i] is
 *             the reordering in place (num_src must equal num_out then, and dst's strides src's),
 *             otherwise no dst may overlap a src. In place are all
 *             states of a call or none.
 *   parents   int32 [num_seqs, num_out]
 *   0 <= num_seqs < 2^22, 0 <= num_states; 1 <= num_src, num_out <= LLP_MAX_BEAMS. A state whose
 *   sequences hold 2^32 loads or more together is LLP_ERR_UNSUPPORTED (a load is 16 bytes, or less
 *   where pieces or their strides are no multiples of 16: 4 or 1).
 * States must not overlap each other. */
typedef struct {
  const void* const* src;
  void* const* dst;
  int32_t num_states;
  int32_t num_src;
  int32_t num_out;
  int32_t reserved;
  int64_t num_seqs;
  int64_t outer;
  int64_t inner;
  int64_t src_row_stride;
  int64_t src_outer_stride;
  int64_t dst_row_stride;
  int64_t dst_outer_stride;
  const int32_t* parents;
  int32_t* status_word;
} llp_beam_reorder_request;

/* Loading phase: checks that `device` is a gfx950 GPU and loads the kernels on it; fills
 * `info` (may be NULL). Returns LLP_ERR_UNAVAILABLE when there is no such device. Must
 * succeed on the current device before any execution call. Idempotent. */
LLP_API llp_status llp_open(int32_t device, llp_info* info);

/* Workspace bytes an execution call needs for `req` and `op` (LLP_OP_FORWARD or
 * LLP_OP_BACKWARD): a pure function of the shapes (and, for the backward, of
 * LLP_FLAG_G_SLABS). The caller allocates it (device memory, 256-byte aligned) and passes it
 * to that call. */
LLP_API llp_status llp_workspace_bytes(const llp_request* req, int32_t op, size_t* bytes);

/* Fused forward for one shard: per row, z over the shard's real columns, lse, the target
 * logit, optional entropy and the local logp, without materializing [T, V] logits
 * ([top-p replay, "Changes" table]: fused linear-logp kernel; [CUDA provider, "Motivation"]).
 * Writes every non-NULL field of `out` (target_logit, in_range and lse are required; entropy
 * only with LLP_FLAG_WANT_ENTROPY). */
LLP_API llp_status llp_forward(const llp_request* req, const llp_partials* out,
                               void* workspace, size_t workspace_bytes, void* stream);

/* llp_forward without a caller workspace, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation). The
 * workspace is a static device array of the library, 32 MiB on every device the library is
 * opened on, held until the process ends; the call allocates nothing. Results are bitwise
 * those of llp_forward (the same kernels).
 *   Limit: llp_workspace_bytes(req, LLP_OP_FORWARD) must be at most 32 MiB, else
 *   LLP_ERR_UNSUPPORTED before anything is enqueued: e.g. up to 4608 rows over a 151669-column
 *   shard, or 18432 over a 37984-column one.
 *   Every call on one device shares that device's array. Calls that overlap on a device (on
 *   different streams, or from several threads without ordering) race and give wrong results:
 *   serialize them. No part of the array needs to start at zero (a call writes every value it
 *   reads before reading it), so nothing is cleared between calls. */
LLP_API llp_status llp_forward_noalloc(const llp_request* req, const llp_partials* out,
                                       void* stream);

/* Rank-ordered merge of `world` shards' partials ([top-p replay, "Summary"]: rank-ordered
 * reductions, shards with no candidates handled). `parts` is a HOST array of `world` structs
 * in rank order whose fields are device arrays of length num_tokens (entropy NULL in every
 * part = no merged entropy). Per row: lse = M + log sum_r exp(lse_r - M) over non-empty
 * shards; logp = target_logit of the first shard holding the target minus lse, or -inf
 * (LLP_STATUS_TARGET_NOT_FOUND); entropy = sum_r exp(lse_r - lse)(entropy_r + lse - lse_r).
 * loss_mask (device, may be NULL) zeroes unscored rows. out->entropy may be NULL.
 * 0 <= num_tokens < 2^31 (else LLP_ERR_INVALID_ARGUMENT). */
LLP_API llp_status llp_merge(int32_t world, const llp_partials* parts, int64_t num_tokens,
                             const uint8_t* loss_mask, const llp_final_out* out,
                             int32_t* status_word, void* stream);

/* Backward for one shard: dhidden = G . weight (overwrite), dweight += G^T . hidden,
 * dbias += sum_t G (= instead of += with LLP_FLAG_OVERWRITE_GRADS) (gradients must flow: [CUDA provider, "Motivation"], strict mode rejects
 * detached gradients). Needs the merged lse of every scored row. */
LLP_API llp_status llp_backward(const llp_request* req, const llp_bwd_in* in,
                                const llp_bwd_out* out, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Compact top-p replay scoring for one shard (see llp_topp_request). Follow with llp_merge
 * over the shards for the final log-probability. */
LLP_API llp_status llp_top_p_replay(const llp_topp_request* req, const llp_partials* out,
                                    void* stream);

/* Logits-input forward for one shard: the partials of llp_forward (target_logit, in_range,
 * lse required; entropy with LLP_FLAG_WANT_ENTROPY; logp optional) from the shard's local
 * logits instead of hidden states and weight. Needs no workspace. */
LLP_API llp_status llp_forward_logits(const llp_logits_request* req, const llp_partials* out,
                                      void* stream);

/* Dense keep-mask replay scoring for one shard: the partials of llp_top_p_replay (entropy must
 * be NULL) for the nucleus given as a keep mask. For a nucleus of at most LLP_MAX_REPLAY_IDS
 * ids the results are bitwise those of llp_top_p_replay given the same ids. */
LLP_API llp_status llp_keep_mask_replay(const llp_keep_mask_request* req,
                                        const llp_partials* out, void* stream);

/* 8-bit quantisation of rows (see llp_quant_request). Needs no workspace. */
LLP_API llp_status llp_quantize_rows(const llp_quant_request* req, void* stream);

/* llp_forward with the projection in 8-bit integers (see llp_int8_request): the same partials,
 * checks and guarantees; the workspace size comes from llp_int8_workspace_bytes. */
LLP_API llp_status llp_int8_workspace_bytes(const llp_int8_request* req, size_t* bytes);
LLP_API llp_status llp_forward_int8(const llp_int8_request* req, const llp_partials* out,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* The losses (see llp_policy_request and llp_pref_request): the loss and, where out->dlogp (and
 * out->dentropy) is given, its gradient. Workspace: device memory, 256-byte aligned; where the
 * size is 0 (small calls) none is taken and it may be NULL. */
LLP_API llp_status llp_policy_workspace_bytes(const llp_policy_request* req, size_t* bytes);
LLP_API llp_status llp_policy_loss(const llp_policy_request* req, const llp_policy_out* out,
                                   void* workspace, size_t workspace_bytes, void* stream);
LLP_API llp_status llp_preference_workspace_bytes(const llp_pref_request* req, size_t* bytes);
LLP_API llp_status llp_preference_loss(const llp_pref_request* req, const llp_pref_out* out,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* Token embedding (see llp_embedding_request): `weight` and `out` share weight_dtype; out is
 * [T, hidden_size], every row written. Needs no workspace. */
LLP_API llp_status llp_embedding(const llp_embedding_request* req, const void* weight,
                                 int32_t weight_dtype, int64_t weight_stride, void* out,
                                 int64_t out_stride, void* stream);

/* Its gradient: dweight[v] += scale * sum of dout[t] over the rows with token v, in ascending t
 * within fixed groups of rows (reproducible for a fixed batch). dout [T, hidden_size] of dout_dtype (bf16 or
 * fp32). dweight fp32 [local_size, hidden_size]: ACCUMULATED, rows no token names untouched;
 * with LLP_FLAG_OVERWRITE_GRADS every row is written, those rows as 0. */
LLP_API llp_status llp_embedding_workspace_bytes(const llp_embedding_request* req, size_t* bytes);
LLP_API llp_status llp_embedding_backward(const llp_embedding_request* req, const void* dout,
                                          int32_t dout_dtype, int64_t dout_stride, float* dweight,
                                          int64_t dweight_stride, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Quantisation in 8-bit floating point (see llp_fp8_quant_request) and products of such operands
 * (see llp_fp8_linear_request). No workspace. */
LLP_API llp_status llp_quantize_blocks(const llp_fp8_quant_request* req, void* stream);
/* Two of them in one pass over their common x: `groups` with block_rows 1 and not transposed, `blocks`
 * with block_rows 128 and transposed, as the two gradients of a product take an upstream gradient. */
LLP_API llp_status llp_quantize_both(const llp_fp8_quant_request* groups,
                                     const llp_fp8_quant_request* blocks, void* stream);
LLP_API llp_status llp_linear_fp8(const llp_fp8_linear_request* req, void* stream);
LLP_API llp_status llp_dweight_fp8(const llp_fp8_linear_request* req, void* stream);

/* One step of a beam search (see llp_beam_request, llp_beam_select_request and
 * llp_beam_reorder_request). No workspace. */
LLP_API llp_status llp_beam_candidates(const llp_beam_request* req, const llp_beam_parts* out, void* stream);
LLP_API llp_status llp_beam_select(const llp_beam_select_request* req, const llp_beam_out* out,
                                   void* stream);
LLP_API llp_status llp_beam_reorder(const llp_beam_reorder_request* req, void* stream);

/* Message for the calling thread's last non-OK status ("" if none). */
LLP_API const char* llp_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LLP_H */
