// llp_api_ops.cpp -- C-ABI entry points of the operators around the linear log-prob: 8-bit
// scoring, the policy and preference losses, and the token embedding. As in llp_api.cpp,
// validation runs before any HIP call.
#include <hip/hip_runtime_api.h>
#include <math.h>

#include "llp.h"
#include "llp_host.h"
#include "llp_internal.h"

using namespace llp;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 23) - 256;

// `need` 0: the call takes no workspace.
llp_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return LLP_OK;
  LLP_CHECK(bytes >= need, LLP_ERR_INVALID_ARGUMENT,
            "workspace of %zu bytes is smaller than the %zu required", bytes, need);
  LLP_CHECK(workspace != nullptr && aligned(workspace, 256), LLP_ERR_INVALID_ARGUMENT,
            "workspace must be non-NULL and 256-byte aligned");
  return LLP_OK;
}

// ---- 8-bit scoring --------------------------------------------------------------------------
llp_status check_int8(const llp_int8_request* req) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  const llp_int8_request& p = *req;
  const int64_t T = p.layout.num_tokens, K = p.hidden_size;
  LLP_CHECK(T >= 0, LLP_ERR_INVALID_ARGUMENT, "num_tokens=%lld < 0", (long long)T);
  LLP_CHECK(T <= kMaxRows, LLP_ERR_UNSUPPORTED, "num_tokens %lld too large", (long long)T);
  llp_status st = check_partition(p.vocab);
  if (st != LLP_OK) return st;
  LLP_CHECK(K > 0, LLP_ERR_INVALID_ARGUMENT, "hidden_size must be > 0");
  // (2^17 - 128) * 128 * 128 < 2^31: the int32 sums cannot overflow.
  LLP_CHECK(K % LLP_INT8_COLUMNS == 0 && K < (1 << 17), LLP_ERR_UNSUPPORTED,
            "hidden_size %lld must be a multiple of %d below 2^17", (long long)K, LLP_INT8_COLUMNS);
  LLP_CHECK(p.hidden_stride >= K && p.hidden_stride % 16 == 0, LLP_ERR_INVALID_ARGUMENT,
            "hidden_stride %lld must be >= hidden_size and a multiple of 16",
            (long long)p.hidden_stride);
  LLP_CHECK(p.weight_stride >= K && p.weight_stride % 16 == 0, LLP_ERR_INVALID_ARGUMENT,
            "weight_stride %lld must be >= hidden_size and a multiple of 16",
            (long long)p.weight_stride);
  // Tile rows are addressed with 32-bit byte offsets, as llp_forward's.
  LLP_CHECK(p.hidden_stride < (int64_t(1) << 24) && p.weight_stride < (int64_t(1) << 24),
            LLP_ERR_UNSUPPORTED, "hidden_stride and weight_stride must be < 2^24");
  LLP_CHECK(T * p.hidden_stride < (int64_t(1) << 31), LLP_ERR_UNSUPPORTED,
            "hidden spans T * hidden_stride = %lld bytes; must be < 2^31",
            (long long)(T * p.hidden_stride));
  LLP_CHECK(p.vocab.local_size <= kMaxRows, LLP_ERR_UNSUPPORTED,
            "local_size %lld exceeds 2^23 - 256", (long long)p.vocab.local_size);
  // A K of an odd number of 128s takes a workgroup of 512 threads per tile; a launch holds fewer
  // than 2^32 threads.
  LLP_CHECK(K % (2 * LLP_INT8_COLUMNS) == 0 ||
                round_up(T, 256) / 256 * (round_up(local_real(p.vocab), 256) / 256) < (int64_t(1) << 23),
            LLP_ERR_UNSUPPORTED, "%lld tokens of %lld columns are too many tiles for this hidden_size",
            (long long)T, (long long)local_real(p.vocab));
  if (T > 0) {
    LLP_CHECK(p.hidden && p.hidden_scale, LLP_ERR_INVALID_ARGUMENT,
              "hidden and hidden_scale are required");
    LLP_CHECK(aligned(p.hidden, 16), LLP_ERR_INVALID_ARGUMENT, "hidden not 16-byte aligned");
    LLP_CHECK(p.target_ids != nullptr, LLP_ERR_INVALID_ARGUMENT, "target_ids is NULL");
  }
  if (local_real(p.vocab) > 0) {
    LLP_CHECK(p.weight && p.weight_scale, LLP_ERR_INVALID_ARGUMENT,
              "weight and weight_scale are required");
    LLP_CHECK(aligned(p.weight, 16), LLP_ERR_INVALID_ARGUMENT, "weight not 16-byte aligned");
  }
  LLP_CHECK(aligned(p.hidden_scale, 4) && aligned(p.weight_scale, 4), LLP_ERR_INVALID_ARGUMENT,
            "hidden_scale and weight_scale must be aligned to fp32");
  if (p.bias != nullptr) {
    LLP_CHECK(p.bias_dtype == LLP_DTYPE_BF16 || p.bias_dtype == LLP_DTYPE_F32,
              LLP_ERR_INVALID_ARGUMENT, "bias_dtype %d is not BF16 or F32", p.bias_dtype);
    LLP_CHECK(aligned(p.bias, p.bias_dtype == LLP_DTYPE_F32 ? 4 : 2), LLP_ERR_INVALID_ARGUMENT,
              "bias not aligned to its element type");
  }
  LLP_CHECK(isfinite(p.temperature) && p.temperature > 0.f, LLP_ERR_INVALID_ARGUMENT,
            "temperature must be finite and > 0");
  LLP_CHECK((p.flags & ~uint32_t(LLP_FLAG_WANT_ENTROPY)) == 0, LLP_ERR_INVALID_ARGUMENT,
            "unknown flags 0x%x", p.flags);
  if (p.layout.cu_seqlens != nullptr)
    LLP_CHECK(p.layout.num_seqs >= 0, LLP_ERR_INVALID_ARGUMENT, "num_seqs < 0");
  return LLP_OK;
}

// ---- Losses ---------------------------------------------------------------------------------
// One workgroup per sequence: a launch holds fewer than 2^32 threads.
constexpr int32_t kMaxSeqs = 1 << 23;

llp_status check_loss_layout(const llp_token_layout& l) {
  LLP_CHECK(l.num_tokens >= 0 && l.num_tokens < (int64_t(1) << 31), LLP_ERR_INVALID_ARGUMENT,
            "num_tokens out of range");
  if (l.cu_seqlens != nullptr) {
    LLP_CHECK(l.num_seqs >= 0, LLP_ERR_INVALID_ARGUMENT, "num_seqs < 0");
    LLP_CHECK(l.num_seqs <= kMaxSeqs, LLP_ERR_UNSUPPORTED, "num_seqs %d exceeds 2^23", l.num_seqs);
  }
  return LLP_OK;
}

llp_status check_policy(const llp_policy_request* req) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  llp_status st = check_loss_layout(req->layout);
  if (st != LLP_OK) return st;
  const int64_t T = req->layout.num_tokens;
  LLP_CHECK(req->reduction >= LLP_REDUCE_TOKEN_MEAN && req->reduction <= LLP_REDUCE_SUM,
            LLP_ERR_INVALID_ARGUMENT, "reduction %d is unknown", req->reduction);
  LLP_CHECK(req->clip_low >= 0.0 && req->clip_low <= 1.0, LLP_ERR_INVALID_ARGUMENT,
            "clip_low must be in [0, 1]");
  LLP_CHECK(req->clip_high >= 0.0 && isfinite(req->clip_high), LLP_ERR_INVALID_ARGUMENT,
            "clip_high must be finite and >= 0");
  LLP_CHECK(req->dual_clip == 0.0 || (req->dual_clip > 1.0 && isfinite(req->dual_clip)),
            LLP_ERR_INVALID_ARGUMENT, "dual_clip must be 0 or > 1");
  LLP_CHECK(isfinite(req->kl_coef) && isfinite(req->entropy_coef), LLP_ERR_INVALID_ARGUMENT,
            "kl_coef and entropy_coef must be finite");
  if (req->ref_logp != nullptr)
    LLP_CHECK(req->kl_kind >= LLP_KL_K1 && req->kl_kind <= LLP_KL_K3, LLP_ERR_INVALID_ARGUMENT,
              "kl_kind %d is unknown", req->kl_kind);
  else if (T > 0)
    LLP_CHECK(req->kl_coef == 0.0, LLP_ERR_INVALID_ARGUMENT, "kl_coef needs ref_logp");
  if (req->entropy == nullptr && T > 0)
    LLP_CHECK(req->entropy_coef == 0.0, LLP_ERR_INVALID_ARGUMENT, "entropy_coef needs entropy");
  if (T > 0)
    LLP_CHECK(req->logp && req->old_logp && req->advantages, LLP_ERR_INVALID_ARGUMENT,
              "logp, old_logp and advantages are required");
  if (req->reduction == LLP_REDUCE_SEQ_MEAN) {
    LLP_CHECK(req->layout.cu_seqlens != nullptr, LLP_ERR_INVALID_ARGUMENT,
              "LLP_REDUCE_SEQ_MEAN needs cu_seqlens");
    LLP_CHECK(req->layout.num_seqs > 0 || T == 0, LLP_ERR_INVALID_ARGUMENT,
              "rows without a sequence (num_seqs = 0)");
  }
  if (req->reduction == LLP_REDUCE_SUM)
    LLP_CHECK(req->denominator == nullptr, LLP_ERR_INVALID_ARGUMENT,
              "a sum takes no denominator");
  return LLP_OK;
}

struct PolicyWs {
  size_t count, meta, looks, part, total;
  int32_t ncount, nblocks;
};

PolicyWs policy_ws(const llp_policy_request& r) {
  PolicyWs w{};
  const int64_t T = r.layout.num_tokens;
  const bool by_seq = r.reduction == LLP_REDUCE_SEQ_MEAN;
  if (T <= POLICY_SOLO_ROWS && !(by_seq && r.layout.num_seqs > POLICY_SOLO_SEQS))
    return w;   // one workgroup, no workspace
  if (by_seq) w.ncount = r.layout.num_seqs;
  else if (r.reduction == LLP_REDUCE_TOKEN_MEAN && r.layout.loss_mask && !r.denominator)
    w.ncount = (int32_t)((T + POLICY_COUNT_ROWS - 1) / POLICY_COUNT_ROWS);
  int64_t nb = (T + POLICY_BLOCK_ROWS - 1) / POLICY_BLOCK_ROWS;
  if (nb < 1) nb = 1;   // no rows in many sequences
  w.nblocks = (int32_t)(nb < POLICY_BLOCKS ? nb : POLICY_BLOCKS);
  Regions g;
  w.count = g.take((size_t)w.ncount * 4);
  w.meta = g.take(4);
  w.looks = g.take(LAYOUT_LOOKS * 4);
  w.part = g.take((size_t)w.nblocks * LLP_POLICY_STATS * 8);
  w.total = g.off;
  return w;
}

llp_status check_pref(const llp_pref_request* req) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  llp_status st = check_loss_layout(req->layout);
  if (st != LLP_OK) return st;
  const int64_t T = req->layout.num_tokens;
  LLP_CHECK(req->layout.cu_seqlens != nullptr, LLP_ERR_INVALID_ARGUMENT, "cu_seqlens is required");
  LLP_CHECK(req->layout.num_seqs % 2 == 0, LLP_ERR_INVALID_ARGUMENT, "num_seqs %d is not twice a number of pairs",
            req->layout.num_seqs);
  LLP_CHECK(req->layout.num_seqs > 0 || T == 0, LLP_ERR_INVALID_ARGUMENT,
            "rows without a sequence (num_seqs = 0)");
  LLP_CHECK(T == 0 || req->logp != nullptr, LLP_ERR_INVALID_ARGUMENT, "logp is NULL");
  LLP_CHECK(req->kind >= LLP_PREF_SIGMOID && req->kind <= LLP_PREF_IPO, LLP_ERR_INVALID_ARGUMENT,
            "kind %d is unknown", req->kind);
  LLP_CHECK(req->reduction == LLP_REDUCE_TOKEN_MEAN || req->reduction == LLP_REDUCE_SUM,
            LLP_ERR_INVALID_ARGUMENT, "reduction %d is not the mean over pairs or the sum",
            req->reduction);
  LLP_CHECK(req->beta > 0.0 && isfinite(req->beta), LLP_ERR_INVALID_ARGUMENT,
            "beta must be finite and > 0");
  LLP_CHECK(isfinite(req->gamma) && (req->gamma == 0.0 || req->kind != LLP_PREF_IPO),
            LLP_ERR_INVALID_ARGUMENT, "gamma must be finite (and 0 for IPO)");
  LLP_CHECK(req->label_smoothing >= 0.0 && req->label_smoothing < 1.0 &&
                (req->label_smoothing == 0.0 || req->kind == LLP_PREF_SIGMOID),
            LLP_ERR_INVALID_ARGUMENT, "label_smoothing must be in [0, 1) (0 unless SIGMOID)");
  return LLP_OK;
}

struct PrefWs {
  size_t sum, cnt, coef, looks, total;
};

PrefWs pref_ws(const llp_pref_request& r) {
  PrefWs w{};
  if (r.layout.num_tokens <= PREF_SOLO_ROWS && r.layout.num_seqs <= 2 * PREF_SOLO_PAIRS)
    return w;   // one workgroup, no workspace
  Regions g;
  const size_t n = (size_t)r.layout.num_seqs;
  w.sum = g.take(n * PREF_SPLIT * 8);
  w.cnt = g.take(n * PREF_SPLIT * 4);
  w.coef = g.take(n * 4);
  w.looks = g.take(LAYOUT_LOOKS * 4);
  w.total = g.off;
  return w;
}

// ---- Embedding ------------------------------------------------------------------------------
llp_status check_embedding(const llp_embedding_request* req, bool backward) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  llp_status st = check_partition(req->vocab);
  if (st != LLP_OK) return st;
  const int64_t T = req->num_tokens, H = req->hidden_size;
  LLP_CHECK(T >= 0, LLP_ERR_INVALID_ARGUMENT, "num_tokens=%lld < 0", (long long)T);
  LLP_CHECK(T <= kMaxRows, LLP_ERR_UNSUPPORTED, "num_tokens %lld too large", (long long)T);
  LLP_CHECK(req->vocab.local_size <= kMaxRows, LLP_ERR_UNSUPPORTED,
            "local_size %lld exceeds 2^23 - 256", (long long)req->vocab.local_size);
  LLP_CHECK(H > 0, LLP_ERR_INVALID_ARGUMENT, "hidden_size must be > 0");
  LLP_CHECK(H % 8 == 0 && H <= (1 << 20), LLP_ERR_UNSUPPORTED,
            "hidden_size %lld must be a multiple of 8 (and <= 2^20)", (long long)H);
  LLP_CHECK(T == 0 || req->token_ids != nullptr, LLP_ERR_INVALID_ARGUMENT, "token_ids is NULL");
  LLP_CHECK(isfinite(req->scale), LLP_ERR_INVALID_ARGUMENT, "scale must be finite");
  LLP_CHECK((req->flags & ~uint32_t(backward ? LLP_FLAG_OVERWRITE_GRADS : 0)) == 0,
            LLP_ERR_INVALID_ARGUMENT, "unknown flags 0x%x", req->flags);
  return LLP_OK;
}

// A row operand [rows, H]: dtype, stride and alignment (its pointer may be NULL without rows).
llp_status check_rows(const char* name, const void* p, int32_t dtype, int64_t stride, int64_t H,
                      bool needed) {
  LLP_CHECK(dtype == LLP_DTYPE_BF16 || dtype == LLP_DTYPE_F32, LLP_ERR_INVALID_ARGUMENT,
            "%s dtype %d is not BF16 or F32", name, dtype);
  LLP_CHECK(stride >= H && stride % 8 == 0, LLP_ERR_INVALID_ARGUMENT,
            "%s stride %lld must be >= hidden_size and a multiple of 8", name, (long long)stride);
  LLP_CHECK(stride < (int64_t(1) << 40), LLP_ERR_UNSUPPORTED, "%s stride %lld too large", name,
            (long long)stride);
  LLP_CHECK(!needed || (p != nullptr && aligned(p, 16)), LLP_ERR_INVALID_ARGUMENT,
            "%s must be non-NULL and 16-byte aligned", name);
  return LLP_OK;
}

struct EmbWs {
  size_t loc, start, order, row, span, part, total;
};

EmbWs embedding_ws(const llp_embedding_request& r) {
  EmbWs w{};
  Regions g;
  const int64_t T = r.num_tokens, units = (T + emb_unit(T) - 1) / emb_unit(T);
  w.loc = g.take((size_t)T * 4);
  w.start = g.take((size_t)(local_real(r.vocab) + 1) * 4);
  w.order = g.take((size_t)T * 4);
  w.row = g.take((size_t)T * 4);
  w.span = g.take((size_t)units * 4);
  w.part = g.take((size_t)units * 2 * (size_t)r.hidden_size * 4);
  w.total = g.off;
  return w;
}

}  // namespace

extern "C" {

LLP_API llp_status llp_quantize_rows(const llp_quant_request* req, void* stream) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  LLP_CHECK(req->rows >= 0 && req->rows < (int64_t(1) << 31), LLP_ERR_INVALID_ARGUMENT,
            "rows=%lld out of range", (long long)req->rows);
  LLP_CHECK(req->cols >= 1 && req->cols <= (1 << 20), LLP_ERR_INVALID_ARGUMENT,
            "cols=%lld outside [1, 2^20]", (long long)req->cols);
  LLP_CHECK(req->x_dtype == LLP_DTYPE_BF16 || req->x_dtype == LLP_DTYPE_F32,
            LLP_ERR_INVALID_ARGUMENT, "x_dtype %d is not BF16 or F32", req->x_dtype);
  const int64_t colsp = round_up(req->cols, LLP_INT8_COLUMNS);
  LLP_CHECK(req->x_stride >= req->cols && req->x_stride < (int64_t(1) << 40),
            LLP_ERR_INVALID_ARGUMENT, "x_stride %lld must be >= cols", (long long)req->x_stride);
  LLP_CHECK(req->q_stride >= colsp && req->q_stride % 16 == 0 && req->q_stride < (int64_t(1) << 40),
            LLP_ERR_INVALID_ARGUMENT, "q_stride %lld must be >= %lld and a multiple of 16",
            (long long)req->q_stride, (long long)colsp);
  const size_t es = req->x_dtype == LLP_DTYPE_F32 ? 4 : 2;
  if (req->rows > 0) {
    LLP_CHECK(req->x && req->q && req->scale, LLP_ERR_INVALID_ARGUMENT, "x, q and scale are required");
    LLP_CHECK(aligned(req->x, es), LLP_ERR_INVALID_ARGUMENT, "x not aligned to its element type");
    LLP_CHECK(aligned(req->q, 16), LLP_ERR_INVALID_ARGUMENT, "q not 16-byte aligned");
  }
  llp_status st = check_device();
  if (st != LLP_OK) return st;
  if (req->rows == 0) return LLP_OK;
  QuantArgs a{};
  a.x = req->x;
  a.bf16 = req->x_dtype == LLP_DTYPE_BF16;
  a.ldx = req->x_stride;
  a.rows = req->rows;
  a.cols = (int32_t)req->cols;
  a.colsp = (int32_t)colsp;
  a.q = req->q;
  a.ldq = req->q_stride;
  a.scale = req->scale;
  LLP_HIP(launch_quant(a, static_cast<hipStream_t>(stream)), "quantise kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_int8_workspace_bytes(const llp_int8_request* req, size_t* bytes) {
  llp_status st = check_int8(req);
  if (st != LLP_OK) return st;
  LLP_CHECK(bytes != nullptr, LLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = ws_layout(req->layout.num_tokens, local_real(req->vocab), req->hidden_size,
                     LLP_OP_FORWARD).total;
  return LLP_OK;
}

LLP_API llp_status llp_forward_int8(const llp_int8_request* req, const llp_partials* out,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  llp_status st = check_int8(req);
  if (st != LLP_OK) return st;
  const int64_t T = req->layout.num_tokens;
  const bool want_ent = (req->flags & LLP_FLAG_WANT_ENTROPY) != 0;
  const Ws w = ws_layout(T, local_real(req->vocab), req->hidden_size, LLP_OP_FORWARD);
  st = check_forward_out(T, want_ent, out, w, workspace, workspace_bytes);
  if (st != LLP_OK) return st;
  int num_cus = 0;
  st = check_device(&num_cus);
  if (st != LLP_OK) return st;
  if (T == 0) return LLP_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const ForwardArgs f = forward_args(req->vocab, req->layout, req->target_ids, req->temperature,
                                     want_ent, req->status_word, w, out, workspace, num_cus);
  Fwd8Args a{};
  a.f = f.fa;
  a.f.W = reinterpret_cast<const uint16_t*>(req->weight);
  a.f.ldw = req->weight_stride / 2;
  a.f.h = reinterpret_cast<const uint16_t*>(req->hidden);
  a.f.ldh = req->hidden_stride / 2;
  a.f.bias = req->bias;
  a.f.bias_f32 = req->bias_dtype == LLP_DTYPE_F32;
  a.f.H = (int32_t)(req->hidden_size / 2);
  a.la = f.la;
  a.ca = f.ca;
  a.hs = req->hidden_scale;
  a.ws = req->weight_scale;
  if (T <= FEW_ROWS) {
    LLP_HIP(launch_fwd8_few(a, s), "few-row forward kernel launch");
    return LLP_OK;
  }
  LLP_HIP(launch_layout(f.la, s), "layout kernel launch");
  LLP_HIP(launch_fwd8(a, s), "forward kernel launch");
  LLP_HIP(launch_combine(f.ca, w.T_cap, s), "combine kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_policy_workspace_bytes(const llp_policy_request* req, size_t* bytes) {
  llp_status st = check_policy(req);
  if (st != LLP_OK) return st;
  LLP_CHECK(bytes != nullptr, LLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = policy_ws(*req).total;
  return LLP_OK;
}

LLP_API llp_status llp_policy_loss(const llp_policy_request* req, const llp_policy_out* out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  llp_status st = check_policy(req);
  if (st != LLP_OK) return st;
  LLP_CHECK(out != nullptr && out->loss != nullptr, LLP_ERR_INVALID_ARGUMENT, "out.loss is required");
  LLP_CHECK(out->dentropy == nullptr || req->entropy != nullptr || req->layout.num_tokens == 0,
            LLP_ERR_INVALID_ARGUMENT, "out.dentropy needs entropy");
  const PolicyWs w = policy_ws(*req);
  st = check_workspace(workspace, workspace_bytes, w.total);
  if (st != LLP_OK) return st;
  st = check_device();
  if (st != LLP_OK) return st;
  PolicyArgs a{};
  a.T = req->layout.num_tokens;
  a.logp = req->logp;
  a.old = req->old_logp;
  a.adv = req->advantages;
  a.ref = req->ref_logp;
  a.ent = req->entropy;
  a.mask = req->layout.loss_mask;
  a.cu = req->layout.cu_seqlens;
  a.S = req->layout.num_seqs;
  a.log_lo = log1p(-req->clip_low);
  a.log_hi = log1p(req->clip_high);
  a.log_dual = req->dual_clip > 0.0 ? log(req->dual_clip) : INFINITY;
  a.lo = (float)(1.0 - req->clip_low);
  a.hi = (float)(1.0 + req->clip_high);
  a.dual = (float)req->dual_clip;
  a.klc64 = req->kl_coef;
  a.entc64 = req->entropy_coef;
  a.kl_kind = req->kl_kind;
  a.reduction = req->reduction;
  a.denom = req->denominator;
  a.nblocks = w.nblocks;
  a.ncount = w.ncount;
  a.count = at<int32_t>(workspace, w.count);
  a.meta = at<int32_t>(workspace, w.meta);
  a.looks = at<int32_t>(workspace, w.looks);
  a.first = req->reduction == LLP_REDUCE_SEQ_MEAN && layout_first(req->layout);
  a.part = at<double>(workspace, w.part);
  a.loss = out->loss;
  a.stats = out->stats;
  a.dloss = out->dloss;
  a.dlogp = out->dlogp;
  a.dent = out->dentropy;
  a.status = req->status_word;
  LLP_HIP(launch_policy(a, static_cast<hipStream_t>(stream)), "policy loss kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_preference_workspace_bytes(const llp_pref_request* req, size_t* bytes) {
  llp_status st = check_pref(req);
  if (st != LLP_OK) return st;
  LLP_CHECK(bytes != nullptr, LLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = pref_ws(*req).total;
  return LLP_OK;
}

LLP_API llp_status llp_preference_loss(const llp_pref_request* req, const llp_pref_out* out,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  llp_status st = check_pref(req);
  if (st != LLP_OK) return st;
  LLP_CHECK(out != nullptr && out->loss != nullptr, LLP_ERR_INVALID_ARGUMENT, "out.loss is required");
  const PrefWs w = pref_ws(*req);
  st = check_workspace(workspace, workspace_bytes, w.total);
  if (st != LLP_OK) return st;
  st = check_device();
  if (st != LLP_OK) return st;
  PrefArgs a{};
  a.T = req->layout.num_tokens;
  a.logp = req->logp;
  a.ref = req->ref_logp;
  a.weight = req->pair_weight;
  a.mask = req->layout.loss_mask;
  a.cu = req->layout.cu_seqlens;
  a.P = req->layout.num_seqs / 2;
  a.beta = req->beta;
  a.gamma = req->gamma;
  a.smooth = req->label_smoothing;
  a.kind = req->kind;
  a.average = req->average != 0;
  a.mean = req->reduction == LLP_REDUCE_TOKEN_MEAN;
  a.solo = w.total == 0;
  a.sum = at<double>(workspace, w.sum);
  a.cnt = at<int32_t>(workspace, w.cnt);
  a.coef = at<float>(workspace, w.coef);
  a.looks = at<int32_t>(workspace, w.looks);
  a.first = layout_first(req->layout);
  a.loss = out->loss;
  a.pair_loss = out->pair_loss;
  a.chosen = out->chosen;
  a.rejected = out->rejected;
  a.dloss = out->dloss;
  a.dlogp = out->dlogp;
  a.status = req->status_word;
  LLP_HIP(launch_preference(a, static_cast<hipStream_t>(stream)), "preference loss kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_embedding(const llp_embedding_request* req, const void* weight,
                                 int32_t weight_dtype, int64_t weight_stride, void* out,
                                 int64_t out_stride, void* stream) {
  llp_status st = check_embedding(req, false);
  if (st != LLP_OK) return st;
  const int64_t T = req->num_tokens, H = req->hidden_size, n_real = local_real(req->vocab);
  st = check_rows("weight", weight, weight_dtype, weight_stride, H, T > 0 && n_real > 0);
  if (st != LLP_OK) return st;
  st = check_rows("out", out, weight_dtype, out_stride, H, T > 0);
  if (st != LLP_OK) return st;
  st = check_device();
  if (st != LLP_OK) return st;
  if (T == 0) return LLP_OK;
  EmbArgs a{};
  a.ids = req->token_ids;
  a.mask = req->token_mask;
  a.T = T;
  a.offset = req->vocab.offset;
  a.n_real = n_real;
  a.real_vocab = req->vocab.real_vocab;
  a.H = (int32_t)H;
  a.scale = req->scale;
  a.W = weight;
  a.bf16 = weight_dtype == LLP_DTYPE_BF16;
  a.ldw = weight_stride;
  a.out = out;
  a.ldo = out_stride;
  a.status = req->status_word;
  LLP_HIP(launch_embedding(a, static_cast<hipStream_t>(stream)), "embedding kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_embedding_workspace_bytes(const llp_embedding_request* req, size_t* bytes) {
  llp_status st = check_embedding(req, true);
  if (st != LLP_OK) return st;
  LLP_CHECK(bytes != nullptr, LLP_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = embedding_ws(*req).total;
  return LLP_OK;
}

LLP_API llp_status llp_embedding_backward(const llp_embedding_request* req, const void* dout,
                                          int32_t dout_dtype, int64_t dout_stride, float* dweight,
                                          int64_t dweight_stride, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  llp_status st = check_embedding(req, true);
  if (st != LLP_OK) return st;
  const int64_t T = req->num_tokens, H = req->hidden_size;
  st = check_rows("dout", dout, dout_dtype, dout_stride, H, T > 0);
  if (st != LLP_OK) return st;
  st = check_rows("dweight", dweight, LLP_DTYPE_F32, dweight_stride, H, req->vocab.local_size > 0);
  if (st != LLP_OK) return st;
  const EmbWs w = embedding_ws(*req);
  st = check_workspace(workspace, workspace_bytes, w.total);
  if (st != LLP_OK) return st;
  st = check_device();
  if (st != LLP_OK) return st;
  EmbBwdArgs a{};
  a.ids = req->token_ids;
  a.mask = req->token_mask;
  a.T = T;
  a.offset = req->vocab.offset;
  a.n_real = local_real(req->vocab);
  a.real_vocab = req->vocab.real_vocab;
  a.local_size = req->vocab.local_size;
  a.H = (int32_t)H;
  // One group of local rows per compute unit, within what the sort's counters hold.
  const int64_t R = (a.n_real + 255) / 256;
  a.rows_per_group = (int32_t)(R < 1 ? 1 : R > EMB_ROWS_MAX ? EMB_ROWS_MAX : R);
  a.unit = emb_unit(T);
  a.scale = req->scale;
  a.overwrite = (req->flags & LLP_FLAG_OVERWRITE_GRADS) != 0;
  a.dout = dout;
  a.bf16 = dout_dtype == LLP_DTYPE_BF16;
  a.ldo = dout_stride;
  a.dW = dweight;
  a.ldw = dweight_stride;
  a.loc = at<int32_t>(workspace, w.loc);
  a.start = at<int32_t>(workspace, w.start);
  a.order = at<int32_t>(workspace, w.order);
  a.row = at<int32_t>(workspace, w.row);
  a.span = at<int32_t>(workspace, w.span);
  a.part = at<float>(workspace, w.part);
  a.status = req->status_word;
  hipStream_t s = static_cast<hipStream_t>(stream);
  LLP_HIP(launch_embedding_sort(a, s), "embedding sort kernel launch");
  LLP_HIP(launch_embedding_sum(a, s), "embedding gradient kernel launch");
  return LLP_OK;
}

}  // extern "C"
