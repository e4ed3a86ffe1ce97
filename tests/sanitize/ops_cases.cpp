// ops_cases.cpp -- drives llp_api_ops.cpp under the host sanitizers: exactly sized buffers for
// well-formed calls over sizes and options, and malformed calls that must be refused.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "llp.h"

extern "C" int64_t llp_stub_ops();

namespace {
int g_run = 0, g_failed = 0;
std::vector<void*> g_mem;
void* mem(int64_t bytes) {  // exactly sized, 256-byte aligned start
  if (bytes <= 0) return nullptr;
  void* p = nullptr;
  if (posix_memalign(&p, 256, (size_t)bytes) != 0) abort();
  g_mem.push_back(p);
  return p;
}
template <class T>
T* arr(int64_t n) { return static_cast<T*>(mem(n * (int64_t)sizeof(T))); }
void done() {
  for (void* p : g_mem) free(p);
  g_mem.clear();
}
void check(const char* what, llp_status got, llp_status want) {
  ++g_run;
  if (got != want) {
    ++g_failed;
    printf("%s: status %d, expected %d (%s)\n", what, (int)got, (int)want, llp_last_error());
  }
}
llp_vocab_partition part(int64_t off, int64_t local, int64_t real, int64_t padded, int world) {
  llp_vocab_partition v;
  v.offset = off; v.local_size = local; v.real_vocab = real; v.padded_vocab = padded;
  v.rank = 0; v.world = world;
  return v;
}

void quant(int64_t R, int64_t K, int32_t dt) {
  const int64_t Kp = (K + 127) / 128 * 128, es = dt == LLP_DTYPE_F32 ? 4 : 2;
  llp_quant_request r = {};
  r.x = mem(((R - 1) * (K + 3) + K) * es);
  r.x_dtype = dt; r.x_stride = K + 3; r.rows = R; r.cols = K;
  r.q = arr<int8_t>((R - 1) * (Kp + 16) + Kp); r.q_stride = Kp + 16;
  r.scale = arr<float>(R);
  check("quant", llp_quantize_rows(&r, nullptr), LLP_OK);
  done();
}

void int8(int64_t T, int64_t K, const llp_vocab_partition& v, int bias, bool ent) {
  int64_t n = v.real_vocab - v.offset;
  n = n < 0 ? 0 : n > v.local_size ? v.local_size : n;
  llp_int8_request r = {};
  r.hidden = arr<int8_t>((T - 1) * (K + 32) + K); r.hidden_stride = K + 32; r.hidden_scale = arr<float>(T);
  r.weight = arr<int8_t>(n > 0 ? (n - 1) * (K + 16) + K : 0); r.weight_stride = K + 16;
  r.weight_scale = arr<float>(n);
  if (bias) { r.bias = mem(n * (bias == LLP_DTYPE_F32 ? 4 : 2)); r.bias_dtype = bias; }
  r.flags = ent ? LLP_FLAG_WANT_ENTROPY : 0;
  r.hidden_size = K; r.vocab = v; r.layout.num_tokens = T; r.layout.loss_mask = arr<uint8_t>(T);
  r.target_ids = arr<int64_t>(T); r.temperature = 0.7f;
  llp_partials o = {arr<float>(T), arr<uint8_t>(T), arr<float>(T), ent ? arr<float>(T) : nullptr, arr<float>(T)};
  size_t b = 0;
  check("int8 workspace", llp_int8_workspace_bytes(&r, &b), LLP_OK);
  void* ws = mem((int64_t)b);
  check("int8", llp_forward_int8(&r, &o, ws, b, nullptr), LLP_OK);
  check("int8 short workspace", llp_forward_int8(&r, &o, ws, b - 1, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void policy(int64_t T, int32_t S, int red, bool mask, bool full) {
  llp_policy_request r = {};
  r.logp = arr<float>(T); r.old_logp = arr<float>(T); r.advantages = arr<float>(T);
  if (full) { r.ref_logp = arr<float>(T); r.entropy = arr<float>(T); r.kl_coef = 0.1; r.entropy_coef = 0.1; }
  r.kl_kind = LLP_KL_K3; r.reduction = red; r.clip_low = 0.2; r.clip_high = 0.2;
  r.layout.num_tokens = T;
  if (mask) r.layout.loss_mask = arr<uint8_t>(T);
  if (S >= 0) { r.layout.num_seqs = S; r.layout.cu_seqlens = arr<int32_t>(S + 1); }
  llp_policy_out o = {arr<float>(1), arr<float>(LLP_POLICY_STATS), arr<float>(1), arr<float>(T), full ? arr<float>(T) : nullptr};
  size_t b = 0;
  check("policy workspace", llp_policy_workspace_bytes(&r, &b), LLP_OK);
  void* ws = mem((int64_t)b);
  check("policy", llp_policy_loss(&r, &o, ws, b, nullptr), LLP_OK);
  if (b > 0) check("policy short workspace", llp_policy_loss(&r, &o, ws, b - 1, nullptr), LLP_ERR_INVALID_ARGUMENT);
  o.loss = nullptr;
  check("policy without loss", llp_policy_loss(&r, &o, ws, b, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void pref(int64_t T, int32_t P) {
  llp_pref_request r = {};
  r.logp = arr<float>(T); r.ref_logp = arr<float>(T); r.pair_weight = arr<float>(P);
  r.layout.num_tokens = T; r.layout.num_seqs = 2 * P; r.layout.cu_seqlens = arr<int32_t>(2 * P + 1);
  r.beta = 0.1; r.kind = LLP_PREF_SIGMOID; r.reduction = LLP_REDUCE_SUM;
  llp_pref_out o = {arr<float>(1), arr<float>(P), arr<float>(P), arr<float>(P), nullptr, arr<float>(T)};
  size_t b = 0;
  check("pref workspace", llp_preference_workspace_bytes(&r, &b), LLP_OK);
  void* ws = mem((int64_t)b);
  check("pref", llp_preference_loss(&r, &o, ws, b, nullptr), LLP_OK);
  if (b > 0) check("pref short workspace", llp_preference_loss(&r, &o, ws, b - 1, nullptr), LLP_ERR_INVALID_ARGUMENT);
  r.layout.num_seqs = 2 * P + 1;
  check("pref odd sequences", llp_preference_loss(&r, &o, ws, b, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void embed(int64_t T, int64_t H, const llp_vocab_partition& v, int32_t dt, uint32_t flags) {
  const int64_t es = dt == LLP_DTYPE_F32 ? 4 : 2;
  int64_t n = v.real_vocab - v.offset;
  n = n < 0 ? 0 : n > v.local_size ? v.local_size : n;
  llp_embedding_request r = {};
  r.token_ids = arr<int64_t>(T); r.token_mask = arr<uint8_t>(T); r.num_tokens = T;
  r.vocab = v; r.hidden_size = H; r.scale = 2.f;
  const void* w = mem(n > 0 ? ((n - 1) * (H + 8) + H) * es : 0);
  void* out = mem(((T - 1) * (H + 16) + H) * es);
  check("embedding", llp_embedding(&r, w, dt, H + 8, out, H + 16, nullptr), LLP_OK);
  r.flags = flags;
  float* dw = arr<float>(v.local_size > 0 ? (v.local_size - 1) * (H + 8) + H : 0);
  size_t b = 0;
  check("embedding workspace", llp_embedding_workspace_bytes(&r, &b), LLP_OK);
  void* ws = mem((int64_t)b);
  check("embedding backward", llp_embedding_backward(&r, out, dt, H + 16, dw, H + 8, ws, b, nullptr), LLP_OK);
  check("embedding short workspace", llp_embedding_backward(&r, out, dt, H + 16, dw, H + 8, ws, b - 1, nullptr),
        LLP_ERR_INVALID_ARGUMENT);
  done();
}
}  // namespace

int main() {
  llp_info info;
  check("open", llp_open(0, &info), LLP_OK);
  for (int32_t dt : {LLP_DTYPE_BF16, LLP_DTYPE_F32})
    for (int64_t K : {1, 127, 128, 129, 4096}) quant(5, K, dt);
  const llp_vocab_partition vs[] = {part(0, 1000, 900, 1000, 1), part(600, 300, 900, 1000, 2),
                                    part(900, 100, 900, 1000, 2), part(0, 700000, 700000, 700000, 1)};
  for (const auto& v : vs)
    for (int64_t T : {1, 64, 65, 300})
      for (int bias : {0, (int)LLP_DTYPE_BF16, (int)LLP_DTYPE_F32})
        if (v.local_size <= 1000 || (bias == 0 && T <= 65)) int8(T, 128, v, bias, T != 64);
  for (int64_t T : {0, 1, 8192, 8193, 40000, 2000000})
    for (int red : {(int)LLP_REDUCE_TOKEN_MEAN, (int)LLP_REDUCE_SEQ_MEAN, (int)LLP_REDUCE_SUM})
      for (int32_t S : {1, 1024, 1025, 5000})
        for (bool m : {false, true}) policy(T, S, red, m, m);
  policy(100, -1, LLP_REDUCE_TOKEN_MEAN, true, true);
  for (int32_t P : {1, 128, 129, 3000})
    for (int64_t T : {1, 5000}) pref(T, P);
  pref(0, 0);
  for (const auto& v : vs)
    if (v.local_size <= 1000)
      for (int64_t T : {1, 16, 17, 4096, 4097, 20000})
        for (int32_t dt : {LLP_DTYPE_BF16, LLP_DTYPE_F32})
          for (uint32_t f : {0u, (uint32_t)LLP_FLAG_OVERWRITE_GRADS}) embed(T, 24, v, dt, f);
  printf("%d run, %d failed, %lld launches\n", g_run, g_failed, (long long)llp_stub_ops());
  return g_failed != 0 || llp_stub_ops() == 0;
}
