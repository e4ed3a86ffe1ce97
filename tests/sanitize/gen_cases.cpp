// gen_cases.cpp -- drives llp_api_gen.cpp under the host sanitizers: exactly sized buffers for
// well-formed calls over sizes and options, and malformed calls that must be refused.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "llp.h"

extern "C" int64_t llp_stub_gen();

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
int64_t span(int64_t n, int64_t ld, int64_t cols) { return n > 0 && cols > 0 ? (n - 1) * ld + cols : 0; }

void quant(int64_t R, int64_t K, int32_t dt, int block, int tr) {
  const int64_t M = tr ? K : R, D = tr ? R : K, G = (D + 127) / 128;
  llp_fp8_quant_request r = {};
  r.x = mem(span(R, K + 3, K) * (dt == LLP_DTYPE_F32 ? 4 : 2));
  r.x_dtype = dt; r.x_stride = K + 3; r.rows = R; r.cols = K; r.block_rows = block; r.transpose = tr;
  r.q_stride = G * 128 + 16; r.q = arr<uint8_t>(span(M, r.q_stride, G * 128));
  const int64_t n = block == 1 ? G : (M + 127) / 128, w = block == 1 ? M : G;
  r.scale_stride = w + 1; r.scale = arr<float>(span(n, w + 1, w));
  check("quant", llp_quantize_blocks(&r, nullptr), LLP_OK);
  if (block == 1 && !tr) {
    llp_fp8_quant_request t = r;
    const int64_t Gr = (R + 127) / 128;
    t.block_rows = 128; t.transpose = 1; t.q_stride = Gr * 128; t.q = arr<uint8_t>(span(K, Gr * 128, Gr * 128));
    t.scale_stride = Gr; t.scale = arr<float>(span(G, Gr, Gr));
    check("both", llp_quantize_both(&r, &t, nullptr), LLP_OK);
    check("both swapped", llp_quantize_both(&t, &r, nullptr), LLP_ERR_INVALID_ARGUMENT);
    t.x_stride += 1;
    check("both apart", llp_quantize_both(&r, &t, nullptr), LLP_ERR_INVALID_ARGUMENT);
  }
  done();
}

void linear(int64_t T, int64_t V, int64_t K, int32_t out, int bias, bool grad, uint32_t flags) {
  llp_fp8_linear_request r = {};
  r.rows = T; r.cols = V; r.depth = K; r.flags = flags; r.out_dtype = out;
  r.x_stride = K + 16; r.x = arr<uint8_t>(span(T, r.x_stride, K));
  r.weight_stride = K + 32; r.weight = arr<uint8_t>(span(V, r.weight_stride, K));
  r.x_scale_stride = T + 1; r.x_scale = arr<float>(span(K / 128, T + 1, T));
  r.weight_scale_stride = K / 128 + 2; r.weight_scale = arr<float>(span((V + 127) / 128, K / 128 + 2, K / 128));
  if (bias) { r.bias = mem(V * (bias == LLP_DTYPE_F32 ? 4 : 2)); r.bias_dtype = bias; }
  const int64_t n = grad ? V : T, w = grad ? T : V;
  r.out_stride = w + 1; r.out = mem(span(n, w + 1, w) * (out == LLP_DTYPE_F32 ? 4 : 2));
  check("linear", (grad ? llp_dweight_fp8 : llp_linear_fp8)(&r, nullptr), LLP_OK);
  r.x_stride = 24;
  check("linear stride", (grad ? llp_dweight_fp8 : llp_linear_fp8)(&r, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void candidates(int64_t R, int64_t local, int64_t real, int num, int32_t dt) {
  llp_beam_request r = {};
  const int64_t n = real < local ? real : local;
  r.vocab.local_size = local; r.vocab.real_vocab = real > 0 ? real : 1; r.vocab.padded_vocab = local + (real > 0 ? 0 : 8);
  r.vocab.world = 1;
  if (real <= 0) { r.vocab.world = 2; r.vocab.rank = 1; r.vocab.offset = 8; }
  r.num = num; r.num_rows = R; r.logits_dtype = dt; r.temperature = 0.7f;
  r.logits_stride = (local + 15) / 8 * 8;
  r.logits = n > 0 ? mem(span(R, r.logits_stride, n) * (dt == LLP_DTYPE_F32 ? 4 : 2)) : nullptr;
  r.status_word = arr<int32_t>(1);
  llp_beam_parts o = {arr<float>(R * num), arr<int64_t>(R * num), arr<float>(R), arr<double>(R)};
  check("candidates", llp_beam_candidates(&r, &o, nullptr), LLP_OK);
  r.num = LLP_MAX_BEAMS + 1;
  check("candidates num", llp_beam_candidates(&r, &o, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void select(int64_t B, int K, int num, int out, int world, bool fin) {
  std::vector<llp_beam_parts> p;
  for (int i = 0; i < world; ++i)
    p.push_back({arr<float>(B * K * num), arr<int64_t>(B * K * num), arr<float>(B * K), arr<double>(B * K)});
  llp_beam_select_request r = {};
  r.world = world; r.num = num; r.parts = p.data(); r.num_seqs = B; r.num_beams = K; r.num_out = out;
  r.scores = arr<float>(B * K); r.finished = fin ? arr<uint8_t>(B * K) : nullptr; r.temperature = 1.f;
  r.status_word = arr<int32_t>(1);
  llp_beam_out o = {arr<int64_t>(B * out), arr<int32_t>(B * out), arr<float>(B * out)};
  check("select", llp_beam_select(&r, &o, nullptr), LLP_OK);
  r.num_out = num + 1;
  check("select num_out", llp_beam_select(&r, &o, nullptr), LLP_ERR_INVALID_ARGUMENT);
  done();
}

void reorder(int n, int64_t B, int K, int N, int64_t outer, int64_t inner, bool place, int64_t shift) {
  llp_beam_reorder_request r = {};
  r.num_states = n; r.num_seqs = B; r.num_src = K; r.num_out = N; r.outer = outer; r.inner = inner;
  r.src_outer_stride = r.dst_outer_stride = inner + 48;
  r.src_row_stride = r.dst_row_stride = outer * (inner + 48) + 16;
  std::vector<const void*> s;
  std::vector<void*> d;
  for (int i = 0; i < n; ++i) {
    char* p = (char*)mem((B * K - 1) * r.src_row_stride + (outer - 1) * r.src_outer_stride + inner + shift) + shift;
    s.push_back(p);
    d.push_back(place ? p : (char*)mem((B * N - 1) * r.dst_row_stride + (outer - 1) * r.dst_outer_stride + inner));
  }
  r.src = s.data(); r.dst = d.data(); r.parents = arr<int32_t>(B * N); r.status_word = arr<int32_t>(1);
  check("reorder", llp_beam_reorder(&r, nullptr), LLP_OK);
  if (n > 1) {
    d[n - 1] = d[0];
    s[n - 1] = s[0];
    check("reorder twice", llp_beam_reorder(&r, nullptr), LLP_ERR_INVALID_ARGUMENT);
  }
  done();
}
}  // namespace

int main() {
  check("open", llp_open(0, nullptr), LLP_OK);
  for (int64_t R : {1, 127, 128, 129, 1000})
    for (int64_t K : {1, 128, 200, 4096})
      for (int b : {1, 128})
        for (int tr : {0, 1}) quant(R, K, K % 3 ? LLP_DTYPE_BF16 : LLP_DTYPE_F32, b, tr);
  quant(0, 5, LLP_DTYPE_F32, 1, 0);
  quant(5, 0, LLP_DTYPE_F32, 128, 1);
  for (int64_t T : {0, 1, 32, 33, 300, 4096})
    for (int64_t V : {0, 1, 129, 1000})
      for (int64_t K : {0, 128, 640}) {
        linear(T, V, K, LLP_DTYPE_F32, 0, false, 0);
        linear(T, V, K, LLP_DTYPE_BF16, LLP_DTYPE_BF16, false, 0);
        linear(T, V, K, LLP_DTYPE_F32, 0, true, 0);
        linear(T, V, K, LLP_DTYPE_BF16, 0, true, LLP_FLAG_OVERWRITE_GRADS);
      }
  for (int64_t R : {0, 1, 3, 700, 5000})
    for (int64_t V : {1, 2048, 2049, 37984})
      for (int num : {1, 16, 64}) candidates(R, V, V > 2 ? V - 1 : V, num, num == 16 ? LLP_DTYPE_BF16 : LLP_DTYPE_F32);
  candidates(4, 100, 0, 8, LLP_DTYPE_F32);
  for (int K : {1, 5, 64})
    for (int w : {1, 64}) select(3, K, 16, 10, w, w == 1);
  select(0, 4, 8, 8, 1, false);
  for (int n : {0, 1, 3, 70, 130})
    for (int64_t inner : {1, 6, 64, 4096})
      for (int K : {1, 4, 40}) {
        reorder(n, 3, K, K, 5, inner, true, 0);
        reorder(n, 2, K, K == 1 ? 4 : K - 1, 2, inner, false, inner == 6 ? 2 : 0);
      }
  printf("%d run, %d failed, %lld launches\n", g_run, g_failed, (long long)llp_stub_gen());
  return g_failed ? 1 : 0;
}
