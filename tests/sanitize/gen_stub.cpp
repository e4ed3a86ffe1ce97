// gen_stub.cpp -- stand-in launchers, beside hip_stub.cpp, for the fp8 and beam-search operators: each
// touches the first and last element of every array its kernels address.
#include <string.h>

#include "llp_internal.h"

namespace {
volatile unsigned char g_sink;
void bytes(const void* p, int64_t n) {
  if (p == nullptr || n <= 0) return;
  for (int64_t at : {int64_t(0), n - 1}) {
    volatile unsigned char* q = (volatile unsigned char*)p + at;
    const unsigned char v = *q;
    *q = v;
    g_sink = v;
  }
}
template <class T>
void extent(const T* p, int64_t n) { bytes(p, n * (int64_t)sizeof(T)); }
void rows(const void* p, int64_t n, int64_t ld, int64_t cols, int es) {
  if (n > 0 && cols > 0) bytes(p, ((n - 1) * ld + cols) * es);
}
int64_t g_gen = 0;
}  // namespace

extern "C" int64_t llp_stub_gen() { return g_gen; }

namespace llp {

hipError_t launch_quant8(const Quant8Args& a, hipStream_t) {
  ++g_gen;
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  const int64_t M = a.transpose ? a.cols : a.rows, K = a.transpose ? a.rows : a.cols;
  const int64_t G = (K + 127) / 128;
  rows(a.x, a.rows, a.ldx, a.cols, a.bf16 ? 2 : 4);
  rows(a.q, M, a.ldq, G * 128, 1);
  if (a.block) rows(a.scale, (M + 127) / 128, a.lds, G, 4);
  else rows(a.scale, G, a.lds, M, 4);
  return hipSuccess;
}

hipError_t launch_quant8_both(const Quant8Args& a, const Quant8Args& t, hipStream_t s) {
  const hipError_t e = launch_quant8(a, s);
  --g_gen;
  return e != hipSuccess ? e : launch_quant8(t, s);
}

hipError_t launch_linear8(const Linear8Args& a, hipStream_t) {
  ++g_gen;
  const int64_t K = (int64_t)a.steps * 128;
  rows(a.x, a.T, a.ldx, K, 1);
  rows(a.W, a.V, a.ldw, K, 1);
  rows(a.xs, a.steps, a.ldxs, a.T, 4);
  rows(a.ws, (a.V + 127) / 128, a.ldws, a.steps, 4);
  if (a.bias) bytes(a.bias, a.V * (a.bias_f32 ? 4 : 2));
  if (a.grad) rows(a.out, a.V, a.ldo, a.T, a.out_bf16 ? 2 : 4);
  else rows(a.out, a.T, a.ldo, a.V, a.out_bf16 ? 2 : 4);
  return hipSuccess;
}

hipError_t launch_beam_candidates(const BeamArgs& a, hipStream_t) {
  ++g_gen;
  if (a.blocks > 0) rows(a.logits, a.rows, a.ld, a.n_real, a.bf16 ? 2 : 4);
  extent(a.value, a.rows * a.num);
  extent(a.token, a.rows * a.num);
  extent(a.max, a.rows);
  extent(a.sum, a.rows);
  extent(a.status, 1);
  return hipSuccess;
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t) {
  ++g_gen;
  const int64_t R = a.seqs * a.K;
  for (int r = 0; r < a.world && a.seqs > 0; ++r) {
    extent(a.value[r], R * a.num);
    extent(a.token[r], R * a.num);
    extent(a.max[r], R);
    extent(a.sum[r], R);
  }
  extent(a.scores, R);
  extent(a.finished, R);
  extent(a.out_token, a.seqs * a.num_out);
  extent(a.out_parent, a.seqs * a.num_out);
  extent(a.out_score, a.seqs * a.num_out);
  extent(a.status, 1);
  return hipSuccess;
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t) {
  ++g_gen;
  for (int i = 0; i < a.states; ++i) {
    if (a.inner % a.unit != 0 || (uintptr_t)a.src[i] % a.unit != 0 || (uintptr_t)a.dst[i] % a.unit != 0)
      return hipErrorInvalidValue;
    bytes(a.src[i], (a.seqs * a.K - 1) * a.sr + (a.outer - 1) * a.so + a.inner);
    bytes(a.dst[i], (a.seqs * a.N - 1) * a.dr + (a.outer - 1) * a.dout + a.inner);
  }
  extent(a.parents, a.seqs * a.N);
  extent(a.status, 1);
  return hipSuccess;
}

}  // namespace llp
