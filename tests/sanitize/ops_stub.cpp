// ops_stub.cpp -- stand-in launchers, beside hip_stub.cpp, for the operators around the linear
// log-prob: each touches the first and last element of every array its kernels address.
#include <string.h>

#include "llp_internal.h"

namespace {
volatile unsigned char g_sink;
void touch(const void* p, size_t at) {
  volatile unsigned char* q = (volatile unsigned char*)p + at;
  const unsigned char v = *q;
  *q = v;
  g_sink = v;
}
template <class T>
void extent(const T* p, int64_t n) {
  if (p == nullptr || n <= 0) return;
  touch(p, 0);
  touch(p, (size_t)n * sizeof(T) - 1);
}
void rows(const void* p, int64_t n, int64_t ld, int64_t cols, int es) {
  if (p == nullptr || n <= 0 || cols <= 0) return;
  extent((const unsigned char*)p, ((n - 1) * ld + cols) * es);
}
int64_t g_ops = 0;
}  // namespace

extern "C" int64_t llp_stub_ops() { return g_ops; }

namespace llp {

hipError_t launch_quant(const QuantArgs& a, hipStream_t) {
  ++g_ops;
  rows(a.x, a.rows, a.ldx, a.cols, a.bf16 ? 2 : 4);
  rows(a.q, a.rows, a.ldq, a.colsp, 1);
  extent(a.scale, a.rows);
  return hipSuccess;
}
static void fwd8(const Fwd8Args& a, int64_t T) {
  ++g_ops;
  rows(a.f.W, a.f.n_real, a.f.ldw, a.f.H, 2);
  rows(a.f.h, T, a.f.ldh, a.f.H, 2);
  extent(a.hs, T);
  extent(a.ws, a.f.n_real);
  if (a.f.bias) extent((const unsigned char*)a.f.bias, a.f.n_real * (a.f.bias_f32 ? 4 : 2));
  for (const float* p : {a.f.pm, a.f.ps, a.f.pq}) extent(p, (int64_t)a.f.nvt * a.f.pstride);
  extent(a.f.tz, (int64_t)a.f.ntb * 256);
}
hipError_t launch_fwd8(const Fwd8Args& a, hipStream_t) {
  fwd8(a, a.la.T);
  extent(a.f.qctr, QCTR_INTS);
  return hipSuccess;
}
hipError_t launch_fwd8_few(const Fwd8Args& a, hipStream_t) {
  if (a.la.T > FEW_ROWS) return hipErrorInvalidValue;
  fwd8(a, a.la.T);
  extent(a.la.mask, a.la.T);
  extent(a.la.targets, a.la.T);
  if (a.la.cu_seqlens) extent(a.la.cu_seqlens, (int64_t)a.la.num_seqs + 1);
  extent(a.ca.out_t, a.la.T); extent(a.ca.out_f, a.la.T); extent(a.ca.out_l, a.la.T);
  extent(a.ca.out_e, a.la.T); extent(a.ca.out_p, a.la.T);
  extent(a.la.out_t, a.la.T); extent(a.la.out_e, a.la.T);
  extent(a.la.status, 1);
  return hipSuccess;
}
hipError_t launch_embedding(const EmbArgs& a, hipStream_t) {
  ++g_ops;
  extent(a.ids, a.T);
  extent(a.mask, a.T);
  rows(a.W, a.n_real, a.ldw, a.H, a.bf16 ? 2 : 4);
  rows(a.out, a.T, a.ldo, a.H, a.bf16 ? 2 : 4);
  return hipSuccess;
}
hipError_t launch_embedding_sort(const EmbBwdArgs& a, hipStream_t) {
  ++g_ops;
  if (a.rows_per_group < 1 || a.rows_per_group > EMB_ROWS_MAX) return hipErrorInvalidValue;
  extent(a.ids, a.T);
  extent(a.mask, a.T);
  extent(a.loc, a.T);
  extent(a.order, a.T);
  extent(a.row, a.T);
  extent(a.start, a.n_real + 1);
  extent(a.status, 1);
  return hipSuccess;
}
hipError_t launch_embedding_sum(const EmbBwdArgs& a, hipStream_t) {
  ++g_ops;
  const int64_t units = (a.T + a.unit - 1) / a.unit;
  extent(a.span, units);
  extent(a.part, units * 2 * a.H);
  rows(a.dout, a.T, a.ldo, a.H, a.bf16 ? 2 : 4);
  rows(a.dW, a.overwrite ? a.local_size : a.n_real, a.ldw, a.H, 4);
  return hipSuccess;
}
hipError_t launch_policy(const PolicyArgs& a, hipStream_t) {
  ++g_ops;
  for (const float* p : {a.logp, a.old, a.adv, a.ref, a.ent}) extent(p, a.T);
  extent(a.mask, a.T);
  if (a.cu) extent(a.cu, (int64_t)a.S + 1);
  if (a.nblocks > 0) {
    extent(a.count, a.ncount);
    extent(a.meta, 1);
    extent(a.part, (int64_t)a.nblocks * LLP_POLICY_STATS);
  } else if (a.T > POLICY_SOLO_ROWS || (a.reduction == LLP_REDUCE_SEQ_MEAN && a.S > POLICY_SOLO_SEQS)) {
    return hipErrorInvalidValue;
  }
  extent(a.loss, 1);
  extent(a.stats, LLP_POLICY_STATS);
  extent(a.dloss, 1);
  extent(a.dlogp, a.T);
  extent(a.dent, a.T);
  extent(a.denom, 1);
  return hipSuccess;
}
hipError_t launch_preference(const PrefArgs& a, hipStream_t) {
  ++g_ops;
  extent(a.logp, a.T); extent(a.ref, a.T); extent(a.mask, a.T);
  extent(a.cu, 2 * (int64_t)a.P + 1);
  extent(a.weight, a.P);
  if (!a.solo) {
    extent(a.sum, 2 * (int64_t)a.P * PREF_SPLIT);
    extent(a.cnt, 2 * (int64_t)a.P * PREF_SPLIT);
    extent(a.coef, 2 * (int64_t)a.P);
  } else if (a.P > PREF_SOLO_PAIRS || a.T > PREF_SOLO_ROWS) {
    return hipErrorInvalidValue;
  }
  extent(a.loss, 1);
  extent(a.pair_loss, a.P); extent(a.chosen, a.P); extent(a.rejected, a.P);
  extent(a.dlogp, a.T);
  return hipSuccess;
}

}  // namespace llp
