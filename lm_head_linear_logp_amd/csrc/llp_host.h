// llp_host.h -- host-side helpers shared by the C-ABI entry points (llp_api.cpp,
// llp_api_ops.cpp): status reporting, request checks, the forward's workspace layout and
// kernel arguments. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "llp.h"
#include "llp_internal.h"

namespace llp {

// Records the calling thread's error message and returns `st`.
llp_status fail(llp_status st, const char* fmt, ...);

#define LLP_CHECK(cond, st, ...) \
  do {                           \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

llp_status check_partition(const llp_vocab_partition& v);
// The current device must have been opened; `num_cus` (optional) receives its compute units.
llp_status check_device(int* num_cus = nullptr);
llp_status hip_status(hipError_t e, const char* what);

#define LLP_HIP(expr, what)                         \
  do {                                              \
    llp_status s_ = hip_status((expr), (what));     \
    if (s_ != LLP_OK) return s_;                    \
  } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

inline int64_t local_real(const llp_vocab_partition& v) {
  int64_t n = v.real_vocab - v.offset;
  if (n < 0) n = 0;
  if (n > v.local_size) n = v.local_size;
  return n;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Byte offsets of workspace regions, each 256-byte aligned.
struct Regions {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += (size_t)round_up((int64_t)(bytes > 0 ? bytes : 1), 256);
    return o;
  }
};

// Workspace regions (byte offsets, each 256-byte aligned).
struct Ws {
  size_t count, qctr, scored, pos, tloc, tz, pm, ps, pq, G, hgT, P, dbp, total;
  int64_t T_cap, nvt, ldg;
  int64_t slab_tiles, nslab;   // vocabulary tiles per slab of G and slabs per backward call
};

// `slabs` (backward only): G is held one vocabulary slab of G_SLAB_TILES tiles at a time, so
// its region (and the bias-gradient partials) take one slab's columns, ldg = the slab width.
Ws ws_layout(int64_t T, int64_t n_real, int64_t H, int op, bool slabs = false);

// The forward's outputs and workspace, checked as every forward call does before a launch.
llp_status check_forward_out(int64_t T, bool want_ent, const llp_partials* out, const Ws& w,
                             const void* workspace, size_t workspace_bytes);

// The forward's launches over a workspace, but for what describes the operands.
struct ForwardArgs {
  LayoutArgs la{};
  FwdArgs fa{};
  CombineArgs ca{};
};

inline ForwardArgs forward_args(const llp_vocab_partition& vocab, const llp_token_layout& layout,
                                const int64_t* target_ids, float temperature, bool want_ent,
                                int32_t* status_word, const Ws& w, const llp_partials* out,
                                void* workspace, int num_cus) {
  float* ent = want_ent ? out->entropy : nullptr;
  ForwardArgs f;
  LayoutArgs& la = f.la;
  la.T = layout.num_tokens;
  la.mask = layout.loss_mask;
  la.cu_seqlens = layout.cu_seqlens;
  la.num_seqs = layout.num_seqs;
  la.world = vocab.world;
  la.targets = target_ids;
  la.offset = vocab.offset;
  la.n_real = local_real(vocab);
  la.real_vocab = vocab.real_vocab;
  la.count = at<int32_t>(workspace, w.count);
  la.scored = at<int32_t>(workspace, w.scored);
  la.pos = at<int32_t>(workspace, w.pos);
  la.tloc = at<int32_t>(workspace, w.tloc);
  la.out_t = out->target_logit;
  la.out_f = out->in_range;
  la.out_l = out->lse;
  la.out_e = ent;
  la.out_p = out->logp;
  la.status = status_word;
  la.qctr = at<int32_t>(workspace, w.qctr);   // the forward kernel's tile-queue counters
  la.nqctr = QCTR_INTS;

  FwdArgs& fa = f.fa;
  fa.n_real = la.n_real;
  fa.nvt = (int32_t)w.nvt;
  fa.ntb = (int32_t)(w.T_cap / TILE);
  fa.c1 = (float)(1.0 / (double)temperature);
  fa.count = la.count;
  fa.scored = la.scored;
  fa.tloc = la.tloc;
  fa.pm = at<float>(workspace, w.pm);
  fa.ps = at<float>(workspace, w.ps);
  fa.pq = at<float>(workspace, w.pq);
  fa.tz = at<float>(workspace, w.tz);
  fa.pstride = w.T_cap;
  fa.qctr = la.qctr;
  fa.workers = num_cus;

  CombineArgs& ca = f.ca;
  ca.nvt = (int32_t)w.nvt;
  ca.rows = layout.num_tokens;
  ca.pstride = w.T_cap;
  ca.count = la.count;
  ca.scored = la.scored;
  ca.tloc = la.tloc;
  ca.pm = fa.pm;
  ca.ps = fa.ps;
  ca.pq = fa.pq;
  ca.tz = fa.tz;
  ca.out_t = out->target_logit;
  ca.out_f = out->in_range;
  ca.out_l = out->lse;
  ca.out_e = ent;
  ca.out_p = out->logp;
  return f;
}

}  // namespace llp
