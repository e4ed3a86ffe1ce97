// reorder_launches.cpp -- the launches that llp_beam_reorder makes, recorded by a stand-in launcher: each
// holds fewer than 2^32 threads, and together they take every state once, in order.
#include <stdio.h>

#include <vector>

#include "llp.h"
#include "llp_internal.h"

namespace {
int g_failed = 0;
std::vector<void*> g_taken;
long long g_most = 0;
}  // namespace

namespace llp {
hipError_t launch_quant8(const Quant8Args&, hipStream_t) { return hipSuccess; }
hipError_t launch_quant8_both(const Quant8Args&, const Quant8Args&, hipStream_t) { return hipSuccess; }
hipError_t launch_linear8(const Linear8Args&, hipStream_t) { return hipSuccess; }
hipError_t launch_beam_candidates(const BeamArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_beam_select(const BeamSelectArgs&, hipStream_t) { return hipSuccess; }
// The kernel's grid: 256 threads for every 256 units of a sequence's pieces, for each sequence and state.
hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t) {
  const long long per = (a.outer * (a.inner / a.unit) + 255) / 256;
  const long long threads = per * a.seqs * a.states * 256;
  if (threads > g_most) g_most = threads;
  for (int i = 0; i < a.states; ++i) g_taken.push_back(a.dst[i]);
  return threads < (1LL << 32) && a.states >= 1 && a.states <= REORDER_STATES ? hipSuccess : hipErrorInvalidConfiguration;
}
}  // namespace llp

namespace {
void reorder(int states, int64_t seqs, int beams, int64_t outer, int64_t inner, llp_status want) {
  llp_beam_reorder_request r = {};
  r.num_states = states; r.num_seqs = seqs; r.num_src = r.num_out = beams; r.outer = outer; r.inner = inner;
  r.src_outer_stride = r.dst_outer_stride = inner;
  r.src_row_stride = r.dst_row_stride = outer * inner;
  // Nothing is read or written: addresses that are apart, aligned like `inner`.
  std::vector<void*> d;
  std::vector<const void*> s;
  for (int i = 0; i < states; ++i) {
    d.push_back(reinterpret_cast<void*>((uintptr_t)1 << 48 | (uintptr_t)i << 38));
    s.push_back(d.back());
  }
  int32_t parents = 0;
  r.src = s.data(); r.dst = d.data(); r.parents = &parents;
  g_taken.clear();
  const llp_status got = llp_beam_reorder(&r, nullptr);
  if (got != want || (want == LLP_OK && g_taken != d)) {
    ++g_failed;
    printf("%d states, %lld sequences of %d, %lld x %lld bytes: status %d (%s), %d states taken\n", states,
           (long long)seqs, beams, (long long)outer, (long long)inner, (int)got, llp_last_error(), (int)g_taken.size());
  }
}
}  // namespace

int main() {
  if (llp_open(0, nullptr) != LLP_OK) return 2;
  // Grids of a state that divide 2^24 workgroups evenly, and their neighbours.
  for (int states : {1, 2, 3, 16, 63, 64, 65, 128, 200})
    for (int shift = 0; shift < 24; ++shift)
      for (int64_t groups : {(int64_t(1) << shift) - 1, int64_t(1) << shift, (int64_t(1) << shift) + 1}) {
        if (groups < 1) continue;
        reorder(states, 1, 2, 1, groups * 256 * 16, LLP_OK);   // 16 bytes a thread
        reorder(states, 1, 2, 1, groups * 256 - 255, LLP_OK);  // a byte a thread
        if (groups % 3 == 0) reorder(states, groups / 3, 4, 3, 256 * 16, LLP_OK);
      }
  reorder(64, 64, 2, 8, 8192 * 128 * 2, LLP_OK);   // 64 layers' keys of 64 sequences, long prefixes
  reorder(64, 1024, 2, 1, 65535, LLP_OK);
  reorder(1, 1, 2, 1, (int64_t(1) << 24) * 256 * 16, LLP_ERR_UNSUPPORTED);
  reorder(3, 2, 2, 1, (int64_t(1) << 23) * 256 * 16, LLP_ERR_UNSUPPORTED);
  printf("%d failed, %lld threads at most\n", g_failed, g_most);
  return g_failed != 0;
}
