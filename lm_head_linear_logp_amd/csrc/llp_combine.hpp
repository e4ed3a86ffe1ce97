// llp_combine.hpp -- the cross-tile combine of one row's partials, shared by the kernels that end
// a forward.
#pragma once

#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

// ------------------------------------------------------------------------------------
// Cross-tile combine, in vocabulary-tile order: chain c of 16 folds tiles c, c+16, ... of a row,
// then the row's 16 chains are folded in order c = 0..15. A workgroup takes 32 rows x 16 chains
// (thread = chain * 32 + row), so the 4096 rows of a chunk spread over 128 workgroups; the
// arithmetic of a row does not depend on that grouping. With d_k = m_k - M:
// S = sum_k s_k e^{d_k}, Q = sum_k e^{d_k}(q_k + s_k d_k log2 e); lse = M + ln S and
// entropy = ln S - ln2 * Q / S. An empty shard gives lse = -inf, entropy 0, target logit 0,
// in_range 0 and logp -inf ([top-p replay, "Changes" table]: empty vocabulary rows).
// ------------------------------------------------------------------------------------
// Each rounding of a combine is written out, here and below, so that every kernel that combines
// gives the same bits however the compiler would contract its products.
// q + s d log2 e:
__device__ __forceinline__ float weighed(float q, float s, float d) { return fmaf(kLog2e, s * d, q); }

// Q = wa (Q + S da log2 e) + wb (q + s db log2 e) and S = wa S + wb s.
__device__ __forceinline__ void fold_sums(float& S, float& Q, float wa, float wb, float da, float db,
                                          float s, float q) {
  const float x = weighed(Q, S, da), y = weighed(q, s, db);
  Q = fmaf(wb, y, wa * x);
  S = fmaf(wb, s, wa * S);
}

__device__ __forceinline__ void fold(float& M, float& S, float& Q, float m, float s, float q) {
  // Combine (M, S, Q) with a partial (m, s, q); both may be empty (-inf max, zero sums).
  if (m == -INFINITY) return;
  if (M == -INFINITY) {
    M = m; S = s; Q = q;
    return;
  }
  const float N = fmaxf(M, m);
  const float da = M - N, db = m - N;
  fold_sums(S, Q, expf(da), expf(db), da, db, s, q);
  M = N;
}

// 32 rows: a wave's loads of one partial are 32 consecutive floats, a whole 128-byte line
// (with 16 rows two workgroups each fetched half of every line: 70 MB for 29 MB of partials).
constexpr int COMBINE_ROWS = 32, COMBINE_CHAINS = 16;

// One chain of a row: tiles c, c + 16, ... of nvt, `get(vt, m, s, q)` reading a tile's partial.
// Unrolled so that each thread has several independent loads in flight.
template <class Max, class Get>
__device__ __forceinline__ void combine_chain(int c, int nvt, Max max_of, Get get, float& M, float& S,
                                              float& Q) {
  float mmax = -INFINITY;
#pragma unroll 8
  for (int vt = c; vt < nvt; vt += COMBINE_CHAINS) mmax = fmaxf(mmax, max_of(vt));
  if (mmax != -INFINITY) {
#pragma unroll 8
    for (int vt = c; vt < nvt; vt += COMBINE_CHAINS) {
      float m, s, q;
      get(vt, m, s, q);
      const float d = m - mmax;
      const float e = expf(d);
      S = fmaf(e, s, S);
      Q = fmaf(e, weighed(q, s, d), Q);
    }
    M = mmax;
  }
}

// A row's finished sums to its outputs; `target` is its target's logit where there is a hit.
__device__ __forceinline__ void combine_out(const CombineArgs& a, int row, bool hit, float target, float M,
                                            float S, float Q) {
  float lse, ent;
  if (M == -INFINITY || !(S > 0.f)) {
    lse = -INFINITY;
    ent = 0.f;
  } else {
    const float ls = logf(S);
    lse = M + ls;
    ent = fmaf(-kLn2, Q / S, ls);
  }
  const float tz = hit ? target : 0.f;
  a.out_t[row] = tz;
  a.out_f[row] = hit ? 1 : 0;
  a.out_l[row] = lse;
  if (a.out_e) a.out_e[row] = ent;
  if (a.out_p) a.out_p[row] = hit ? tz - lse : -INFINITY;
}

// A row by a whole workgroup of COMBINE_FEW_THREADS, for calls with few rows: there k_combine's
// one or two workgroups wait for 2 x nvt / 16 loads one after the other (17.6 us for one row of
// 151669 columns; us of a replayed bf16 forward of that head with H = 64 with it and with k_combine:
// 1 row 35.1 and 40.1, 64 rows 38.1 and 43.5, 256 rows 41.5 and 44.8, so the border, FEW_ROWS, could
// lie higher; with H = 4096 64 rows take 334 and 340). All threads fetch the partials at once and work out every exponential; what is
// left in order are the chains' additions and the fold of the 16 chains. The same operations on
// the same values as k_combine's, so the same bits. Thread 0 gets the result.
constexpr int COMBINE_FEW_THREADS = 256, COMBINE_FEW_TILES = 2048;

struct CombineFewLds {
  float m[COMBINE_FEW_TILES], s[COMBINE_FEW_TILES], q[COMBINE_FEW_TILES];
  float part[COMBINE_FEW_THREADS];
  float rm[COMBINE_CHAINS], rs[COMBINE_CHAINS], rq[COMBINE_CHAINS];
  float da[COMBINE_CHAINS], db[COMBINE_CHAINS], wa[COMBINE_CHAINS], wb[COMBINE_CHAINS];
};

__device__ __forceinline__ void combine_few(const CombineArgs& a, int j, CombineFewLds& l, float& M,
                                            float& S, float& Q) {
  const int tid = threadIdx.x, c = tid % COMBINE_CHAINS;
#pragma unroll 4
  for (int vt = tid; vt < a.nvt; vt += COMBINE_FEW_THREADS) {
    const int64_t o = (int64_t)vt * a.pstride + j;
    l.m[vt] = a.pm[o];
    l.s[vt] = a.ps[o];
    l.q[vt] = a.pq[o];
  }
  // COMBINE_FEW_THREADS is a multiple of the chains: a thread's own tiles belong to one chain.
  float top = -INFINITY;
  for (int vt = tid; vt < a.nvt; vt += COMBINE_FEW_THREADS) top = fmaxf(top, l.m[vt]);
  l.part[tid] = top;
  __syncthreads();
  float mmax = -INFINITY;
#pragma unroll
  for (int k = 0; k < COMBINE_FEW_THREADS / COMBINE_CHAINS; ++k) mmax = fmaxf(mmax, l.part[c + k * COMBINE_CHAINS]);
  if (mmax != -INFINITY)
    for (int vt = tid; vt < a.nvt; vt += COMBINE_FEW_THREADS) {
      const float d = l.m[vt] - mmax, s = l.s[vt], q = l.q[vt];
      l.m[vt] = expf(d);
      l.q[vt] = weighed(q, s, d);
    }
  __syncthreads();
  if (tid < COMBINE_CHAINS) {
    M = -INFINITY;
    S = 0.f;
    Q = 0.f;
    if (mmax != -INFINITY) {
#pragma unroll 8
      for (int vt = c; vt < a.nvt; vt += COMBINE_CHAINS) {
        const float e = l.m[vt];
        S = fmaf(e, l.s[vt], S);
        Q = fmaf(e, l.q[vt], Q);
      }
      M = mmax;
    }
    l.rm[c] = M;
    l.rs[c] = S;
    l.rq[c] = Q;
  }
  __syncthreads();
  if (tid < COMBINE_CHAINS) {
    // fold()'s weights for chain c, whose running maximum is that of the chains before it.
    float before = -INFINITY;
    for (int g = 0; g < c; ++g) before = fmaxf(before, l.rm[g]);
    const float N = fmaxf(before, l.rm[c]);
    const float da = before - N, db = l.rm[c] - N;
    l.da[c] = da;
    l.db[c] = db;
    l.wa[c] = expf(da);
    l.wb[c] = expf(db);
  }
  __syncthreads();
  if (tid != 0) return;
  M = -INFINITY;
  S = 0.f;
  Q = 0.f;
#pragma unroll
  for (int g = 0; g < COMBINE_CHAINS; ++g) {
    const float m = l.rm[g], s = l.rs[g], q = l.rq[g];
    const float da = l.da[g], db = l.db[g], wa = l.wa[g], wb = l.wb[g];
    if (m == -INFINITY) continue;
    if (M == -INFINITY) {
      M = m; S = s; Q = q;
      continue;
    }
    fold_sums(S, Q, wa, wb, da, db, s, q);
    M = fmaxf(M, m);
  }
}

}  // namespace llp
