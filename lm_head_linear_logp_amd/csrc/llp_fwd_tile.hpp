// llp_fwd_tile.hpp -- what the fused forward's kernels share: the operands' loaders, the bias
// as starting accumulators, the tile epilogue (max, sum-exp, entropy sum, target logit), and the
// two ways a launch walks its tiles.
#pragma once

#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

// ------------------------------------------------------------------------------------
// Fused forward tile: z = (h W^T + b) * (1/tau) for 256 vocabulary columns x 256 scored
// rows, then per row of the tile the max m, s = sum exp(z - m) and q = sum exp(z - m) (z - m)
// log2(e), plus the target logit when the target column lies in the tile. Columns at or
// past the shard's real vocabulary are excluded ([CUDA provider, "Megatron integration"]:
// real/padded vocabulary sizes). The [T, V] logits never leave registers.
// MFMA operand A = weight rows (vocabulary, M), B = hidden rows (tokens, N): each lane owns
// one token column, so the per-row reductions run down its own registers first.
// ------------------------------------------------------------------------------------
// The bias enters as the accumulators' starting value: z * tau = bias + h.W^T comes straight
// out of the MFMAs, so neither epilogue reads the bias, and every bias mode runs the no-bias
// epilogue with its register footprint. The forward and the gradient tile start the same way,
// so both see the same z.
//
// Bias of this lane's 16 accumulator rows of the 32-row block at vb: rows
// vb + 8g + 4(lane/32) + 0..3 for g = 0..3 (mfma_row), i.e. four runs of four consecutive
// rows, each read with one vector load (the bias is 16-byte aligned for fp32, 8-byte for
// bf16). Rows at or past n_real (only in the shard's last tile) read as 0.
template <bool F32>
__device__ __forceinline__ void bias16(const void* bias, int vb, int lane, int64_t n_real,
                                       float (&b)[16]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int v = vb + 8 * g + 4 * (lane >> 5);
    if (v + 3 < n_real) {
      if constexpr (F32) {
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(bias) + v);
        b[4 * g] = x.x;
        b[4 * g + 1] = x.y;
        b[4 * g + 2] = x.z;
        b[4 * g + 3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(bias) + v);
        b[4 * g] = __builtin_bit_cast(float, x.x << 16);
        b[4 * g + 1] = __builtin_bit_cast(float, x.x & 0xFFFF0000u);
        b[4 * g + 2] = __builtin_bit_cast(float, x.y << 16);
        b[4 * g + 3] = __builtin_bit_cast(float, x.y & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x = 0.f;
        if (v + u < n_real)
          x = F32 ? reinterpret_cast<const float*>(bias)[v + u]
                  : bf16_to_f32(reinterpret_cast<const uint16_t*>(bias)[v + u]);
        b[4 * g + u] = x;
      }
    }
  }
}

// Starting accumulators of a vocabulary x token tile at v0: each lane's rows get their bias (the
// same for all its token blocks).
template <bool F32, int NFB>
__device__ __forceinline__ void bias_acc(f32x16 (&acc)[4][NFB], const void* bias, int v0,
                                         int64_t n_real) {
  const int lane = threadIdx.x & 63, wm = (threadIdx.x >> 6) & 1;
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
    float b[16];
    bias16<F32>(bias, v0 + wm * 128 + mi * 32, lane, n_real, b);
#pragma unroll
    for (int ni = 0; ni < NFB; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mi][ni][r] = b[r];
  }
}

// The same, or 0 without a bias (mode chosen at run time).
template <int NFB>
__device__ __forceinline__ void init_acc(f32x16 (&acc)[4][NFB], const void* bias, bool bias_f32,
                                         int v0, int64_t n_real) {
  if (bias == nullptr) zero_acc(acc);
  else if (bias_f32) bias_acc<true, NFB>(acc, bias, v0, n_real);
  else bias_acc<false, NFB>(acc, bias, v0, n_real);
}

constexpr int BIAS_NONE = 0, BIAS_BF16 = 1, BIAS_F32 = 2;

// NFB = 4: 4 waves (2 x 2) of 128 vocabulary columns x 128 tokens; NFB = 2: 8 waves (2 x 4)
// of 128 x 64. Either way a token's values are reduced in the same order: down the lane's
// 64 values of its wave's 128 columns (mi, r), the lane pair, then the two column halves.
template <bool TAIL, int NFB>
__device__ __forceinline__ void fwd_epilogue(const f32x16 (&acc)[4][NFB], const FwdArgs& a, int vt,
                                             int v0, int j0, int Ts, float* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave & 1, wn = wave >> 1;
  constexpr int TW = 32 * NFB;  // tokens per wave
  const int vbase = v0 + wm * 128;
  // red: [6][256] in LDS: max0 max1 s0 s1 q0 q1. The exchange between waves goes through LDS
  // only, so the barriers wait for LDS alone (DMA loads of a next tile may be in flight).
  // Pass 1: per-token max of x over this lane's 64 columns, the lane pair (l, l^32) and the two
  // waves holding the tile's two column halves. z = x * c1 with c1 > 0 and rounding is
  // monotonic, so fl(max x * c1) is the max of z.
  float mx[NFB];
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) mx[ni] = -INFINITY;
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
#pragma unroll
    for (int ni = 0; ni < NFB; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float x = acc[mi][ni][r];
        if (TAIL && vbase + mi * 32 + mfma_row(r, lane) >= a.n_real) x = -INFINITY;
        mx[ni] = fmaxf(mx[ni], x);
      }
  }
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) {
    mx[ni] = fmaxf(mx[ni], __shfl_xor(mx[ni], 32));
    if (lane < 32) red[wm * 256 + wn * TW + ni * 32 + lane] = mx[ni];
  }
  dma::lds_barrier();
  // Pass 2: s = sum 2^d2, q = sum 2^d2 * d2 with d2 = (z - M) log2(e) = x c1 log2(e) - M log2(e).
  const float c1l = a.c1 * kLog2e;
  float ml[NFB];
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) {
    const int tn = wn * TW + ni * 32 + (lane & 31);
    mx[ni] = fmaxf(red[tn], red[256 + tn]) * a.c1;
    ml[ni] = mx[ni] * kLog2e;
  }
  float sv[NFB], qv[NFB];
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) sv[ni] = qv[ni] = 0.f;
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
#pragma unroll
    for (int ni = 0; ni < NFB; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float d2 = fmaf(acc[mi][ni][r], c1l, -ml[ni]);
        // Excluded column: 2^-1e30 = 0 and 0 * -1e30 = 0.
        if (TAIL && vbase + mi * 32 + mfma_row(r, lane) >= a.n_real) d2 = -1e30f;
        const float e = __builtin_amdgcn_exp2f(d2);
        sv[ni] += e;
        qv[ni] = fmaf(e, d2, qv[ni]);
      }
  }
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) {
    // (x + y) == (y + x): both lanes of a pair hold the same sum.
    sv[ni] += __shfl_xor(sv[ni], 32);
    qv[ni] += __shfl_xor(qv[ni], 32);
    if (lane < 32) {
      const int tn = wn * TW + ni * 32 + lane;
      red[512 + wm * 256 + tn] = sv[ni];
      red[1024 + wm * 256 + tn] = qv[ni];
    }
  }
  dma::lds_barrier();
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) {
    const int tn = wn * TW + ni * 32 + (lane & 31);
    const int j = j0 + tn;
    if (wm == 0 && lane < 32 && j < Ts) {
      const int64_t o = (int64_t)vt * a.pstride + j;
      a.pm[o] = mx[ni];
      a.ps[o] = red[512 + tn] + red[768 + tn];
      a.pq[o] = red[1024 + tn] + red[1280 + tn];
    }
    // Target logit: the one lane holding column tloc[j] copies its z (rare: skipped unless
    // some lane of the wave holds a target).
    const int tl = (j < Ts) ? a.tloc[j] - vbase : -1;
    const bool mine = tl >= 0 && tl < 128 && (((tl & 31) >> 2) & 1) == (lane >> 5);
    if (__builtin_amdgcn_ballot_w64(mine)) {
      const int mt = tl >> 5, rt = (((tl & 31) >> 3) << 2) | (tl & 3);
      float t = 0.f;
#pragma unroll
      for (int mi = 0; mi < 4; ++mi)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (mi == mt && r == rt) t = acc[mi][ni][r];
      if (mine) a.tz[j] = t * a.c1;
    }
  }
}

// Loaders of the fused tiles: weight rows v0 .. (clamped below n_real) and the scored hidden
// rows j0 .. (clamped below the count), gathered through `scored` (ascending). The hidden
// resource starts at the tile's first scored row; the host keeps all T rows within 2^31 bytes
// (T * hidden_stride * 2 < 2^31), so every lane offset, plus the K step's scalar offset, stays
// below 2^31 and inside the resource's range.
template <int NW>
__device__ __forceinline__ void weight_hidden_loaders(const uint16_t* W, int64_t ldw, int64_t n_real,
                                                      int v0, const uint16_t* h, int64_t ldh,
                                                      const int32_t* scored, int j0, int Ts, int H,
                                                      dma::LoaderT<NW>& la, dma::LoaderT<NW>& lb) {
  const int nv = n_real - v0 < BM ? (int)(n_real - v0) : BM;
  const int nj = Ts - j0 < BN ? Ts - j0 : BN;
  // One address for the whole wave: readfirstlane keeps the resources in scalar registers also
  // where the compiler reads `scored` with vector loads (after stores it cannot prove
  // disjoint), which would otherwise put every DMA instruction in a per-lane loop.
  const int64_t h0 = __builtin_amdgcn_readfirstlane(scored[j0]);
  const int64_t hl = __builtin_amdgcn_readfirstlane(scored[j0 + nj - 1]);
  la.init(W + (int64_t)v0 * ldw, (uint64_t)((nv - 1) * ldw + H) * 2);
  lb.init(h + h0 * ldh, (uint64_t)((hl - h0) * ldh + H) * 2);
#pragma unroll
  for (int u = 0; u < dma::LoaderT<NW>::NIW; ++u) {
    const int r = dma::LoaderT<NW>::row_of(u);
    la.set(u, r < nv ? r : nv - 1, ldw);
    lb.set(u, scored[j0 + (r < nj ? r : nj - 1)] - h0, ldh);
  }
}

// The forward's LDS: the pipeline's two stages, then the epilogue's 6 x 256 fp32 partials and a
// word for tile claims. One array, not several: with a second LDS object the compiler can no
// longer tell the stages' DMA writes from the fragment reads and waits for every DMA load
// before each read.
constexpr int FWD_LDS_HALFS = dma::LDS_BYTES / 2 + 6 * 256 * 2 + 8;   // + the tile-claim slot
static_assert(dma::BKD == KSTEP, "K step shared with the host");
static_assert(QCTR_INTS > NUM_XCD, "queue counters and the all-empty flag");

// The forward tile runs FWD_WAVES = 8 waves, two per SIMD: each wave holds 128 x 64 outputs (128
// accumulators), so one wave's LDS reads, DMA issue and barrier waits overlap the other's
// MFMAs. Every output's MFMA chain and every token's reduction order are those of the 4-wave
// tile (1 wave per SIMD, 128 x 128 per wave). Kernels come one per bias mode, differing only in
// how the accumulators start: a run-time choice there makes the compiler spill accumulators in
// the epilogue.
constexpr int FWD_WAVES = 8;

template <int BMODE, int NFB>
__device__ __forceinline__ void fwd_init_acc(f32x16 (&acc)[4][NFB], const FwdArgs& a, int v0) {
  if constexpr (BMODE == BIAS_NONE) zero_acc(acc);
  else bias_acc<BMODE == BIAS_F32, NFB>(acc, a.bias, v0, a.n_real);
}

template <int NFB>
__device__ __forceinline__ void fwd_tile_epilogue(const f32x16 (&acc)[4][NFB], const FwdArgs& a,
                                                  int vt, int tb, int Ts, float* red) {
  const int v0 = vt * BM, j0 = tb * BN;
  if (v0 + BM > a.n_real) fwd_epilogue<true, NFB>(acc, a, vt, v0, j0, Ts, red);
  else fwd_epilogue<false, NFB>(acc, a, vt, v0, j0, Ts, red);
}

// The forward GEMM as persistent workers (the host launches one per compute unit, a multiple
// of NUM_XCD, when the K steps are even). XCD x owns a contiguous share of the logical tiles
// (its queue, as for the backward kernels). Worker wi of the XCD runs positions wi, wi + nwx,
// ... of the queue's static first three quarters, in the order one workgroup per tile would
// start them, then claims tiles of the dynamic last quarter one at a time (own XCD first, then
// the others'), so that workers of a faster XCD take over the tail of a slower one. Against
// one workgroup per tile this saves each tile's launch, address setup and first DMA round
// trip: the last two K steps of a tile load the first two of the worker's next tile, which
// land during the epilogue. Tiles past the scored rows are skipped. A tile's arithmetic is
// that of fwd_one_tile, whoever runs it: results are bitwise the same.
// `init` sets the starting accumulators of tile (vt, tb), `epilogue` takes the finished ones;
// their type (f32x16 or i32x16) picks bf16 or int8 products.
template <int NW, class ACC, class Init, class Epilogue>
__device__ __forceinline__ void fwd_persistent(const FwdArgs& a, uint16_t* smem, Init init,
                                               Epilogue epilogue) {
  constexpr int NFB = 16 / NW;
  float* const red = reinterpret_cast<float*>(smem + dma::LDS_BYTES / 2);
  int* const slot = reinterpret_cast<int*>(red + 6 * 256);
  const int Ts = *a.count;
  const int ntiles = a.nvt * a.ntb;
  const int x = blockIdx.x % NUM_XCD, nwx = gridDim.x / NUM_XCD;
  const int qf = queue_first(ntiles, x), s0 = queue_static(queue_size(ntiles, x));
  int pos = blockIdx.x / NUM_XCD;   // the worker's next static position
  // The worker's next tile with scored rows: false when there is none.
  auto next_tile = [&](int& vt, int& tb) -> bool {
    for (;;) {
      int t;
      if (pos < s0) {
        t = qf + pos;
        pos += nwx;
      } else {
        if (threadIdx.x == 0) *slot = claim_dynamic(a.qctr, ntiles, x);
        dma::lds_barrier();
        t = *slot;
        dma::lds_barrier();   // every wave has read the slot before the next claim writes it
        if (t < 0) return false;
      }
      vocab_token_tile(t, a.nvt, a.ntb, vt, tb);
      if (tb * BN < Ts) return true;
    }
  };
  int vt = 0, tb = 0;
  if (!next_tile(vt, tb)) return;
  const int n = a.H / dma::BKD;
  dma::LoaderT<NW> la, lb, la2, lb2;
  weight_hidden_loaders<NW>(a.W, a.ldw, a.n_real, vt * BM, a.h, a.ldh, a.scored, tb * BN, Ts,
                            a.H, la, lb);
  bool primed = false;
  for (;;) {
    int vt2 = 0, tb2 = 0;
    const bool more = next_tile(vt2, tb2);
    if (more) {
      weight_hidden_loaders<NW>(a.W, a.ldw, a.n_real, vt2 * BM, a.h, a.ldh, a.scored, tb2 * BN,
                                Ts, a.H, la2, lb2);
    } else {
      la2 = la;
      lb2 = lb;
    }
    ACC acc[4][NFB];
    init(acc, vt, tb, Ts);
    dma::mainloop_chain(la, lb, la2, lb2, primed, more, n, smem, acc);
    epilogue(acc, vt, tb, Ts, red);
    if (!more) break;
    vt = vt2;
    tb = tb2;
    la = la2;
    lb = lb2;
    primed = true;
  }
}

// One workgroup per tile in the static XCD order: the forward for an odd number of K steps,
// where the persistent workers' stage parity does not carry from one tile to the next.
template <int NW, class ACC, class Init, class Epilogue>
__device__ __forceinline__ void fwd_one_tile(const FwdArgs& a, uint16_t* smem, Init init,
                                             Epilogue epilogue) {
  constexpr int NFB = 16 / NW;
  float* const red = reinterpret_cast<float*>(smem + dma::LDS_BYTES / 2);
  int vt, tb;
  vocab_token_tile(xcd_remap(blockIdx.x, gridDim.x), a.nvt, a.ntb, vt, tb);
  const int Ts = *a.count;
  if (tb * BN >= Ts) return;
  dma::LoaderT<NW> la, lb;
  weight_hidden_loaders<NW>(a.W, a.ldw, a.n_real, vt * BM, a.h, a.ldh, a.scored, tb * BN, Ts,
                            a.H, la, lb);
  ACC acc[4][NFB];
  init(acc, vt, tb, Ts);
  dma::mainloop(la, lb, 0, a.H / dma::BKD, smem, acc);
  epilogue(acc, vt, tb, Ts, red);
}

}  // namespace llp
