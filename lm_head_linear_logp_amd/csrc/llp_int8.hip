// llp_int8.hip -- scoring with a head in 8-bit integers: the quantisation of rows and the fused
// forward on int8 operands.
#include "llp_fwd_tile.hpp"
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

// ------------------------------------------------------------------------------------
// Row quantisation: scale = max(max |x|, 1e-30) / 127, q = x / scale to the nearest integer,
// ties to even. A wave takes a row and holds 8 columns per lane and pass in registers; rows of up to
// QUANT_PASSES * 512 columns are read once, wider ones twice (the second time from L2).
// Bound by memory: one read, half of it (bf16) written.
// ------------------------------------------------------------------------------------
constexpr int QUANT_PASSES = 8;
constexpr int QUANT_WAVES = 4;

// Columns c .. c + 7 of a row (0 past `cols`). VEC: rows are 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void quant_load(const void* row, int c, int cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    if constexpr (BF16) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_bit_cast(float, u[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + c + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (c + i < cols)
        v[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[c + i])
                    : static_cast<const float*>(row)[c + i];
    }
  }
}

// x / scale rounded to an integer (ties to even) as the correctly rounded fp32 quotient gives it.
// With inv = fl(1 / scale), x * inv is off from x / scale by at most 2^-23 of it, 1.6e-5 at
// 127; only where that leaves the rounding open is the division carried out.
__device__ __forceinline__ float quant_round(float x, float scale, float inv) {
  const float p = x * inv;
  const float r = rintf(p);
  if (__builtin_expect(fabsf(fabsf(p - r) - 0.5f) < 1e-4f, 0)) return rintf(x / scale);
  return r;
}

__device__ __forceinline__ uint2 quant_pack(const float (&v)[8], float scale, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[h] |= ((uint32_t)(int)quant_round(v[4 * h + i], scale, inv) & 0xFFu) << (8 * i);
  }
  return make_uint2(w[0], w[1]);
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(64 * QUANT_WAVES) void k_quant(QuantArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * QUANT_WAVES + (threadIdx.x >> 6);
  if (r >= a.rows) return;
  const void* row = static_cast<const char*>(a.x) + r * a.ldx * (BF16 ? 2 : 4);
  float v[QUANT_PASSES][8];
  float top = 0.f;
  bool bad = false;
  for (int c0 = 0; c0 < a.cols; c0 += QUANT_PASSES * 512) {
#pragma unroll
    for (int p = 0; p < QUANT_PASSES; ++p) {
      const int c = c0 + p * 512 + lane * 8;
      quant_load<BF16, VEC>(row, c, a.cols, v[p]);
    }
#pragma unroll
    for (int p = 0; p < QUANT_PASSES; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(v[p][i]);
        bad |= !(m < INFINITY);
        top = fmaxf(top, m);
      }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  bad = __builtin_amdgcn_ballot_w64(bad) != 0;
  const float scale = fmaxf(top, 1e-30f) / 127.f;
  const float inv = 1.f / scale;
  if (lane == 0) a.scale[r] = bad ? __builtin_nanf("") : scale;
  int8_t* q = a.q + r * a.ldq;
  const bool held = a.cols <= QUANT_PASSES * 512;
  for (int c0 = 0; c0 < a.colsp; c0 += QUANT_PASSES * 512) {
#pragma unroll
    for (int p = 0; p < QUANT_PASSES; ++p) {
      const int c = c0 + p * 512 + lane * 8;
      if (c >= a.colsp) continue;
      if (!held) quant_load<BF16, VEC>(row, c, a.cols, v[p]);
      uint2 w = quant_pack(v[p], scale, inv);
      if (bad) w = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(q + c) = w;
    }
  }
}

hipError_t launch_quant(const QuantArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  const dim3 grid((unsigned)((a.rows + QUANT_WAVES - 1) / QUANT_WAVES)), block(64 * QUANT_WAVES);
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * (a.bf16 ? 2 : 4) % 16 == 0;
  if (a.bf16 && vec) hipLaunchKernelGGL((k_quant<true, true>), grid, block, 0, s, a);
  else if (a.bf16) hipLaunchKernelGGL((k_quant<true, false>), grid, block, 0, s, a);
  else if (vec) hipLaunchKernelGGL((k_quant<false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_quant<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Fused forward on int8 operands. The tile, its walk and its epilogue are the bf16 forward's; the
// int32 sums (exact) become z * tau = (sum * weight scale) * hidden scale + bias in fp32 before
// the epilogue: three roundings of 2^-24 and, for sums past 2^24, the conversion's.
// ------------------------------------------------------------------------------------
// The tile's 256 weight scales, 256 biases and 256 hidden scales sit behind the forward's LDS, in
// the same array; they are written while the accumulators start (every wave has by then passed
// the barriers that follow the previous tile's reads of them) and read after the K loop's
// barriers. Read from global memory in the epilogue instead, under the bounds check of the last
// tile, they cost up to 1064 spilled registers.
constexpr int FWD8_LDS_HALFS = FWD_LDS_HALFS + 3 * 256 * 2;

template <int BMODE, int NFB>
__device__ __forceinline__ void int8_init(i32x16 (&acc)[4][NFB], const Fwd8Args& a, int vt, int tb,
                                          int Ts, float* sc) {
  zero_acc(acc);
  const int i = threadIdx.x & 255;
  if (threadIdx.x < 256) {
    const int v = vt * BM + i;
    const bool in = v < a.f.n_real;
    sc[i] = in ? a.ws[v] : 0.f;
    if constexpr (BMODE == BIAS_F32)
      sc[256 + i] = in ? reinterpret_cast<const float*>(a.f.bias)[v] : 0.f;
    if constexpr (BMODE == BIAS_BF16)
      sc[256 + i] = in ? bf16_to_f32(reinterpret_cast<const uint16_t*>(a.f.bias)[v]) : 0.f;
  } else {
    const int j = tb * BN + i;
    sc[512 + i] = a.hs[a.f.scored[j < Ts ? j : Ts - 1]];
  }
}

template <int BMODE, int NFB>
__device__ __forceinline__ void int8_epilogue(const i32x16 (&ai)[4][NFB], const Fwd8Args& a,
                                              int vt, int tb, int Ts, float* red, const float* sc) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave & 1, wn = wave >> 1;
  float hs[NFB];
#pragma unroll
  for (int ni = 0; ni < NFB; ++ni) hs[ni] = sc[512 + (wn * NFB + ni) * 32 + (lane & 31)];
  f32x16 acc[4][NFB];
#pragma unroll
  for (int mi = 0; mi < 4; ++mi)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int v = wm * 128 + mi * 32 + 8 * g + 4 * (lane >> 5);   // rows v .. v + 3 (mfma_row)
      const float4 w = *reinterpret_cast<const float4*>(sc + v);
      float4 b = {0.f, 0.f, 0.f, 0.f};
      if constexpr (BMODE != BIAS_NONE) b = *reinterpret_cast<const float4*>(sc + 256 + v);
#pragma unroll
      for (int ni = 0; ni < NFB; ++ni)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wu = u == 0 ? w.x : u == 1 ? w.y : u == 2 ? w.z : w.w;
          const float bu = u == 0 ? b.x : u == 1 ? b.y : u == 2 ? b.z : b.w;
          const float x = (float)ai[mi][ni][4 * g + u] * wu;
          acc[mi][ni][4 * g + u] = BMODE == BIAS_NONE ? x * hs[ni] : fmaf(x, hs[ni], bu);
        }
      // One group's scales at a time: read ahead together they push accumulators out.
      __builtin_amdgcn_sched_barrier(0);
    }
  fwd_tile_epilogue<NFB>(acc, a.f, vt, tb, Ts, red);
}

template <int BMODE, int NW>
__global__ __launch_bounds__(64 * NW, 1) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void k_fwd8(Fwd8Args a) {
  constexpr int NFB = 16 / NW;
  __shared__ __attribute__((aligned(16))) uint16_t smem[FWD8_LDS_HALFS];
  float* const sc = reinterpret_cast<float*>(smem + FWD_LDS_HALFS);
  fwd_persistent<NW, i32x16>(
      a.f, smem,
      [&](i32x16 (&acc)[4][NFB], int vt, int tb, int Ts) {
        int8_init<BMODE, NFB>(acc, a, vt, tb, Ts, sc);
      },
      [&](const i32x16 (&acc)[4][NFB], int vt, int tb, int Ts, float* red) {
        int8_epilogue<BMODE, NFB>(acc, a, vt, tb, Ts, red, sc);
      });
}

template <int BMODE, int NW>
__global__ __launch_bounds__(64 * NW, 1) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void k_fwd8_tiles(Fwd8Args a) {
  constexpr int NFB = 16 / NW;
  __shared__ __attribute__((aligned(16))) uint16_t smem[FWD8_LDS_HALFS];
  float* const sc = reinterpret_cast<float*>(smem + FWD_LDS_HALFS);
  fwd_one_tile<NW, i32x16>(
      a.f, smem,
      [&](i32x16 (&acc)[4][NFB], int vt, int tb, int Ts) {
        int8_init<BMODE, NFB>(acc, a, vt, tb, Ts, sc);
      },
      [&](const i32x16 (&acc)[4][NFB], int vt, int tb, int Ts, float* red) {
        int8_epilogue<BMODE, NFB>(acc, a, vt, tb, Ts, red, sc);
      });
}

hipError_t launch_fwd8(const Fwd8Args& a, hipStream_t s) {
  if (a.f.nvt <= 0 || a.f.ntb <= 0) return hipGetLastError();
  const int64_t ntiles = (int64_t)a.f.nvt * a.f.ntb;
  const int n = a.f.H / KSTEP;
  const dim3 block(64 * FWD_WAVES);
  const bool b32 = a.f.bias_f32 != 0;
  if (n >= 2 && n % 2 == 0) {
    int64_t workers = a.f.workers > 0 && a.f.workers < ntiles ? a.f.workers : ntiles;
    workers = (workers + NUM_XCD - 1) / NUM_XCD * NUM_XCD;
    const dim3 grid((unsigned)workers);
    if (a.f.bias == nullptr) hipLaunchKernelGGL((k_fwd8<BIAS_NONE, FWD_WAVES>), grid, block, 0, s, a);
    else if (b32) hipLaunchKernelGGL((k_fwd8<BIAS_F32, FWD_WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_fwd8<BIAS_BF16, FWD_WAVES>), grid, block, 0, s, a);
  } else {
    const dim3 grid((unsigned)ntiles);
    if (a.f.bias == nullptr) hipLaunchKernelGGL((k_fwd8_tiles<BIAS_NONE, FWD_WAVES>), grid, block, 0, s, a);
    else if (b32) hipLaunchKernelGGL((k_fwd8_tiles<BIAS_F32, FWD_WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_fwd8_tiles<BIAS_BF16, FWD_WAVES>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace llp
