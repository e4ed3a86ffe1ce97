// llp_int8.hip -- scoring with a head in 8-bit integers: the quantisation of rows and the fused
// forward on int8 operands.
#include "llp_combine.hpp"
#include "llp_fwd_tile.hpp"
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

// ------------------------------------------------------------------------------------
// Row quantisation: scale = max(max |x|, 1e-30) * fl32(1/127), q = x / scale to the nearest
// integer, ties to even. A team of lanes takes a row and holds 8 columns per lane and pass in
// registers; only rows of more than 8192 columns are read twice (the second time from L2).
// Bound by memory: one read, half of it (bf16) written: 97 us for 37984 x 4096 bf16, 4.8 TB/s, a
// copy's rate.
// ------------------------------------------------------------------------------------
constexpr int QUANT_THREADS = 256;

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

// Eight values as bytes: x / scale rounded to an integer (ties to even) as the correctly rounded
// fp32 quotient gives it. With inv = fl(1 / scale), x * inv is off from x / scale by at most
// 2^-23 of it, 1.6e-5 at 127; only where that leaves a lane's rounding open are the wave's
// divisions carried out (2e-4 of the values).
__device__ __forceinline__ uint2 quant_pack(const float (&v)[8], float scale, float inv) {
  float r[8];
  bool open = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = v[i] * inv;
    r[i] = rintf(p);
    open |= fabsf(p - r[i]) > 0.4999f;
  }
  if (__builtin_amdgcn_ballot_w64(open) != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = rintf(v[i] / scale);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)r[i] & 0xFFu) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// TEAM lanes share a row (half a wave, a wave or the workgroup), PASSES x 8 columns each.
template <bool BF16, bool VEC, int TEAM, int PASSES>
__global__ __launch_bounds__(QUANT_THREADS) void k_quant(QuantArgs a) {
  __shared__ float tops[QUANT_THREADS / 64];
  constexpr int STEP = TEAM * 8, ROWS = QUANT_THREADS / TEAM;   // columns per pass, rows at a time
  const int lane = threadIdx.x % TEAM;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / TEAM; r < a.rows; r += step) {
    const void* row = static_cast<const char*>(a.x) + r * a.ldx * (BF16 ? 2 : 4);
    float v[PASSES][8];
    float top = 0.f;   // becomes infinite with an infinity or NaN in the row
    for (int c0 = 0; c0 < a.cols; c0 += PASSES * STEP) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) quant_load<BF16, VEC>(row, c0 + p * STEP + lane * 8, a.cols, v[p]);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float m = fabsf(v[p][i]);
          top = m <= top ? top : m < INFINITY ? m : INFINITY;
        }
    }
#pragma unroll
    for (int off = (TEAM < 64 ? TEAM : 64) / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if constexpr (TEAM > 64) {
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TEAM / 64; ++w) top = fmaxf(top, tops[w]);
      __syncthreads();   // read by all before the next row's are written
    }
    const bool bad = !(top < INFINITY);
    const float scale = fmaxf(top, 1e-30f) * (1.f / 127.f);
    const float inv = 1.f / scale;
    if (lane == 0) a.scale[r] = bad ? __builtin_nanf("") : scale;
    int8_t* q = a.q + r * a.ldq;
    const bool held = a.cols <= PASSES * STEP;
    for (int c0 = 0; c0 < a.colsp; c0 += PASSES * STEP) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int c = c0 + p * STEP + lane * 8;
        if (c >= a.colsp) continue;
        if (!held) quant_load<BF16, VEC>(row, c, a.cols, v[p]);
        uint2 w = quant_pack(v[p], scale, inv);
        if (bad) w = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(q + c) = w;
      }
    }
  }
}

template <bool BF16, bool VEC, int TEAM, int PASSES>
static void launch_quant_team(const QuantArgs& a, hipStream_t s) {
  // A launch holds fewer than 2^32 threads: past 2^22 workgroups each takes several rows.
  constexpr int ROWS = QUANT_THREADS / TEAM;
  const int64_t n = (a.rows + ROWS - 1) / ROWS;
  const dim3 grid((unsigned)(n < (1 << 22) ? n : 1 << 22));
  hipLaunchKernelGGL((k_quant<BF16, VEC, TEAM, PASSES>), grid, dim3(QUANT_THREADS), 0, s, a);
}

template <bool BF16, bool VEC>
static void launch_quant_as(const QuantArgs& a, hipStream_t s) {
  // The smallest team whose registers hold the row (2^27 bf16 values, us a call: 2048 columns 84 by
  // a wave and 117 by the workgroup, 1152 columns 105 and 184, 256 columns 136 by half a wave and
  // 215 by one; a wave that reads the row twice takes 105 for 4096 columns, the workgroup 86).
  if (a.cols <= 512) launch_quant_team<BF16, VEC, 32, 2>(a, s);
  else if (a.cols <= 1024) launch_quant_team<BF16, VEC, 64, 2>(a, s);
  else if (a.cols <= 2048) launch_quant_team<BF16, VEC, 64, 4>(a, s);
  else if (a.cols <= 4096) launch_quant_team<BF16, VEC, 256, 2>(a, s);
  else launch_quant_team<BF16, VEC, 256, 4>(a, s);
}

hipError_t launch_quant(const QuantArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * (a.bf16 ? 2 : 4) % 16 == 0;
  if (a.bf16) vec ? launch_quant_as<true, true>(a, s) : launch_quant_as<true, false>(a, s);
  else vec ? launch_quant_as<false, true>(a, s) : launch_quant_as<false, false>(a, s);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Fused forward on int8 operands. The tile, its walk and its epilogue are the bf16 forward's; the
// int32 sums (exact) become z * tau = (sum * weight scale) * hidden scale + bias in fp32 before
// the epilogue: three roundings of 2^-24 and, for sums past 2^24, the conversion's. A bias costs 3 %
// (4096 rows: 2168 us replayed, 2102 without): the kernels that add one spill 13 registers. Bound by the
// matrix cores: 3686 scored rows of 4096 x 151669 columns take 1906 to 1994 us, 2.3 to 2.4e15
// operations a second, with the MFMA pipes busy 69 % of the time at the 1.56 GHz that such a load
// is left with; the library's plain int8 product of 8192^3 reaches 2.26e15.
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

// ------------------------------------------------------------------------------------
// Few rows (at most FEW_ROWS, one wave's lanes): the weight's bytes bound the forward, so nothing is staged. A
// workgroup takes one vocabulary tile; a wave takes 16 IB columns x all rows (NB blocks of 16)
// over one of KS parts of K, loads its operands straight into MFMA registers and refills a block's
// registers as soon as its MFMAs have read them, so its loads never drain.
//
// v_mfma_i32_16x16x64_i8: lane l supplies A[l % 16][k] and B[k][l % 16] for k = 16 (l / 16) +
// 0..15, and holds D[4 (l / 16) + r][l % 16]. Loaded as the MFMA wants them, neighbouring lanes
// would hold neighbouring rows, every lane a request of its own, and the L1's request rate would
// bound the stream (37 rows of a 37717-column shard: 53 us). So an instruction takes whole
// 128-byte lines of 8 weight rows, once and past the caches, and the fragments are moved to their
// lanes: a DPP move and a ds_bpermute per register. Measured (K of 4096): one row of 151669 columns
// 104 us, 6.0 TB/s of weight (118 us with half lines kept in the caches, 116 with whole ones).
//
// The int32 sums of the K parts meet in LDS (exact in any order), and from there the epilogue's
// waves take them in the wide tile's register layout: its sums run in the same order, so every
// row gets the wide tile's bits.
// ------------------------------------------------------------------------------------
// The layout of so few rows is a ballot: every workgroup works it out for itself, which saves a
// launch in front. Returns the wave's mask of scored rows.
__device__ __forceinline__ uint64_t few_scored(const LayoutArgs& la) {
  const int lane = threadIdx.x & 63;
  return __builtin_amdgcn_ballot_w64(lane < la.T && (la.mask == nullptr || la.mask[lane < la.T ? lane : 0] != 0));
}

// Local column of row t's target, or -1, and the status bits it raises.
__device__ __forceinline__ int few_target(const LayoutArgs& la, int t, int& status) {
  const int64_t tg = la.targets[t];
  const bool valid = tg >= 0 && tg < la.real_vocab;
  if (!valid) status |= LLP_STATUS_TARGET_OUT_OF_RANGE;
  const int64_t loc = tg - la.offset;
  const bool hit = valid && loc >= 0 && loc < la.n_real;
  if (!hit && la.world == 1) status |= LLP_STATUS_TARGET_NOT_FOUND;
  return hit ? (int)loc : -1;
}

template <int BMODE, int NB, int IB, int KS, int BUFS>
__global__ __launch_bounds__(1024 / IB * KS) __attribute__((amdgpu_waves_per_eu(KS * 16 / IB == 4 && NB < 3 ? 3 : 2))) void k_fwd8_few(Fwd8Args a) {
  constexpr int CG = 16 / IB;   // column groups
  constexpr int THREADS = 64 * CG * KS, LDT = BM + 4;   // LDT: ints per row of sums, off the bank stride
  __shared__ __attribute__((aligned(16))) float red[6 * 256];
  __shared__ __attribute__((aligned(16))) float sc[3 * 256];
  __shared__ __attribute__((aligned(16))) int sums[BUFS][16 * NB][LDT];
  __shared__ int scored[FEW_ROWS], tloc[FEW_ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t on = few_scored(a.la);
  const int Ts = __popcll(on);
  if (Ts == 0) return;
  if (wave == 0 && ((on >> lane) & 1) != 0) {
    const int j = __popcll(on & ((1ull << lane) - 1));
    int status = 0;
    scored[j] = lane;
    tloc[j] = few_target(a.la, lane, status);
  }
  __syncthreads();
  const int cg = wave % CG, ks = wave / CG;
  const int vt = blockIdx.x, v0 = vt * BM;
  const int64_t ldw = a.f.ldw * 2, ldh = a.f.ldh * 2;   // bytes
  const char* const W = reinterpret_cast<const char*>(a.f.W) + (int64_t)v0 * ldw;
  const char* const h = reinterpret_cast<const char*>(a.f.h);
  const int rows = a.f.n_real - v0 < BM ? (int)(a.f.n_real - v0) : BM;
  const int l16 = lane & 15;
  const int lr = lane >> 2, kb = (lane & 3) * 16;   // hidden row and bytes this lane loads
  const int from = 4 * (l16 * 4 + (lane >> 4));     // and where its MFMA operand is (bpermute)
  uint32_t oa[IB][2], ob[NB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = cg * 16 * IB + i * 16 + q * 8 + (lane >> 3);
      oa[i][q] = (uint32_t)((r < rows ? r : rows - 1) * ldw) + (lane & 7) * 16;
    }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int j = n * 16 + lr;
    ob[n] = (uint32_t)(scored[j < Ts ? j : Ts - 1] * ldh) + kb;
  }
  const int steps = a.f.H / KSTEP;   // of 128 bytes
  const int s0 = steps * ks / KS, s1 = steps * (ks + 1) / KS;
  i32x4 acc[IB][NB], A[IB][2], B[NB][2], Bn[NB][2];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[i][n] = i32x4{0, 0, 0, 0};
  auto load = [&](i32x4 (&x)[2], const char* base, uint32_t off, int s) {
    const char* p = base + (size_t)(off + (uint32_t)s * 128u);
    x[0] = *reinterpret_cast<const i32x4*>(p);
    x[1] = *reinterpret_cast<const i32x4*>(p + 64);
  };
  auto placed = [&](const i32x4& x) {
    i32x4 y;
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = __builtin_amdgcn_ds_bpermute(from, x[u]);
    return y;
  };
  // The weight: instruction q takes the whole lines of rows 8 q .. 8 q + 7, lane l 16 bytes at
  // 16 (l % 8) of row l / 8.
  auto load_lines = [&](i32x4 (&x)[2], const uint32_t (&off)[2], int s) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      x[q] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(W + (size_t)(off[q] + (uint32_t)s * 128u)));
  };
  // Fragment q of a block: its bytes 64 q .. 64 q + 63 of 16 rows. The lanes that hold the other
  // half of rows 0 .. 7 take rows 8 .. 15's (q = 0), and the other way round (q = 1): a move
  // within rows of 16 lanes. Then ds_bpermute.
  const int from_lines = 4 * ((l16 & 7) * 8 + (l16 >> 3) * 4 + (lane >> 4));
  auto fragment = [&](const i32x4 (&x)[2], int q) {
    i32x4 y;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int lo = x[0][u], hi = x[1][u];
      const int z = q == 0 ? __builtin_amdgcn_update_dpp(lo, hi, 0x114, 0xf, 0xA, false)    // row_shr:4
                           : __builtin_amdgcn_update_dpp(hi, lo, 0x104, 0xf, 0x5, false);   // row_shl:4
      y[u] = __builtin_amdgcn_ds_bpermute(from_lines, z);
    }
    return y;
  };
  auto products = [&](int i) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const i32x4 x = fragment(A[i], q);
#pragma unroll
      for (int n = 0; n < NB; ++n)
        acc[i][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, B[n][q], acc[i][n], 0, 0, 0);
    }
  };
  if (s0 < s1) {
    // Issued in the order they are used: a wait for the first then leaves the rest in flight.
#pragma unroll
    for (int n = 0; n < NB; ++n) load(Bn[n], h, ob[n], s0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      load_lines(A[i], oa[i], s0);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int s = s0; s + 1 < s1; ++s) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) B[n][q] = placed(Bn[n][q]);
#pragma unroll
      for (int n = 0; n < NB; ++n) load(Bn[n], h, ob[n], s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        products(i);
        load_lines(A[i], oa[i], s + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q) B[n][q] = placed(Bn[n][q]);
#pragma unroll
    for (int i = 0; i < IB; ++i) products(i);
  }
  // Scales of the tile's columns and of the rows.
  for (int i = threadIdx.x; i < 256; i += THREADS) {
    const int v = v0 + i;
    const bool in = v < a.f.n_real;
    sc[i] = in ? a.ws[v] : 0.f;
    if constexpr (BMODE == BIAS_F32)
      sc[256 + i] = in ? reinterpret_cast<const float*>(a.f.bias)[v] : 0.f;
    if constexpr (BMODE == BIAS_BF16)
      sc[256 + i] = in ? bf16_to_f32(reinterpret_cast<const uint16_t*>(a.f.bias)[v]) : 0.f;
    if (i < FEW_ROWS) sc[512 + i] = a.hs[scored[i < Ts ? i : Ts - 1]];
  }
  // K parts p, p + BUFS, ... share buffer p: the first writes, the others add in turn.
#pragma unroll
  for (int ph = 0; ph < KS / BUFS; ++ph) {
    if (ks / BUFS == ph) {
#pragma unroll
      for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          i32x4* p = reinterpret_cast<i32x4*>(&sums[ks % BUFS][n * 16 + l16][cg * 16 * IB + i * 16 + (lane >> 4) * 4]);
          *p = ph == 0 ? acc[i][n] : *p + acc[i][n];
        }
    }
    __syncthreads();
  }
  if (wave >= 2 * ((NB + 1) / 2)) {
    // The epilogue's two barriers.
    dma::lds_barrier();
    dma::lds_barrier();
    return;
  }
  const int wm = wave & 1;
  const int token = ((wave >> 1) * 32 + (lane & 31)) % (16 * NB);
  i32x16 x[4][1];
#pragma unroll
  for (int mi = 0; mi < 4; ++mi)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int v = wm * 128 + mi * 32 + 8 * g + 4 * (lane >> 5);   // rows v .. v + 3 (mfma_row)
      i32x4 y = *reinterpret_cast<const i32x4*>(&sums[0][token][v]);
#pragma unroll
      for (int p = 1; p < BUFS; ++p) y += *reinterpret_cast<const i32x4*>(&sums[p][token][v]);
#pragma unroll
      for (int u = 0; u < 4; ++u) x[mi][0][4 * g + u] = y[u];
    }
  Fwd8Args own = a;
  own.f.tloc = tloc;
  int8_epilogue<BMODE, 1>(x, own, vt, 0, Ts, red, sc);
}

// The rest of a few-row forward: a workgroup per row, scored or not, combines its partials and writes
// its outputs and status; the first one checks cu_seqlens.
__global__ __launch_bounds__(COMBINE_FEW_THREADS) void k_fwd8_few_out(Fwd8Args a) {
  __shared__ CombineFewLds lds;
  const LayoutArgs& la = a.la;
  const int t = blockIdx.x;
  int status = 0;
  if (t == 0 && la.cu_seqlens != nullptr)
    for (int i = threadIdx.x; i <= la.num_seqs; i += COMBINE_FEW_THREADS) {
      const int c = la.cu_seqlens[i];
      if ((i == 0 && c != 0) || (i == la.num_seqs && (int64_t)c != la.T) ||
          (i < la.num_seqs && la.cu_seqlens[i + 1] < c))
        status |= LLP_STATUS_LAYOUT_INVALID;
    }
  const uint64_t on = few_scored(la);
  if (((on >> t) & 1) == 0) {
    if (threadIdx.x == 0) {
      la.out_t[t] = 0.f;
      la.out_f[t] = 0;
      la.out_l[t] = 0.f;
      if (la.out_e) la.out_e[t] = 0.f;
      if (la.out_p) la.out_p[t] = 0.f;
    }
  } else {
    const int j = __popcll(on & ((1ull << t) - 1));
    const int loc = few_target(la, t, status);
    const float target = loc >= 0 ? a.ca.tz[j] : 0.f;
    float M = -INFINITY, S = 0.f, Q = 0.f;
    if (a.ca.nvt <= COMBINE_FEW_TILES) {
      combine_few(a.ca, j, lds, M, S, Q);
    } else {
      // More tiles than the LDS takes: the chains read their partials themselves.
      const int c = threadIdx.x;
      if (c < COMBINE_CHAINS) {
        combine_chain(
            c, a.ca.nvt, [&](int vt) { return a.ca.pm[(int64_t)vt * a.ca.pstride + j]; },
            [&](int vt, float& m, float& s, float& q) {
              const int64_t o = (int64_t)vt * a.ca.pstride + j;
              m = a.ca.pm[o];
              s = a.ca.ps[o];
              q = a.ca.pq[o];
            },
            M, S, Q);
        lds.rm[c] = M;
        lds.rs[c] = S;
        lds.rq[c] = Q;
      }
      __syncthreads();
      M = -INFINITY; S = 0.f; Q = 0.f;
      if (threadIdx.x == 0)
        for (int g = 0; g < COMBINE_CHAINS; ++g) fold(M, S, Q, lds.rm[g], lds.rs[g], lds.rq[g]);
    }
    if (threadIdx.x == 0) combine_out(a.ca, t, loc >= 0, target, M, S, Q);
  }
  if (status && la.status) atomicOr(la.status, status);
}

template <int NB, int IB, int KS, int BUFS>
static void launch_few(const Fwd8Args& a, hipStream_t s) {
  const dim3 grid((unsigned)a.f.nvt), block(1024 / IB * KS);
  if (a.f.bias == nullptr) hipLaunchKernelGGL((k_fwd8_few<BIAS_NONE, NB, IB, KS, BUFS>), grid, block, 0, s, a);
  else if (a.f.bias_f32) hipLaunchKernelGGL((k_fwd8_few<BIAS_F32, NB, IB, KS, BUFS>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_fwd8_few<BIAS_BF16, NB, IB, KS, BUFS>), grid, block, 0, s, a);
}

hipError_t launch_fwd8_few(const Fwd8Args& a, hipStream_t s) {
  if (a.f.nvt > 0) {
    // Eight blocks of 16 columns per wave and two parts of K, in 4 waves, while the registers hold
    // them (151936 columns of 4096, us of a replayed call: 16 rows 119, with four parts 137; 32 rows
    // 119, with four parts 137, with four blocks a wave and one part 158; 48 rows 121, with the sums
    // of both parts in LDS, which leaves one workgroup per compute unit, 128, with four blocks a
    // wave 141); 64 rows with four blocks 140, in one part 151 (with eight they spill).
    if (a.la.T <= 16) launch_few<1, 8, 2, 2>(a, s);
    else if (a.la.T <= 32) launch_few<2, 8, 2, 2>(a, s);
    else if (a.la.T <= 48) launch_few<3, 8, 2, 1>(a, s);
    else launch_few<4, 4, 2, 2>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_fwd8_few_out, dim3((unsigned)a.la.T), dim3(COMBINE_FEW_THREADS), 0, s, a);
  return hipGetLastError();
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
