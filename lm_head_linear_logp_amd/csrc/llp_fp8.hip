// llp_fp8.hip -- operands in 8-bit floating point (e4m3) with an fp32 scale for each block of 128:
// their quantisation, their product (logits, input gradient) and the weight gradient.
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------------------
// Quantisation: scale = max(max |x|, 1e-30) * fl32(1/448) over 1 or 128 rows of 128 columns, q =
// x / scale as e4m3 (ties to even). By blocks, or transposed, a workgroup holds a 128 x 128 tile of x in
// registers, 8 x 8 values a thread, so that either costs one read and one write; the transpose goes
// through LDS and out in whole 128-byte rows. x, and a transposed q, go past the caches, which hold neither (90 ->
// 79 us in blocks, 376 -> 345 transposed in blocks, 107 -> 103 by group). Bound by memory: 37984 x 4096 bf16 (467 MB)
// in blocks 79 us, 5.9 TB/s; transposed 95; 4096 x 37984 by group 103, transposed in blocks 102, by group 107.
// (Maxima on the values' bits, moves between lanes instead of LDS shuffles, the hardware's reciprocal and bf16
// kept as it is loaded: together 15 % off.)
// ------------------------------------------------------------------------------------
constexpr int Q8_THREADS = 256;
// Groups from which a team takes four rows instead of one (us: 4096 x 4096 bf16 20.6 and 18.0, 16384 x 4096 51
// and 51, 37984 x 4096 110 and 119).
constexpr int64_t Q8_MANY_GROUPS = 1 << 19;

// Columns c .. c + 7 of a row, 0 at and past `cols`. VEC: rows are 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void q8_load(const void* row, int64_t c, int64_t cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    if constexpr (BF16) {
      const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + c));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_bit_cast(float, u[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
      }
    } else {
      const f32x4* const p = reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + c);
      const f32x4 lo = __builtin_nontemporal_load(p), hi = __builtin_nontemporal_load(p + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
      }
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

__device__ __forceinline__ uint2 q8_bytes(const float (&v)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Eight values as e4m3 of the correctly rounded quotient x / scale. With inv the reciprocal to 2^-23,
// x * inv is off from that quotient by at most 2^-22 of it; only where 2^-21 to either side gives
// another byte are the wave's divisions carried out. |quotient| <= 448 (1 + 2^-22), which
// rounds to 448.
__device__ __forceinline__ uint2 q8_pack(const float (&v)[8], float scale, float inv) {
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = v[i] * inv;
    lo[i] = fmaf(p, -0x1p-21f, p);
    hi[i] = fmaf(p, 0x1p-21f, p);
  }
  uint2 w = q8_bytes(lo);
  const uint2 u = q8_bytes(hi);
  if (__builtin_amdgcn_ballot_w64(w.x != u.x || w.y != u.y) != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = v[i] / scale;
    w = q8_bytes(lo);
  }
  return w;
}

// The largest size of values, as its bits: they order as whole numbers, an infinity above all finite
// values and a NaN above it.
__device__ __forceinline__ uint32_t q8_top(uint32_t top, float x) {
  const uint32_t m = __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
  return m > top ? m : top;
}
__device__ __forceinline__ uint32_t q8_max(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Over the 16 lanes of a team: rotations within rows of 16 lanes.
__device__ __forceinline__ uint32_t q8_team_top(uint32_t x) {
  x = q8_max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, false));
  x = q8_max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xf, 0xf, false));
  x = q8_max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xf, 0xf, false));
  return q8_max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xf, 0xf, false));
}

// Over the lanes l, l ^ 16, l ^ 32 and l ^ 48.
__device__ __forceinline__ uint32_t q8_teams_top(uint32_t x) {
  const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = q8_max(h[0], h[1]);
  const auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  return q8_max(q[0], q[1]);
}

// A block's scale, its reciprocal to 2^-23, and whether all of it is finite.
struct Q8Scale {
  float scale, inv;
  bool fine;
  __device__ __forceinline__ void of(uint32_t top) {
    fine = top < 0x7F800000u;
    scale = fmaxf(__builtin_bit_cast(float, top), 1e-30f) * (1.f / 448.f);
    inv = __builtin_amdgcn_rcpf(scale);
  }
  __device__ __forceinline__ float out() const { return fine ? scale : __builtin_nanf(""); }
};

// Eight values of a row as they were loaded: in bf16 two to a register, so that a thread's 64 leave room for
// twice the waves.
template <bool BF16>
struct __attribute__((aligned(16))) Q8Row {
  uint32_t u[BF16 ? 4 : 8];
  __device__ __forceinline__ float at(int i) const {
    if (!BF16) return __builtin_bit_cast(float, u[i]);
    return __builtin_bit_cast(float, (i & 1) != 0 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
  }
};

// A workgroup's tile. Transposed, neighbours go along the side with fewer tiles, so that one of the two walks, x's
// rows or q's, is whole pages of memory (us along columns and along rows, blocks: 4096 x 37984 111 and 103, 4096 x
// 151936 471 and 378, 37984 x 4096 100 and 113).
template <bool TRANS>
__device__ __forceinline__ void q8_place(const Quant8Args& a, int64_t& rb, int64_t& cb) {
  const int64_t ntr = (a.rows + 127) / 128, ntc = (a.cols + 127) / 128;
  const bool by_row = TRANS && ntr < ntc;
  rb = by_row ? blockIdx.x % ntr : blockIdx.x / ntc;
  cb = by_row ? blockIdx.x / ntr : blockIdx.x % ntc;
}

// Thread (team, lane): rows team * 8 .. + 7 and columns lane * 8 .. + 7 of a tile, 0 past x.
template <bool BF16, bool VEC>
__device__ __forceinline__ void q8_tile(const Quant8Args& a, int64_t r0, int64_t c0, Q8Row<BF16> (&v)[8]) {
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  const int64_t first = r0 + team * 8, c = c0 + lane * 8;
  const char* const x = static_cast<const char*>(a.x);
  constexpr int SIZE = BF16 ? 2 : 4, N = BF16 ? 4 : 8;
  if constexpr (VEC) {
    // No load is behind a lane's branch: rows past the last are read as the last, 8 columns past the last whole
    // ones as those, and the columns behind them, fewer than 8, one by one where the tile holds them.
    const int64_t whole = a.cols & ~(int64_t)7;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const char* const row = x + (first + p < a.rows ? first + p : a.rows - 1) * a.ldx * SIZE;
      if (whole > 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
        *reinterpret_cast<u32x4*>(&v[p].u[i]) =
            __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + (c < whole ? c : whole - 8) * SIZE + 4 * i));
      }
    }
    if (c0 + 128 > whole) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const char* const row = x + (first + p < a.rows ? first + p : a.rows - 1) * a.ldx * SIZE;
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t at = whole + i < a.cols ? whole + i : a.cols - 1;
          y[i] = BF16 ? reinterpret_cast<const uint16_t*>(row)[at] : reinterpret_cast<const uint32_t*>(row)[at];
          if (c > whole || whole + i >= a.cols) y[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c >= whole) v[p].u[i] = BF16 ? y[(2 * i) & 7] | y[(2 * i + 1) & 7] << 16 : y[i];
      }
    }
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) v[p].u[i] = first + p < a.rows ? v[p].u[i] : 0;
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (first + p < a.rows) q8_load<BF16, false>(x + (first + p) * a.ldx * SIZE, c, a.cols, y);
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[p].u[i] = BF16 ? __builtin_bit_cast(uint32_t, y[(2 * i) & 7]) >> 16 | __builtin_bit_cast(uint32_t, y[(2 * i + 1) & 7])
                         : __builtin_bit_cast(uint32_t, y[i]);
    }
  }
}

// Keeps the tile as it was loaded across what follows, not the fp32 values made of it.
template <bool BF16>
__device__ __forceinline__ void q8_keep(Q8Row<BF16> (&v)[8]) {
  if constexpr (BF16) {
#pragma unroll
    for (int p = 0; p < 8; ++p) asm volatile("" : "+v"(v[p].u[0]), "+v"(v[p].u[1]), "+v"(v[p].u[2]), "+v"(v[p].u[3]));
  }
}

// The tile's columns as rows of q, from LDS: 8-byte piece `team` of column c is at (team ^ (c / 8)) * 8 of its 128
// bytes, so that a wave's writes spread over the banks.
__device__ __forceinline__ void q8_turned_put(uint8_t* turned, int k, const uint2& w) {
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  *reinterpret_cast<uint2*>(turned + (lane * 8 + k) * 128 + (team ^ lane) * 8) = w;
}
__device__ __forceinline__ void q8_turned_store(const uint8_t* turned, const Quant8Args& a, int64_t r0, int64_t c0) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int c = p * 32 + (threadIdx.x >> 3), h = threadIdx.x & 7;   // column, 16-byte piece
    const uint2 lo = *reinterpret_cast<const uint2*>(turned + c * 128 + ((2 * h) ^ (c >> 3)) * 8);
    const uint2 hi = *reinterpret_cast<const uint2*>(turned + c * 128 + ((2 * h + 1) ^ (c >> 3)) * 8);
    if (c0 + c < a.cols)
      __builtin_nontemporal_store(u32x4{lo.x, lo.y, hi.x, hi.y}, reinterpret_cast<u32x4*>(a.q + (c0 + c) * a.ldq + r0 + 16 * h));
  }
}

template <bool BF16, bool VEC, bool BLOCK, bool TRANS>
__global__ __launch_bounds__(Q8_THREADS) void k_quant8(Quant8Args a) {
  static_assert(BLOCK || TRANS, "k_quant8_rows");
  __shared__ uint32_t tops[4][128];
  __shared__ __attribute__((aligned(16))) uint8_t turned[TRANS ? 128 * 128 : 16];
  int64_t rb, cb;
  q8_place<TRANS>(a, rb, cb);
  const int64_t r0 = rb * 128, c0 = cb * 128;
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  Q8Row<BF16> v[8];
  q8_tile<BF16, VEC>(a, r0, c0, v);
  uint32_t top[8];   // of this thread's columns, or of all in the first
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& t = top[BLOCK ? 0 : i];
      t = q8_top(t, v[p].at(i));
    }
  q8_keep(v);
  Q8Scale sc[BLOCK ? 1 : 8];
  if constexpr (BLOCK) {
    top[0] = q8_teams_top(q8_team_top(top[0]));
    if ((threadIdx.x & 63) == 0) tops[wave][0] = top[0];
    __syncthreads();
    sc[0].of(q8_max(q8_max(tops[0][0], tops[1][0]), q8_max(tops[2][0], tops[3][0])));
    if (threadIdx.x == 0) a.scale[TRANS ? cb * a.lds + rb : rb * a.lds + cb] = sc[0].out();
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top[i] = q8_teams_top(top[i]);
      if ((threadIdx.x & 63) < 16) tops[wave][lane * 8 + i] = top[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = lane * 8 + i;
      sc[i].of(q8_max(q8_max(tops[0][c], tops[1][c]), q8_max(tops[2][c], tops[3][c])));
      if (team == 0 && c0 + c < a.cols) a.scale[rb * a.lds + c0 + c] = sc[i].out();
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // Row k of this thread's 8 x 8 values, or its column k.
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = TRANS ? v[i].at(k) : v[k].at(i);
    const Q8Scale& own = sc[BLOCK ? 0 : k];
    uint2 w = q8_pack(x, own.scale, own.inv);
    if (!own.fine) w = make_uint2(0, 0);
    if constexpr (TRANS) {
      q8_turned_put(turned, k, w);
    } else {
      const int64_t r = r0 + team * 8 + k;
      if (r < a.rows) *reinterpret_cast<uint2*>(a.q + r * a.ldq + c0 + lane * 8) = w;
    }
  }
  if constexpr (TRANS) {
    __syncthreads();
    q8_turned_store(turned, a, r0, c0);
  }
}

// Both that a weight's gradient step takes of one x: a by group, t in blocks and transposed. One read instead of
// two (4096 x 37984 bf16: 108 and 103 us apart, 181 together, 622 MB at 3.4 TB/s; 4096 x 151936: 424 and 378, 590).
// Every value is packed twice, and a's rows are written 128 bytes at a time: short of a copy's 5.1 TB/s.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(Q8_THREADS) void k_quant8_both(Quant8Args a, Quant8Args t) {
  __shared__ uint32_t tops[4];
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
  int64_t rb, cb;
  q8_place<true>(a, rb, cb);
  const int64_t r0 = rb * 128, c0 = cb * 128;
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  Q8Row<BF16> v[8];
  q8_tile<BF16, VEC>(a, r0, c0, v);
  uint32_t all = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    uint32_t top = 0;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = v[p].at(i);
      top = q8_top(top, x[i]);
    }
    top = q8_team_top(top);
    all = q8_max(all, top);
    Q8Scale sc;
    sc.of(top);
    uint2 q = q8_pack(x, sc.scale, sc.inv);
    if (!sc.fine) q = make_uint2(0, 0);
    const int64_t r = r0 + team * 8 + p;
    if (r < a.rows) {
      *reinterpret_cast<uint2*>(a.q + r * a.ldq + c0 + lane * 8) = q;
      if (lane == 0) a.scale[cb * a.lds + r] = sc.out();
    }
  }
  q8_keep(v);
  all = q8_teams_top(all);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = all;
  __syncthreads();
  Q8Scale sc;
  sc.of(q8_max(q8_max(tops[0], tops[1]), q8_max(tops[2], tops[3])));
  if (threadIdx.x == 0) t.scale[cb * t.lds + rb] = sc.out();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i].at(k);
    uint2 q = q8_pack(x, sc.scale, sc.inv);
    if (!sc.fine) q = make_uint2(0, 0);
    q8_turned_put(turned, k, q);
  }
  __syncthreads();
  q8_turned_store(turned, t, r0, c0);
}

// By group and not transposed: 16 lanes a group and nothing shared; a team takes the same group of ROWS
// rows, whose scales are neighbours.
template <bool BF16, bool VEC, int ROWS>
__global__ __launch_bounds__(Q8_THREADS) void k_quant8_rows(Quant8Args a) {
  const int64_t groups = (a.cols + 127) / 128;
  const int64_t w = (int64_t)blockIdx.x * (Q8_THREADS / 16) + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  const int64_t r0 = w / groups * ROWS, g = w % groups;
  float v[ROWS][8];
#pragma unroll
  for (int p = 0; p < ROWS; ++p) {
    if (r0 + p < a.rows) {
      q8_load<BF16, VEC>(static_cast<const char*>(a.x) + (r0 + p) * a.ldx * (BF16 ? 2 : 4), g * 128 + lane * 8, a.cols, v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = 0.f;
    }
  }
#pragma unroll
  for (int p = 0; p < ROWS; ++p) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = q8_top(top, v[p][i]);
    Q8Scale sc;
    sc.of(q8_team_top(top));
    uint2 q = q8_pack(v[p], sc.scale, sc.inv);
    if (!sc.fine) q = make_uint2(0, 0);
    if (r0 + p < a.rows) {
      *reinterpret_cast<uint2*>(a.q + (r0 + p) * a.ldq + g * 128 + lane * 8) = q;
      if (lane == 0) a.scale[g * a.lds + r0 + p] = sc.out();
    }
  }
}

template <bool BF16, bool VEC, int ROWS>
static void launch_quant8_rows(const Quant8Args& a, hipStream_t s) {
  const int64_t teams = (a.rows + ROWS - 1) / ROWS * ((a.cols + 127) / 128);
  hipLaunchKernelGGL((k_quant8_rows<BF16, VEC, ROWS>), dim3((unsigned)((teams + 15) / 16)), dim3(Q8_THREADS), 0, s, a);
}

template <bool BF16, bool VEC>
static void launch_quant8_as(const Quant8Args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 127) / 128 * ((a.cols + 127) / 128)));
  if (a.block && a.transpose) hipLaunchKernelGGL((k_quant8<BF16, VEC, true, true>), grid, dim3(Q8_THREADS), 0, s, a);
  else if (a.block) hipLaunchKernelGGL((k_quant8<BF16, VEC, true, false>), grid, dim3(Q8_THREADS), 0, s, a);
  else if (a.transpose) hipLaunchKernelGGL((k_quant8<BF16, VEC, false, true>), grid, dim3(Q8_THREADS), 0, s, a);
  else if (a.rows * ((a.cols + 127) / 128) < Q8_MANY_GROUPS) launch_quant8_rows<BF16, VEC, 1>(a, s);
  else launch_quant8_rows<BF16, VEC, 4>(a, s);
}

hipError_t launch_quant8(const Quant8Args& a, hipStream_t s) {
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * (a.bf16 ? 2 : 4) % 16 == 0;
  if (a.bf16) vec ? launch_quant8_as<true, true>(a, s) : launch_quant8_as<true, false>(a, s);
  else vec ? launch_quant8_as<false, true>(a, s) : launch_quant8_as<false, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_quant8_both(const Quant8Args& a, const Quant8Args& t, hipStream_t s) {
  if (a.rows <= 0 || a.cols <= 0) return hipSuccess;
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * (a.bf16 ? 2 : 4) % 16 == 0;
  const dim3 grid((unsigned)((a.rows + 127) / 128 * ((a.cols + 127) / 128)));
  if (a.bf16 && vec) hipLaunchKernelGGL((k_quant8_both<true, true>), grid, dim3(Q8_THREADS), 0, s, a, t);
  else if (a.bf16) hipLaunchKernelGGL((k_quant8_both<true, false>), grid, dim3(Q8_THREADS), 0, s, a, t);
  else if (vec) hipLaunchKernelGGL((k_quant8_both<false, true>), grid, dim3(Q8_THREADS), 0, s, a, t);
  else hipLaunchKernelGGL((k_quant8_both<false, false>), grid, dim3(Q8_THREADS), 0, s, a, t);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// The product. A K step is one group of 128, a 128-byte line of every row: for a block of 16 x 16 one
// v_mfma_f32_16x16x128_f8f6f4 into accumulators that start at 0, then
//   acc = fma(sum of the group, x_scale * weight_scale, acc).
// MFMA operand A = weight rows (M), B = rows of x (N): a lane then holds one row of x per block, whose
// scale is one register, and the weight's scale is the same for all of a wave's rows (they lie in
// one block of 128), so a group costs one fma per element and one product per lane beside the
// matrix cores. The MFMA over the whole group leaves 4 sums per block to scale, where the 32 x 32
// form would hold 16 over two of them: that is what lets 128 x 64 outputs per wave fit 256 registers.
//
// v_mfma_f32_16x16x128_f8f6f4: lane l supplies 32 bytes of A[l % 16] and of B[l % 16] and holds
// D[4 (l / 16) + r][l % 16]. Which 32 of the 128 bytes a lane holds does not matter while A and B
// agree: 16-byte chunks 2 (l / 16) and the next of the line. Chunk c of row r sits at c ^ swz16(r) of its
// line: a ds_read_b128 serves 16 lanes at a time, of which half may be of the next 16-lane group, and
// with neighbouring groups two chunks apart those 16 fall on all banks once (chunks one apart, as a first
// form had them, conflicted in 45 % of the LDS's cycles).
//
// Precision. The e4m3 MFMAs (every form of them) add 8 products at a time cut towards zero at 2^-13
// of the largest one's power of two: measured on values drawn as activations are, a sum of 64 is
// 1.7e-5 of its norm off. That is a hundredth of bf16's rounding of most results, so those written in bf16 take
// it; but the cut goes by the products, not by their sum, and a result whose products nearly cancel keeps less
// (300 rows of 37984, 4096 deep: 1.7 % of the results are not the nearest bf16 value, 0.3 % a step or more off; of
// those below a hundredth of the rows' size, 0.8 % of them, a third). Results in fp32 (FULL) do not take it:
// their bytes become bf16 (exact) in front of the bf16 MFMA, whose sums keep fp32's bits, at half the matrix rate.
//
// Either way every tile runs the same chain for each element, its groups in the same order, so an element
// has the same bits whatever the tile and however many rows the call has.
// ------------------------------------------------------------------------------------
typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma8(const i32x8& a, const i32x8& b) {
  // Scales of 0: the form without block scales; formats 0: e4m3.
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// 16 e4m3 values as bf16, which holds them exactly: two MFMA operands of 8.
__device__ __forceinline__ void widen8(const i32x4& x, bf16x8 (&y)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)x[2 * k + i], 1.f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)x[2 * k + i], 1.f, true);
      y[k][4 * i] = lo[0]; y[k][4 * i + 1] = lo[1];
      y[k][4 * i + 2] = hi[0]; y[k][4 * i + 3] = hi[1];
    }
}

// 16 bytes (or 4) per lane from byte offset voff + soff into the LDS window at `lds`, lane order.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc8(const void* base, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0,
                                           (int)(uint32_t)(bytes < 0xFFFFFFFFull ? bytes : 0xFFFFFFFFull), 0x00020000);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, voff, 0, 0, 0);
}

// One value that a whole wave reads, as a scalar load: a vector load's wait would drain the loads in
// flight behind it.
__device__ __forceinline__ float scalar8(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

__device__ __forceinline__ int swz16(int row) { return (row ^ ((row >> 3) & 1)) & 7; }

// A workgroup's tile: TM weight rows x TN rows of x by WM x WN waves, NST stages in flight. A wave's
// accumulators are MB x NB blocks of S x S: 16 in bf16 results, 32 in fp32 ones.
// Groups of 128 are taken in turn from group (weight row / 1280) % groups on: workgroups that all read the
// same columns of rows 4096 bytes apart crowd a few of the memory's channels (1 row of 37984 x 4096: 37.0 us from
// column 0 on, 33.0 so; of 151936 119 and 107; 64 rows 132 and 123; rows of 8192 bytes 65 and 60. Rows of 1024, 2048
// and 5120 bytes: equal). The row is counted in the call's own weight. 1280: whole tiles of every form, so that a
// column's order of groups is the same in all of them.
constexpr int64_t TURN8 = 1280;
__device__ __forceinline__ int first_group8(int64_t v0, int n) { return n > 0 ? (int)(v0 / TURN8 % n) : 0; }

template <int TM, int TN, int WM, int WN, int NST, bool FULL>
struct Tile8 {
  static constexpr int S = FULL ? 32 : 16, REGS = S * S / 64;
  static constexpr int NW = WM * WN, ROWS = TM + TN;
  static constexpr int MW = TM / WM, NWV = TN / WN;            // a wave's rows of the weight and of x
  static constexpr int MB = MW / S, NB = NWV / S;
  static constexpr int NIA = TM / 8 / NW, NIB = TN / 8 / NW;   // loads per wave and step
  static constexpr int LOADS = NIA + NIB + 1;                  // and the scales'
  static constexpr int STAGE = ROWS * 128 + NW * 256;          // bytes
  static constexpr int OUT_LD = MW + 4;                        // floats per row of x of the output's staging
  static constexpr int OUT = NW * S * OUT_LD * 4;
  static constexpr int LDS = NST * STAGE > OUT ? NST * STAGE : OUT;
  // Where 16-byte chunk 0 of a row sits in its line; the others are exclusive-or'd with it.
  static __device__ __forceinline__ int swz(int row) { return FULL ? dma::swz8(row) : swz16(row); }
  typedef float Acc[MB][NB][REGS];
  static_assert(TM % (8 * NW) == 0 && TN % (8 * NW) == 0, "whole loads");
  static_assert(MW <= 128 && 128 % MW == 0, "a wave's rows lie in one block");
  static_assert(NWV <= 64 && LDS <= 160 * 1024, "scales by lane, LDS");
  static_assert((NST - 2) * LOADS < 64, "loads in flight");
};

// A wave's own LDS, written by some lanes and read by others.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// 16 bytes of a result; PAST: past the caches, for results far larger than they are, whose lines would
// push out operands that other tiles read (weight gradient of a shard: 538 -> 512 us).
template <bool PAST>
__device__ __forceinline__ void store16(uint16_t* p, const uint4& w) {
  const u32x4 v = {w.x, w.y, w.z, w.w};
  if constexpr (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = v;
}

// A wave's accumulators as rows of `out`: S rows of x at a time through the wave's own part of the
// LDS, from where each row's columns are stored together.
template <class T, bool PAST>
__device__ __forceinline__ void store_rows8(const typename T::Acc& acc, const Linear8Args& a, int64_t v0,
                                            int64_t t0, float* st) {
  const int lane = threadIdx.x & 63;
  const int64_t nv = a.V - v0;
  // 8 columns per lane.
  constexpr int LANES = T::MW / 8, STEP = 64 / LANES;
  const int c = lane % LANES * 8;
  float b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    b[i] = 0.f;
    if (a.bias != nullptr && c + i < nv)
      b[i] = a.bias_f32 ? static_cast<const float*>(a.bias)[v0 + c + i]
                        : bf16_to_f32(static_cast<const uint16_t*>(a.bias)[v0 + c + i]);
  }
#pragma unroll
  for (int ni = 0; ni < T::NB; ++ni) {
    wave_sync();
#pragma unroll
    for (int mi = 0; mi < T::MB; ++mi)
#pragma unroll
      for (int g = 0; g < T::REGS / 4; ++g) {
        float4 y;
        y.x = acc[mi][ni][4 * g]; y.y = acc[mi][ni][4 * g + 1];
        y.z = acc[mi][ni][4 * g + 2]; y.w = acc[mi][ni][4 * g + 3];
        *reinterpret_cast<float4*>(st + lane % T::S * T::OUT_LD + mi * T::S + 8 * g + 4 * (lane / T::S)) = y;
      }
    wave_sync();
#pragma unroll
    for (int j = 0; j < T::S; j += STEP) {
      const int row = j + lane / LANES;
      const int64_t t = t0 + ni * T::S + row;
      if (lane >= STEP * LANES || row >= T::S || t >= a.T) continue;
      const float* p = st + row * T::OUT_LD + c;
      const float4 lo = *reinterpret_cast<const float4*>(p), hi = *reinterpret_cast<const float4*>(p + 4);
      float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += b[i];
      }
      if constexpr (T::S == 16) {
        uint16_t* o = static_cast<uint16_t*>(a.out) + t * a.ldo + v0 + c;
        const uint4 w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                   pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        if (a.vec && c + 8 <= nv) {
          store16<PAST>(o, w);
        } else {
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < nv) o[i] = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
        }
      } else {
        float* o = static_cast<float*>(a.out) + t * a.ldo + v0 + c;
        if (a.vec && c + 8 <= nv) {
          *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(y[4], y[5], y[6], y[7]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < nv) o[i] = y[i];
        }
      }
    }
  }
}

// The weight gradient's layout, out[weight row][row of x]. In fp32 a register holds 32 neighbouring
// columns of one row per half wave, two whole lines: stored (and the old values added) from there. A
// buffer resource over each 32 rows (the host keeps a row's stride below 2^24 elements) drops what
// lies past the last row, and lanes past the last column point past it.
template <class T>
__device__ __forceinline__ void store_cols_f32(const typename T::Acc& acc, const Linear8Args& a, int64_t v0,
                                               int64_t t0) {
  static_assert(T::S == 32, "fp32 results");
  const int lane = threadIdx.x & 63;
  const uint32_t ld = (uint32_t)(a.ldo * 4);
#pragma unroll
  for (int mi = 0; mi < T::MB; ++mi) {
    const int64_t v = v0 + mi * 32;
    const int64_t left = a.V - v;
    if (left <= 0) break;
    const __amdgpu_buffer_rsrc_t r = rsrc8(static_cast<float*>(a.out) + v * a.ldo,
                                           (uint64_t)((left < 32 ? left : 32) - 1) * ld + (uint64_t)a.T * 4);
#pragma unroll
    for (int ni = 0; ni < T::NB; ++ni) {
      const int64_t h = t0 + ni * 32 + (lane & 31);
      const bool in = h < a.T;
      const uint32_t at = (uint32_t)h * 4 + (lane >> 5) * 4 * ld;
      auto place = [&](int k) { return (int)(in ? at + ((k >> 2) * 8 + (k & 3)) * ld : 0xFFFFFFFFu); };
      float old[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        old[k] = a.accumulate ? __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, place(k), 0, 0)) : 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        __builtin_amdgcn_raw_buffer_store_b32(
            __builtin_bit_cast(uint32_t, a.accumulate ? old[k] + acc[mi][ni][k] : acc[mi][ni][k]), r, place(k), 0, 0);
    }
  }
}

// In bf16 a block's rows are 32 bytes long: 16 rows of the wave at a time go through its part of the
// LDS and are stored as rows of all the wave's columns.
template <class T, bool PAST>
__device__ __forceinline__ void store_cols_bf16(const typename T::Acc& acc, const Linear8Args& a, int64_t v0,
                                                int64_t t0, float* st) {
  static_assert(T::S == 16, "bf16 results");
  constexpr int LD = T::NWV + 4, LANES = T::NWV / 8, STEP = 64 / LANES;
  static_assert(16 * LD <= T::S * T::OUT_LD, "within the wave's part");
  const int lane = threadIdx.x & 63;
  const int c = lane % LANES * 8;
  const int64_t nt = a.T - t0;
#pragma unroll
  for (int mi = 0; mi < T::MB; ++mi) {
    wave_sync();
#pragma unroll
    for (int ni = 0; ni < T::NB; ++ni)
#pragma unroll
      for (int r = 0; r < 4; ++r) st[(4 * (lane >> 4) + r) * LD + ni * 16 + (lane & 15)] = acc[mi][ni][r];
    wave_sync();
#pragma unroll
    for (int j = 0; j < 16; j += STEP) {
      const int64_t v = v0 + mi * 16 + j + lane / LANES;
      if (lane >= STEP * LANES || j + lane / LANES >= 16 || v >= a.V) continue;
      const float* p = st + (j + lane / LANES) * LD + c;
      const float4 lo = *reinterpret_cast<const float4*>(p), hi = *reinterpret_cast<const float4*>(p + 4);
      uint16_t* o = static_cast<uint16_t*>(a.out) + v * a.ldo + t0 + c;
      const uint32_t u[4] = {pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w), pack_bf16x2(hi.x, hi.y),
                             pack_bf16x2(hi.z, hi.w)};
      if (a.vec && c + 8 <= nt) {
        store16<PAST>(o, make_uint4(u[0], u[1], u[2], u[3]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < nt) o[i] = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

template <class T, bool GRAD, bool PAST>
__device__ __forceinline__ void store8(const typename T::Acc& acc, const Linear8Args& a, int64_t v0, int64_t t0,
                                       uint8_t* smem, int wave) {
  float* const st = reinterpret_cast<float*>(smem) + wave * T::S * T::OUT_LD;
  if constexpr (!GRAD) store_rows8<T, PAST>(acc, a, v0, t0, st);
  else if constexpr (T::S == 32) store_cols_f32<T>(acc, a, v0, t0);
  else store_cols_bf16<T, PAST>(acc, a, v0, t0, st);
}

template <class T>
__device__ __forceinline__ void zero8(typename T::Acc& acc) {
#pragma unroll
  for (int mi = 0; mi < T::MB; ++mi)
#pragma unroll
    for (int ni = 0; ni < T::NB; ++ni)
#pragma unroll
      for (int r = 0; r < T::REGS; ++r) acc[mi][ni][r] = 0.f;
}

// The plain form, NST steps in flight: few rows, which the weight's bytes bound (fp32, 1 row of 151936 x 4096:
// 106 us, 5.9 TB/s; 37 rows of 37984: 38, 4.1 TB/s, where x's lines take as much of the loads as the weight's),
// and fp32 results of many (4096 x 37984 x 4096: 1170 us, 1.09e15/s of 1.54e15 that the library's bf16
// product reaches).
template <int TM, int TN, int WM, int WN, int NST, bool GRAD, bool FULL, int EU>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(EU, EU))) void k_linear8(Linear8Args a) {
  using T = Tile8<TM, TN, WM, WN, NST, FULL>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[T::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  int vt, tb;
  vocab_token_tile(xcd_remap(blockIdx.x, gridDim.x), a.nvt, a.ntb, vt, tb);
  const int64_t v0 = (int64_t)vt * TM, t0 = (int64_t)tb * TN;
  const int nv = a.V - v0 < TM ? (int)(a.V - v0) : TM;
  const int nt = a.T - t0 < TN ? (int)(a.T - t0) : TN;
  const int n = a.steps;
  // The wave's loads: instruction i moves rows 8 q .. 8 q + 7, q = i NW + wave, lane l the 16-byte
  // chunk (l % 8) ^ swz(row) of row 8 q + l / 8. Rows past the last are read as the last.
  const __amdgpu_buffer_rsrc_t ra = rsrc8(a.W + v0 * a.ldw, (uint64_t)(nv - 1) * a.ldw + n * 128);
  const __amdgpu_buffer_rsrc_t rb = rsrc8(a.x + t0 * a.ldx, (uint64_t)(nt - 1) * a.ldx + n * 128);
  uint32_t va[T::NIA], vb[T::NIB];
#pragma unroll
  for (int i = 0; i < T::NIA; ++i) {
    const int r = 8 * (i * T::NW + wave) + (lane >> 3);
    va[i] = (uint32_t)((r < nv ? r : nv - 1) * a.ldw) + (((lane & 7) ^ T::swz(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < T::NIB; ++i) {
    const int r = 8 * (i * T::NW + wave) + (lane >> 3);
    vb[i] = (uint32_t)((r < nt ? r : nt - 1) * a.ldx) + (((lane & 7) ^ T::swz(r)) << 4);
  }
  const int ts = wn * T::NWV + lane % T::NWV;   // the row whose scale this lane loads
  const uint32_t vs = 4 * (ts < nt ? ts : nt - 1);
  const float* const xs = a.xs + t0;
  const int turn = first_group8(v0, n);
  auto group = [&](int s) { return s + turn < n ? s + turn : s + turn - n; };
  auto issue = [&](int step, int stage) {
    const int s = group(step);
    uint8_t* const st = smem + stage * T::STAGE;
#pragma unroll
    for (int i = 0; i < T::NIA; ++i) dma16(ra, st + (i * T::NW + wave) * 1024, va[i], s * 128);
#pragma unroll
    for (int i = 0; i < T::NIB; ++i) dma16(rb, st + TM * 128 + (i * T::NW + wave) * 1024, vb[i], s * 128);
    dma4(rsrc8(xs + s * a.ldxs, (uint64_t)nt * 4), st + T::ROWS * 128 + wave * 256, vs);
  };
  // A wave past the last row reads the last block's.
  const float* const ws = a.ws + (v0 + (wm * T::MW < nv ? wm * T::MW : nv - 1)) / 128 * a.ldws;
  // The lane's q-th chunk of its row of a block.
  auto chunk = [&](const uint8_t* st, int r0, int q) {
    const int r = r0 + lane % T::S;
    const int c = FULL ? 2 * q + lane / 32 : 2 * (lane / 16) + q;
    return *reinterpret_cast<const i32x4*>(st + r * 128 + ((c ^ T::swz(r)) << 4));
  };
  typename T::Acc acc;
  zero8<T>(acc);
  if (n > 0) {
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(s < n ? s : n - 1, s);
    int stage = 0, fill = NST - 1;
    for (int s = 0; s < n; ++s) {
      // Step s has landed, and every wave is past its reads of the stage that is filled next.
      dma::wait_vmem_le<(NST - 2) * T::LOADS>();
      dma::lds_barrier();
      issue(s + NST - 1 < n ? s + NST - 1 : n - 1, fill);
      const uint8_t* const sa = smem + stage * T::STAGE;
      const uint8_t* const sb = sa + TM * 128;
      const float* const sc = reinterpret_cast<const float*>(sa + T::ROWS * 128 + wave * 256);
      const float w = scalar8(ws + group(s));
      float scale[T::NB];
#pragma unroll
      for (int ni = 0; ni < T::NB; ++ni) scale[ni] = sc[ni * T::S + lane % T::S] * w;
      if constexpr (FULL) {
        f32x16 p[T::MB][T::NB];
#pragma unroll
        for (int mi = 0; mi < T::MB; ++mi)
#pragma unroll
          for (int ni = 0; ni < T::NB; ++ni)
#pragma unroll
            for (int r = 0; r < 16; ++r) p[mi][ni][r] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bf16x8 b[T::NB][2];
#pragma unroll
          for (int ni = 0; ni < T::NB; ++ni) widen8(chunk(sb, wn * T::NWV + ni * 32, q), b[ni]);
#pragma unroll
          for (int mi = 0; mi < T::MB; ++mi) {
            bf16x8 x[2];
            widen8(chunk(sa, wm * T::MW + mi * 32, q), x);
#pragma unroll
            for (int ni = 0; ni < T::NB; ++ni) {
              dma::mfma1(x[0], b[ni][0], p[mi][ni]);
              dma::mfma1(x[1], b[ni][1], p[mi][ni]);
            }
          }
        }
#pragma unroll
        for (int mi = 0; mi < T::MB; ++mi)
#pragma unroll
          for (int ni = 0; ni < T::NB; ++ni)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[mi][ni][r] = fmaf(p[mi][ni][r], scale[ni], acc[mi][ni][r]);
      } else {
        i32x8 b[T::NB];
#pragma unroll
        for (int ni = 0; ni < T::NB; ++ni)
          b[ni] = __builtin_shufflevector(chunk(sb, wn * T::NWV + ni * 16, 0), chunk(sb, wn * T::NWV + ni * 16, 1),
                                          0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int mi = 0; mi < T::MB; ++mi) {
          const i32x8 x = __builtin_shufflevector(chunk(sa, wm * T::MW + mi * 16, 0), chunk(sa, wm * T::MW + mi * 16, 1),
                                                  0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int ni = 0; ni < T::NB; ++ni) {
            const f32x4 p = mfma8(x, b[ni]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[mi][ni][r] = fmaf(p[r], scale[ni], acc[mi][ni][r]);
          }
        }
      }
      stage = stage + 1 < NST ? stage + 1 : 0;
      fill = fill + 1 < NST ? fill + 1 : 0;
    }
    dma::wait_vmem_le<0>();
    __syncthreads();   // the output's staging takes the stages' place
  }
  store8<T, GRAD, false>(acc, a, v0 + wm * T::MW, t0 + wn * T::NWV, smem, wave);
}

// The wide form of the bf16 results: 32 MB x 64 NB outputs by 8 waves of 16 MB x 16 NB, two per SIMD. The
// same chain with every read ahead of its use: 16 weight rows' NB MFMAs run while the next 16 are read and
// the sums before them are scaled; the next step's first fragments are read under the last rows'
// MFMAs. The barrier in front of those frees the step's stage, into which from there on a later step is
// loaded, one load after an MFMA (nine in a row hold up the wave's MFMAs: 5 % slower).
//
// 4096 x 37984 x 4096: 545 to 640 us over boxes and the clock that power leaves, 2.0 to 2.3e15/s; 4096 x 151936: 2.13
// to 2.26 ms, 2.3 to 2.4e15/s; the shard's gradients 480 to 535 (x) and 507 to 632 (weight); the library's
// product of the same bytes with one scale a matrix 517, 1769 and 384 (x). Bound by LDS and matrix
// cores alike: a step's operands are 196 KB of reads and 64 KB of writes, 2030 cycles at 128 bytes each, and its MFMAs
// 2048; eight waves of 128 x 64 are what the registers hold with sums that vector instructions scale.
template <int MB_, int NB_>
struct Wide8 {
  static constexpr int S = 16, REGS = 4, MB = MB_, NB = NB_;
  static constexpr int MW = 16 * MB, NWV = 16 * NB, TM = 2 * MW, TN = 4 * NWV;
  static constexpr int STAGE = (TM + TN) * 128, SCALES = TN * 4;
  static constexpr int FIT = 160 * 1024 / (STAGE + SCALES), NST = FIT < 4 ? FIT : 4;
  static constexpr int S0 = NST * STAGE;                       // where the scales' stages begin
  static constexpr int GROUPS = (TM + TN) / 8;                 // of 8 rows, one load each
  static constexpr int ROWS = (GROUPS + 7) / 8;                // loads of a wave and step,
  static constexpr int LOADS = ROWS + 1;                       // and the scales'
  static constexpr int OUT_LD = (MW > NWV ? MW : NWV) + 4;
  static constexpr int OUT = 8 * S * OUT_LD * 4;
  static constexpr int LDS = NST * (STAGE + SCALES) > OUT ? NST * (STAGE + SCALES) : OUT;
  static constexpr bool SPLIT = 128 % MW != 0;                 // a wave's rows may lie in two blocks of 128
  typedef float Acc[MB][NB][REGS];
  // Loads behind a row's MFMAs; the first three of a step come behind the last row's.
  static constexpr int EACH = NB < 3 ? NB : 3;
  static_assert(NST >= 2 && LDS <= 160 * 1024 && MW <= 128 && LOADS - 3 <= (MB - 1) * EACH && NB >= 2, "shape");
  static_assert(TURN8 % TM == 0, "one order of groups");
};

template <int MB, int NB, bool GRAD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_linear8_wide(Linear8Args a) {
  using T = Wide8<MB, NB>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[T::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  int vt, tb;
  vocab_token_tile(xcd_remap(blockIdx.x, gridDim.x), a.nvt, a.ntb, vt, tb);
  const int64_t v0 = (int64_t)vt * T::TM, t0 = (int64_t)tb * T::TN;
  const int nv = a.V - v0 < T::TM ? (int)(a.V - v0) : T::TM;
  const int nt = a.T - t0 < T::TN ? (int)(a.T - t0) : T::TN;
  const int n = a.steps;
  const __amdgpu_buffer_rsrc_t ra = rsrc8(a.W + v0 * a.ldw, (uint64_t)(nv - 1) * a.ldw + n * 128);
  const __amdgpu_buffer_rsrc_t rb = rsrc8(a.x + t0 * a.ldx, (uint64_t)(nt - 1) * a.ldx + n * 128);
  // Load k of a step moves 8 rows, the weight's in front of those of x; past the last the last again.
  // A step's last load is the scales' of 64 rows of x.
  uint32_t at[T::ROWS];
#pragma unroll
  for (int k = 0; k < T::ROWS; ++k) {
    const int g = k * 8 + wave < T::GROUPS ? k * 8 + wave : T::GROUPS - 1;
    const bool is_x = g >= T::TM / 8;
    const int r = 8 * g + (lane >> 3) - (is_x ? T::TM : 0), last = (is_x ? nt : nv) - 1;
    at[k] = (uint32_t)((r < last ? r : last) * (is_x ? a.ldx : a.ldw)) + (((lane & 7) ^ swz16(r)) << 4);
  }
  const int part = wave < NB ? wave : NB - 1;
  const int ts = part * 64 + lane;
  const uint32_t vs = 4 * (ts < nt ? ts : nt - 1);
  const float* const xs = a.xs + t0;
  const int turn = first_group8(v0, n);
  auto load = [&](int k, int s, int stage) {
    if (k < T::ROWS) {
      const int g = k * 8 + wave < T::GROUPS ? k * 8 + wave : T::GROUPS - 1;
      uint8_t* const to = smem + stage * T::STAGE + g * 1024;
      if (8 * (k + 1) <= T::TM / 8 || (8 * k < T::TM / 8 && g < T::TM / 8)) dma16(ra, to, at[k], s * 128);
      else dma16(rb, to, at[k], s * 128);
    } else {
      dma4(rsrc8(xs + s * a.ldxs, (uint64_t)nt * 4), smem + T::S0 + stage * T::SCALES + part * 256, vs);
    }
  };
  // Scales of the weight: those of the block of the wave's first row, and of the next (past the last row,
  // the last block's) from 16-row block `split` on.
  const int64_t r0 = v0 + wm * T::MW;
  const int64_t blk = r0 / 128, end = (a.V - 1) / 128;
  const int split = T::SPLIT ? (int)(128 - r0 % 128) / 16 : MB;
  const float* const ws = a.ws + (blk < end ? blk : end) * a.ldws;
  const float* const ws2 = a.ws + (blk + 1 < end ? blk + 1 : end) * a.ldws;
  // The lane's two chunks of its row of 16-row block i: at ad[0] and ad[1] + 2048 i of the weight's, bd of
  // x's.
  int ad[2], bd[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = lane & 15, c = r * 128 + (((2 * (lane >> 4) + q) ^ swz16(r)) << 4);
    ad[q] = wm * T::MW * 128 + c;
    bd[q] = (T::TM + wn * T::NWV) * 128 + c;
  }
  auto read = [&](const int (&p)[2], int so, int i) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(smem + (p[0] + so) + 2048 * i);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(smem + (p[1] + so) + 2048 * i);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  typename T::Acc acc;
  zero8<T>(acc);
  if (n > 0) {
    f32x4 p[NB];
    float sc[NB], last[NB];   // the rows' scales (times the weight's where there is one), and a block's before
#pragma unroll
    for (int ni = 0; ni < NB; ++ni) {
      p[ni] = f32x4{0.f, 0.f, 0.f, 0.f};
      last[ni] = 0.f;
    }
    auto upto = [&](int s) {   // the group of step s; past the last step the last again
      s = (s < n ? s : n - 1) + turn;
      return s < n ? s : s - n;
    };
#pragma unroll
    for (int s = 0; s < T::NST - 1; ++s)
#pragma unroll
      for (int k = 0; k < T::LOADS; ++k) load(k, upto(s), s);
#pragma unroll
    for (int k = 0; k < 3; ++k) load(k, upto(T::NST - 1), T::NST - 1);
    dma::wait_vmem_le<(T::NST - 2) * T::LOADS + 3>();
    dma::lds_barrier();
    i32x8 A[2], B[NB];
    const int sa = T::S0 + wn * T::NWV * 4 + (lane & 15) * 4;
    A[0] = read(ad, 0, 0);
    float w = scalar8(ws + turn), w2 = T::SPLIT ? scalar8(ws2 + turn) : 0.f;
#pragma unroll
    for (int ni = 0; ni < NB; ++ni) {
      B[ni] = read(bd, 0, ni);
      sc[ni] = *reinterpret_cast<const float*>(smem + sa + ni * 64);
      if (!T::SPLIT) sc[ni] *= w;
    }
    auto promote = [&](float (&c)[4], const f32x4& q, float f) {
#pragma unroll
      for (int r = 0; r < 4; ++r) c[r] = fmaf(q[r], f, c[r]);
      // The sums are taken here: without this the compiler puts all of a step's fmas at its end, and
      // every block's sums into registers until then (184 spilled).
      asm volatile("" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
    };
    auto scale = [&](int mi, int ni) { return T::SPLIT ? sc[ni] * (mi < split ? w : w2) : sc[ni]; };
    int stage = 0, fill = T::NST - 1;
    for (int s = 0; s < n; ++s) {
      const int next = stage + 1 < T::NST ? stage + 1 : 0, so = stage * T::STAGE, sn = next * T::STAGE;
      const float wn1 = scalar8(ws + upto(s + 1)), wn2 = T::SPLIT ? scalar8(ws2 + upto(s + 1)) : 0.f;
      const int k1 = upto(s + T::NST - 1), k2 = upto(s + T::NST);
#pragma unroll
      for (int mi = 0; mi < MB - 1; ++mi) {
        A[(mi + 1) & 1] = read(ad, so, mi + 1);
#pragma unroll
        for (int ni = 0; ni < NB; ++ni) {
          if (mi == 0) promote(acc[MB - 1][ni], p[ni], last[ni]);
          else promote(acc[mi - 1][ni], p[ni], scale(mi - 1, ni));
          p[ni] = mfma8(A[mi & 1], B[ni]);
          const int k = 3 + mi * T::EACH + ni;
          if (ni < T::EACH && k < T::LOADS) load(k, k1, fill);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // Step s + 1 has landed, and every wave holds the last of step s.
      dma::wait_vmem_le<(T::NST - 2) * T::LOADS>();
      dma::lds_barrier();
      i32x8 first = read(ad, sn, 0);
#pragma unroll
      for (int ni = 0; ni < NB; ++ni) {
        promote(acc[MB - 2][ni], p[ni], scale(MB - 2, ni));
        p[ni] = mfma8(A[(MB - 1) & 1], B[ni]);
        B[ni] = read(bd, sn, ni);
        if (ni < 3) load(ni, k2, stage);
        if (NB == 2 && ni == 1) load(2, k2, stage);
        __builtin_amdgcn_sched_barrier(0);
      }
      A[0] = first;
#pragma unroll
      for (int ni = 0; ni < NB; ++ni) {
        last[ni] = scale(MB - 1, ni);
        sc[ni] = *reinterpret_cast<const float*>(smem + sa + next * T::SCALES + ni * 64);
        if (!T::SPLIT) sc[ni] *= wn1;
      }
      w = wn1;
      w2 = wn2;
      fill = stage;
      stage = next;
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int ni = 0; ni < NB; ++ni) promote(acc[MB - 1][ni], p[ni], last[ni]);
    dma::wait_vmem_le<0>();
    __syncthreads();   // the output's staging takes the stages' place
  }
  store8<T, GRAD, true>(acc, a, r0, t0 + wn * T::NWV, smem, wave);
}

template <int TM, int TN, int WM, int WN, int NST, bool GRAD, bool FULL, int EU>
static hipError_t launch_linear8_as(Linear8Args a, hipStream_t s) {
  a.nvt = (int32_t)((a.V + TM - 1) / TM);
  a.ntb = (int32_t)((a.T + TN - 1) / TN);
  hipLaunchKernelGGL((k_linear8<TM, TN, WM, WN, NST, GRAD, FULL, EU>), dim3((unsigned)(a.nvt * a.ntb)),
                     dim3(64 * WM * WN), 0, s, a);
  return hipGetLastError();
}

template <int MB, int NB, bool GRAD>
static hipError_t launch_linear8_wide(Linear8Args a, hipStream_t s) {
  using T = Wide8<MB, NB>;
  a.nvt = (int32_t)((a.V + T::TM - 1) / T::TM);
  a.ntb = (int32_t)((a.T + T::TN - 1) / T::TN);
  hipLaunchKernelGGL((k_linear8_wide<MB, NB, GRAD>), dim3((unsigned)(a.nvt * a.ntb)), dim3(512), 0, s, a);
  return hipGetLastError();
}

// The wide form's shape. A compute unit holds one workgroup, so a call takes as long as its rounds of 256
// workgroups times what one takes: in units of a block's MFMA its MB NB, 10 for a step's other work and 2
// where a wave's rows lie in two of the weight's blocks (every shape measured at 40 sizes: the one that the rule
// takes is 0.6 % slower than the best of them on average, 12 % at most, 180 rows of 18992 x 2048). us of a shard, 37984 x 4096, with the shape it
// takes and with 8 x 4: 128 rows 37 and 59, 180 rows 42 and 60, 300 rows 56 and 102, 512 rows 91 and 108, 600
// rows 104 and 114.
template <bool GRAD>
static hipError_t launch_linear8_bf16(const Linear8Args& a, hipStream_t s) {
  int64_t least = 0;
  int mb = 8, nb = 4;
  for (int m : {8, 5, 4})
    for (int n : {5, 4, 3, 2}) {
      if (m * n > 32) continue;   // accumulators past the registers
      const int64_t tiles = (a.V + 32 * m - 1) / (32 * m) * ((a.T + 64 * n - 1) / (64 * n));
      const int64_t cost = (tiles + 255) / 256 * (m * n + 10 + (m == 5 ? 2 : 0));
      if (least == 0 || cost < least) {
        least = cost;
        mb = m;
        nb = n;
      }
    }
  switch (mb * 10 + nb) {
    case 42: return launch_linear8_wide<4, 2, GRAD>(a, s);
    case 43: return launch_linear8_wide<4, 3, GRAD>(a, s);
    case 44: return launch_linear8_wide<4, 4, GRAD>(a, s);
    case 45: return launch_linear8_wide<4, 5, GRAD>(a, s);
    case 52: return launch_linear8_wide<5, 2, GRAD>(a, s);
    case 53: return launch_linear8_wide<5, 3, GRAD>(a, s);
    case 54: return launch_linear8_wide<5, 4, GRAD>(a, s);
    case 55: return launch_linear8_wide<5, 5, GRAD>(a, s);
    case 82: return launch_linear8_wide<8, 2, GRAD>(a, s);
    case 83: return launch_linear8_wide<8, 3, GRAD>(a, s);
    default: return launch_linear8_wide<8, 4, GRAD>(a, s);
  }
}

hipError_t launch_linear8(const Linear8Args& a, hipStream_t s) {
  if (a.T <= 0 || a.V <= 0) return hipSuccess;
  // Results that two tiles of 64 x 64 a compute unit hold: latency, so the smallest tiles (us, these and the forms
  // below, 4096 deep unless noted: 64 rows of 4096 fp32 20 and 24, bf16 15 and 17; 200 rows of 4096 fp32 23 and 39,
  // bf16 16 and 23, 37984 deep 114 and 162; with 600 tiles and more they are slower, 200 rows of 9000 bf16 29 and 23).
  if ((a.grad || a.T > 32) && (a.V + 63) / 64 * ((a.T + 63) / 64) <= 512) {
    if (a.grad) return a.out_bf16 ? launch_linear8_as<64, 64, 2, 2, 3, true, false, 2>(a, s)
                                  : launch_linear8_as<64, 64, 2, 2, 3, true, true, 2>(a, s);
    return a.out_bf16 ? launch_linear8_as<64, 64, 2, 2, 3, false, false, 2>(a, s)
                      : launch_linear8_as<64, 64, 2, 2, 3, false, true, 2>(a, s);
  }
  if (a.grad) {
    if (a.out_bf16) return launch_linear8_bf16<true>(a, s);
    return launch_linear8_as<128, 128, 2, 2, 2, true, true, 2>(a, s);
  }
  // Few rows, the weight's bytes bound them: 64 or 128 columns a workgroup, whichever leaves the busiest of 256
  // compute units fewer columns, 128 where they are alike, and from 65536 on (us of 4096 deep fp32, 64 and 128
  // columns: 1 row of 16384 19.9 and 22.1, of 24000 24.8 and 23.0, of 33500 31.4 and 35.4, of 37984 32.8 and 36.5, of
  // 48000 38.6 and 40.7, of 50000 43.8 and 40.6, of 70000 60.2 and 61.9, of 98304 76.4 and 70.7; 33 rows of 37984 38.2
  // and 42.4, of 48000 41.7 and 45.0, of 50000 55.8 and 45.2, of 65536 64.4 and 52.6; alike in bf16 and 2048 deep). More
  // steps in flight (4 to 6) or 256 columns are no faster.
  const bool narrow = a.V < 65536 && (a.V + 16383) / 16384 % 2 != 0;
  if (a.out_bf16) {
    if (a.T <= 32) return narrow ? launch_linear8_as<64, 32, 2, 1, 3, false, false, 2>(a, s)
                                 : launch_linear8_as<128, 32, 4, 1, 3, false, false, 2>(a, s);
    if (a.T <= 64) return narrow ? launch_linear8_as<64, 64, 2, 1, 3, false, false, 2>(a, s)
                                 : launch_linear8_as<128, 64, 4, 1, 3, false, false, 2>(a, s);
    return launch_linear8_bf16<false>(a, s);
  }
  if (a.T <= 32) return narrow ? launch_linear8_as<64, 32, 2, 1, 3, false, true, 2>(a, s)
                               : launch_linear8_as<128, 32, 4, 1, 3, false, true, 2>(a, s);
  if (a.T <= 64) return narrow ? launch_linear8_as<64, 64, 2, 1, 3, false, true, 2>(a, s)
                               : launch_linear8_as<128, 64, 4, 1, 3, false, true, 2>(a, s);
  return launch_linear8_as<128, 128, 2, 2, 2, false, true, 2>(a, s);
}

}  // namespace llp
