// llp_beam.hip -- one step of a beam search: the most likely tokens of every row of logits, the
// selection over a sequence's beams and shards, and the reordering of what is kept per beam.
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

#include <type_traits>

namespace llp {

// ------------------------------------------------------------------------------------
// Ordered keys. A value and its place become one number that is larger the better the candidate:
// the value's bits in an order that compares as unsigned, then the place inverted, so that no two
// candidates are equal and ties go to the lowest place. 0 is no candidate.
// ------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);   // -0 is 0
  return u ^ ((u >> 31) != 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// The value of lane l ^ J, without the LDS's latency: moves within rows of 16 lanes, swaps of rows
// and of halves. (A sort of 64 keys through ds_bpermute took about 2700 cycles, so about 1000.)
template <int J>
__device__ __forceinline__ uint32_t across(uint32_t x) {
  if constexpr (J == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, false);       // quad 1 0 3 2
  else if constexpr (J == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, false);  // quad 2 3 0 1
  else if constexpr (J == 4) {
    const int up = __builtin_amdgcn_update_dpp(0, (int)x, 0x104, 0xf, 0x5, false);                             // row_shl:4
    return (uint32_t)__builtin_amdgcn_update_dpp(up, (int)x, 0x114, 0xf, 0xA, false);                          // row_shr:4
  } else if constexpr (J == 8) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, false);  // row_ror:8
  else if constexpr (J == 16) {
    const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (threadIdx.x & 16) != 0 ? y[0] : y[1];
  } else {
    const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return (threadIdx.x & 32) != 0 ? y[0] : y[1];
  }
}
template <int J>
__device__ __forceinline__ float across(float x) {
  return __builtin_bit_cast(float, across<J>(__builtin_bit_cast(uint32_t, x)));
}

__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, across<1>(x));
  x = fmaxf(x, across<2>(x));
  x = fmaxf(x, across<4>(x));
  x = fmaxf(x, across<8>(x));
  x = fmaxf(x, across<16>(x));
  return fmaxf(x, across<32>(x));
}
__device__ __forceinline__ double wave_sum(double x) {
  auto add = [&](auto j) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = across<decltype(j)::value>((uint32_t)u), hi = across<decltype(j)::value>((uint32_t)(u >> 32));
    x += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  add(std::integral_constant<int, 1>());
  add(std::integral_constant<int, 2>());
  add(std::integral_constant<int, 4>());
  add(std::integral_constant<int, 8>());
  add(std::integral_constant<int, 16>());
  add(std::integral_constant<int, 32>());
  return x;
}

struct Key64 {   // logit, column
  uint64_t k;
  __device__ __forceinline__ bool above(const Key64& o) const { return k > o.k; }
  __device__ __forceinline__ Key64 from(int lane) const {
    const int lo = __shfl((int)(uint32_t)k, lane), hi = __shfl((int)(k >> 32), lane);
    return {(uint64_t)(uint32_t)hi << 32 | (uint32_t)lo};
  }
  template <int J>
  __device__ __forceinline__ Key64 other() const {
    return {(uint64_t)across<J>((uint32_t)(k >> 32)) << 32 | across<J>((uint32_t)k)};
  }
  __device__ __forceinline__ bool any() const { return k != 0; }
  static __device__ __forceinline__ Key64 none() { return {0}; }
};

struct Key128 {   // total, then beam and token
  uint64_t k, at;
  __device__ __forceinline__ bool above(const Key128& o) const { return k > o.k || (k == o.k && at > o.at); }
  __device__ __forceinline__ Key128 from(int lane) const {
    const Key64 a = Key64{k}.from(lane), b = Key64{at}.from(lane);
    return {a.k, b.k};
  }
  template <int J>
  __device__ __forceinline__ Key128 other() const {
    const Key64 a = Key64{k}.other<J>(), b = Key64{at}.other<J>();
    return {a.k, b.k};
  }
  __device__ __forceinline__ bool any() const { return k != 0; }
  static __device__ __forceinline__ Key128 none() { return {0, 0}; }
};

struct Key32 {   // a logit alone
  uint32_t k;
  __device__ __forceinline__ bool above(const Key32& o) const { return k > o.k; }
  template <int J>
  __device__ __forceinline__ Key32 other() const { return {across<J>(k)}; }
};

// One step of a bitonic network: runs of SIZE lanes are left largest first, every other one last.
template <int SIZE, int J, class K>
__device__ __forceinline__ void exchange(K& x) {
  const int lane = threadIdx.x & 63;
  const K y = x.template other<J>();
  // The lower lane of a pair takes the larger key in a descending run.
  const bool larger = ((lane & J) == 0) == ((lane & SIZE) == 0 || SIZE == 64);
  if (y.above(x) == larger) x = y;
}
template <int SIZE, int J, class K>
__device__ __forceinline__ void exchanges(K& x) {
  exchange<SIZE, J>(x);
  if constexpr (J > 1) exchanges<SIZE, J / 2>(x);
}

// The wave's 64 keys, largest first.
template <class K>
__device__ __forceinline__ K sort64(K x) {
  exchanges<2, 1>(x);
  exchanges<4, 2>(x);
  exchanges<8, 4>(x);
  exchanges<16, 8>(x);
  exchanges<32, 16>(x);
  exchanges<64, 32>(x);
  return x;
}

// The 64 largest of two runs of 64, each largest first.
template <class K>
__device__ __forceinline__ K merge64(K x, K y) {
  y = y.from(63 - (threadIdx.x & 63));
  if (y.above(x)) x = y;
  exchanges<64, 32>(x);
  return x;
}

// A wave's best `num` keys so far: sorted in its lanes, and up to 63 later ones in LDS that are
// above the worst of them as it was when it was last looked at.
template <class K>
struct Best {
  K list;      // lane i: the i-th largest
  K bar;       // only larger keys can still enter
  K* buf;      // [128] of LDS, this wave's
  int held;    // keys in buf

  __device__ __forceinline__ void init(K* b) {
    list = bar = K::none();
    buf = b;
    held = 0;
  }
  __device__ __forceinline__ void fold(int n, int num) {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const K x = lane < n ? buf[lane] : K::none();
    list = merge64(list, sort64(x));
    const K b = list.from(num - 1);
    if (b.above(bar)) bar = b;
  }
  // Each lane's key, where it is above the bar. Called by the whole wave.
  __device__ __forceinline__ void add(K x, int num) {
    const int lane = threadIdx.x & 63;
    const bool in = x.above(bar);
    const uint64_t m = __builtin_amdgcn_ballot_w64(in);
    if (m == 0) return;
    if (in) buf[held + __popcll(m & ((1ull << lane) - 1))] = x;
    held += __popcll(m);
    if (held < 64) return;
    fold(64, num);
    held -= 64;
    K y = K::none();
    if (lane < held) y = buf[64 + lane];
    __builtin_amdgcn_wave_barrier();
    if (lane < held) buf[lane] = y;
  }
  __device__ __forceinline__ void finish(int num) {
    if (held > 0) fold(held, num);
    held = 0;
  }
};

// ------------------------------------------------------------------------------------
// Candidates: a workgroup a row. Each wave takes blocks of 2048 columns, 32 values a lane in registers,
// and leaves the sum of the block's exponentials and the largest value of each 16 lanes' 512, a piece, in
// LDS (so the row's normaliser does not depend on how many waves share it). The num-th largest of some
// pieces' maxima is a bar that num values reach: only the pieces whose maximum reaches it, few more
// than num, are read again for the values that do, and sorted.
//
// Bound by memory with many rows: one read of the logits, past the caches (512 rows of 151669 fp32 columns, 311
// MB: 58 us, 5.4 TB/s). With few, a row is one compute unit's, and its exponentials and their sums bound it (4
// rows: 19 us; 80 bf16 rows of a shard of 37984: 11). Several workgroups a row and a second launch that joins them
// took 7.3 + 6 us on the device for 4 rows (where this form, with sums in fp32, took 17; 62 + 6 for the 512, 10 +
// 4.6 for the 80), but 17.8 instead of 10.9 us a call on the host, which bounds a beam search's step.
//
// exp((x - max) c) as 2^t, t = (x - max) c log2 e with the constant in two parts: its rounding would shift
// every term alike, by 2e-7 for the bulk of a row. A term e in fp32 is off by an ulp of the exponential and by t's
// two roundings, 2^-23 e (1 + (max - x) c) together at most; a block's largest is 1 exactly. Sums are in fp64:
// in fp32 a token with most of a row's mass takes the last bits of all that is added to it (measured up to 2.9e-7
// of the sum; fp64 costs 5 to 11 % of the time with few rows, 1 to 5 % with many). What is left is at most 2^-23
// of the mass beside the largest token times that factor (measured: flat rows 3e-9 of the sum, 12 likely tokens 2e-9
// to 7e-9 rms, 5001 columns of one lower value 4e-8).
// ------------------------------------------------------------------------------------
constexpr int BEAM_WAVES = 16;   // of a workgroup, at most
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ float beam_value(const void* row, int64_t c) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[c]) : static_cast<const float*>(row)[c];
}
// 32 values of a lane, a block's 16 bytes at c0, c0 + 1024, ..: -inf past the last column. No load is
// conditional per lane (each would be waited for by itself: 32 in a row, 20 us): past the last whole 16
// bytes the last are loaded again, and the columns behind them, fewer than 16 bytes, come one by
// one for all lanes.
template <bool BF16>
__device__ __forceinline__ void beam_load(const void* row, int64_t c0, int64_t n_real, float (&x)[32]) {
  constexpr int V = BF16 ? 8 : 4;   // values per 16 bytes
  const int64_t whole = n_real / V * V;
  if (whole > 0) {
#pragma unroll
    for (int i = 0; i < 32 / V; ++i) {
      const int64_t c = c0 + i * 64 * V;
      const int64_t at = c < whole ? c : whole - V;
      if constexpr (BF16) {
        const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + at));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[i * V + 2 * k] = __builtin_bit_cast(float, u[k] << 16);
          x[i * V + 2 * k + 1] = __builtin_bit_cast(float, u[k] & 0xFFFF0000u);
        }
      } else {
        const f32x4 u = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + at));
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i * V + k] = u[k];
      }
    }
  }
  if (__builtin_amdgcn_ballot_w64(c0 + (32 / V - 1) * 64 * V >= whole) != 0) {
    float rest[V];
#pragma unroll
    for (int k = 0; k < V; ++k) rest[k] = beam_value<BF16>(row, whole + k < n_real ? whole + k : n_real - 1);
#pragma unroll
    for (int i = 0; i < 32 / V; ++i) {
      const int64_t c = c0 + i * 64 * V;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c >= whole) x[i * V + k] = c + k < n_real ? rest[k] : -INFINITY;
    }
  }
}

// LDS of a row: keys that wait for each wave, each wave's best, the blocks' sums, the pieces' largest values
// and the pieces to read again (64 KB at most).
static size_t beam_lds(int waves, int blocks) { return (size_t)waves * 192 * sizeof(Key64) + (size_t)blocks * 32; }

template <bool BF16>
__global__ __launch_bounds__(64 * BEAM_WAVES) void k_beam_rows(BeamArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ float shared_bar;
  __shared__ int shared_bad, shared_count;
  constexpr int V = BF16 ? 8 : 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6, pieces = 4 * a.blocks;
  Key64* const room = reinterpret_cast<Key64*>(smem);
  Key64* const lists = room + waves * 128;
  double* const sums = reinterpret_cast<double*>(lists + waves * 64);
  float* const tops = reinterpret_cast<float*>(sums + a.blocks);
  uint16_t* const reread = reinterpret_cast<uint16_t*>(tops + pieces);   // the host keeps pieces at 4096
  const int64_t r = blockIdx.x;
  const char* const row = static_cast<const char*>(a.logits) + r * a.ld * (BF16 ? 2 : 4);
  const double cl = (double)a.c1 * 1.4426950408889634074;
  // The high part is the smaller one, so that the low part is above 0 and -inf times it is -inf.
  const float near = (float)cl;
  const float ch = (double)near < cl ? near : __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, near) - 1);
  const float clo = (float)(cl - (double)ch);
  for (int b = wave; b < a.blocks; b += waves) {
    float x[32];
    beam_load<BF16>(row, (int64_t)b * BEAM_BLOCK + lane * V, a.n_real, x);
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; ++e) top = fmaxf(top, x[e]);
    top = fmaxf(top, across<1>(top));
    top = fmaxf(top, across<2>(top));
    top = fmaxf(top, across<4>(top));
    top = fmaxf(top, across<8>(top));
    if ((lane & 15) == 0) tops[4 * b + (lane >> 4)] = top;
    top = fmaxf(top, across<16>(top));
    top = fmaxf(top, across<32>(top));
    // A NaN, which the maxima pass over, or +inf makes the sum NaN.
    const float base = top > -INFINITY ? top : 0.f;
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float d = x[e] - base;
      s[e & 1] += (double)__builtin_amdgcn_exp2f(fmaf(d, ch, d * clo));
    }
    const double sum = wave_sum(s[0] + s[1]);
    if (lane == 0) sums[b] = sum;
  }
  __syncthreads();
  if (wave == 0) {
    float most = -INFINITY;
    for (int i = lane; i < pieces; i += 64) most = fmaxf(most, tops[i]);
    const Key32 m = sort64(Key32{most > -INFINITY ? ordered(most) : 0});
    const uint32_t at = (uint32_t)__shfl((int)m.k, a.num - 1);
    const float bar = at != 0 ? unordered(at) : -INFINITY;
    int n = 0;
    for (int i = 0; i < pieces; i += 64) {
      const float top = i + lane < pieces ? tops[i + lane] : -INFINITY;
      const bool in = top >= bar && top > -INFINITY;
      const uint64_t all = __builtin_amdgcn_ballot_w64(in);
      if (in) reread[n + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)(i + lane);
      n += __popcll(all);
    }
    if (lane == 0) {
      shared_bar = bar;
      shared_count = n;
    }
  }
  if (wave == waves - 1) {
    float M = -INFINITY;
    bool bad = false;
    for (int i = lane; i < pieces; i += 64) M = fmaxf(M, tops[i]);
    for (int i = lane; i < a.blocks; i += 64) bad |= __builtin_isnan(sums[i]);
    M = wave_max(M);
    bad = __builtin_amdgcn_ballot_w64(bad) != 0;
    double S = 0.0;
    if (!bad && M > -INFINITY) {
      for (int i = lane; i < a.blocks; i += 64) {
        const float m = fmaxf(fmaxf(tops[4 * i], tops[4 * i + 1]), fmaxf(tops[4 * i + 2], tops[4 * i + 3]));
        if (m > -INFINITY) S += sums[i] * exp(((double)m - (double)M) * (double)a.c1);
      }
      S = wave_sum(S);
    }
    if (lane == 0) {
      shared_bad = bad;
      a.max[r] = bad ? -INFINITY : M;
      a.sum[r] = bad ? -1.0 : S;
      if (bad && a.status) atomicOr(a.status, LLP_STATUS_VALUE_NOT_FINITE);
    }
  }
  __syncthreads();
  const float bar = shared_bar;
  const bool bad = shared_bad != 0;
  Best<Key64> best;
  best.init(room + wave * 128);
  if (bar > -INFINITY) best.bar = Key64{((uint64_t)ordered(bar) << 32) - 1};
  // Four pieces at a time, 16 lanes each; lanes without one repeat the first.
  const int count = bad ? 0 : shared_count;
  for (int i = wave * 4; i < count; i += waves * 4) {
    const int mine = i + (lane >> 4);
    const bool has = mine < count;
    const int q = reread[has ? mine : i];
    const int64_t c0 = (int64_t)(q >> 2) * BEAM_BLOCK + ((q & 3) * 16 + (lane & 15)) * V;
    float x[32];
    beam_load<BF16>(row, c0, a.n_real, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const bool may = has && x[e] >= bar && x[e] > -INFINITY;
      if (__builtin_amdgcn_ballot_w64(may) == 0) continue;
      const uint32_t c = (uint32_t)c0 + (e / V) * 64 * V + e % V;
      best.add(Key64{may ? (uint64_t)ordered(x[e]) << 32 | (uint32_t)~c : 0}, a.num);
    }
  }
  best.finish(a.num);
  // Half of the waves that read pieces hand their best to the others until one wave holds the row's.
  const int active = (count + 3) / 4 < waves ? (count + 3) / 4 : waves;
  lists[wave * 64 + lane] = best.list;
  __syncthreads();
  for (int step = 1; step < active; step *= 2) {
    if (wave % (2 * step) == 0 && wave + step < active) {
      best.list = merge64(best.list, lists[(wave + step) * 64 + lane]);
      lists[wave * 64 + lane] = best.list;
    }
    __syncthreads();
  }
  if (wave == 0 && lane < a.num) {
    const bool in = best.list.any();
    a.value[r * a.num + lane] = in ? unordered((uint32_t)(best.list.k >> 32)) : -INFINITY;
    a.token[r * a.num + lane] = in ? a.offset + (int64_t)(uint32_t)~(uint32_t)best.list.k : -1;
  }
}

hipError_t launch_beam_candidates(const BeamArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  // Waves on a row: a compute unit holds 20 (us a call for 4, 8 and 16 waves: 4 rows of 151669 fp32 26, 21 and 20;
  // 512 rows 59, 60 and 64; 1000 rows 111, 107 and 120; of 37917 bf16 512 rows 23, 19 and 26, 2000 rows 50, 61 and 91).
  int waves = a.rows <= 256 ? 16 : a.rows <= 1024 ? 8 : 4;
  if (waves > a.blocks) waves = a.blocks > 0 ? a.blocks : 1;
  const dim3 grid((unsigned)a.rows), block(64 * waves);
  const size_t lds = beam_lds(waves, a.blocks);
  if (a.bf16) hipLaunchKernelGGL((k_beam_rows<true>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_beam_rows<false>), grid, block, lds, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Selection: one wave a sequence. Totals and the normalisers' sums over shards in fp64, so that the
// choice between two beams' candidates is the formula's. Candidates come rank by rank, so the bar
// rises early. Latency: a few hundred keys (1 sequence of 4 x 8: 5.5 us, 16 of 4 shards x 5 x 10: 11).
// ------------------------------------------------------------------------------------
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  return u ^ ((u >> 63) != 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered64(uint64_t k) {
  return __builtin_bit_cast(double, k ^ ((k >> 63) != 0 ? 1ull << 63 : ~0ull));
}
constexpr uint64_t BEAM_AT = 40;   // bits of a token in a key; the host keeps ids below 2^40

__global__ __launch_bounds__(64) void k_beam_select(BeamSelectArgs a) {
  __shared__ Key128 room[128];
  __shared__ double norm[LLP_MAX_BEAMS], score[LLP_MAX_BEAMS];
  __shared__ float top[LLP_MAX_BEAMS];
  __shared__ int kind[LLP_MAX_BEAMS];   // 0: no candidates, 1: its row's, 2: end_id
  const int lane = threadIdx.x;
  const int64_t b = blockIdx.x;
  const double c = (double)a.c1;
  Best<Key128> best;
  best.init(room);
  const int per = a.world * a.K, total = per * a.num;
  // The first candidates of each lane are loaded in front of all else.
  struct Item {
    int k, r;
    int64_t at;
  };
  auto item = [&](int i) {
    const int rank = i / per, in = i - rank * per, k = in / a.world;
    return Item{k, in - k * a.world, (b * a.K + k) * a.num + rank};
  };
  constexpr int AHEAD = 4;
  float value[AHEAD];
  int64_t token[AHEAD];
#pragma unroll
  for (int q = 0; q < AHEAD; ++q) {
    const Item t = item(q * 64 + lane < total ? q * 64 + lane : 0);
    value[q] = a.value[t.r][t.at];
    token[q] = a.token[t.r][t.at];
  }
  Key128 end = Key128::none();
  if (lane < a.K) {
    const int64_t row = b * a.K + lane;
    const float sc = a.scores[row];
    const bool over = a.finished != nullptr && a.finished[row] != 0;
    bool bad = !(sc < INFINITY);
    float M = -INFINITY;
    double S = 0.0;
    if (!over) {
      for (int r = 0; r < a.world; ++r) {
        M = fmaxf(M, a.max[r][row]);
        bad |= !(a.sum[r][row] >= 0.0);
      }
      if (M > -INFINITY && !bad)
        for (int r = 0; r < a.world; ++r) {
          const float m = a.max[r][row];
          if (m == M) S += a.sum[r][row];
          else if (m > -INFINITY) S += a.sum[r][row] * exp(((double)m - (double)M) * c);
        }
    }
    if (bad && a.status) atomicOr(a.status, LLP_STATUS_VALUE_NOT_FINITE);
    const bool live = !bad && sc > -INFINITY;
    kind[lane] = !live ? 0 : over ? 2 : M > -INFINITY ? 1 : 0;
    norm[lane] = log(S);
    score[lane] = (double)sc;
    top[lane] = M;
    if (live && over) end = Key128{ordered64((double)sc), ~((uint64_t)lane << BEAM_AT)};
  }
  __syncthreads();
  best.add(end, a.num_out);
  auto take = [&](int i, float v, int64_t id) {
    Key128 x = Key128::none();
    const int k = item(i < total ? i : 0).k;
    if (i < total && kind[k] == 1) {
      const double t = score[k] + (((double)v - (double)top[k]) * c - norm[k]);
      if ((uint64_t)id >> BEAM_AT == 0 && t > -INFINITY) x = Key128{ordered64(t), ~((uint64_t)k << BEAM_AT | (uint64_t)id)};
    }
    best.add(x, a.num_out);
  };
#pragma unroll
  for (int q = 0; q < AHEAD; ++q)
    if (q * 64 < total) take(q * 64 + lane, value[q], token[q]);
  for (int i = AHEAD * 64; i < total; i += 64) {
    const Item t = item(i + lane < total ? i + lane : 0);
    take(i + lane, a.value[t.r][t.at], a.token[t.r][t.at]);
  }
  best.finish(a.num_out);
  if (lane < a.num_out) {
    const int64_t o = b * a.num_out + lane;
    const bool in = best.list.any();
    const uint64_t at = ~best.list.at;
    const int k = in ? (int)(at >> BEAM_AT) : -1;
    a.out_parent[o] = k;
    a.out_token[o] = !in ? -1 : kind[k] == 2 ? a.end_id : (int64_t)(at & ((1ull << BEAM_AT) - 1));
    a.out_score[o] = in ? (float)unordered64(best.list.k) : -INFINITY;
  }
}

hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t s) {
  if (a.seqs <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_beam_select, dim3((unsigned)a.seqs), dim3(64), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Reordering. A thread takes one unit (16 bytes) of every slot of a sequence: all of a slot's loads
// come before the first store, so the reordering is done in place without a copy, and a slot that
// keeps its own rows costs nothing. Bound by memory: the moved slots read and written (a beam that
// several slots take is read from the caches after the first; 16 sequences of 8, 4.9 GB moved: 947 us, 5.1 TB/s,
// a copy's rate).
// No load is conditional (a slot that is not moved reads the state's first unit): behind a branch each
// would be waited for before the next.
// ------------------------------------------------------------------------------------
template <int SLOTS, class U>
__global__ __launch_bounds__(256) void k_beam_reorder(ReorderArgs a, uint32_t units, uint32_t per) {
  const uint32_t w = blockIdx.x / per;   // state, then sequence
  const uint32_t st = w / (uint32_t)a.seqs;
  const int64_t b = w - st * (uint32_t)a.seqs;
  const int lane = threadIdx.x & 63;
  int p = -1;
  bool wrong = false;
  const char* const src = static_cast<const char*>(a.src[st]);
  char* const dst = static_cast<char*>(a.dst[st]);
  if (lane < a.N) {
    p = a.parents[b * a.N + lane];
    wrong = p < -1 || p >= a.K;
    if (wrong || (src == dst && p == lane)) p = -1;
  }
  if (wrong && a.status && st == 0 && blockIdx.x % per == 0 && threadIdx.x < 64)
    atomicOr(a.status, LLP_STATUS_PARENT_INVALID);
  const uint32_t u = (blockIdx.x % per) * 256 + threadIdx.x;   // below 2^32: the host's limit
  const uint32_t o = u / units;
  const bool mine = o < a.outer;
  const int64_t at = (int64_t)(u - o * units) * sizeof(U);
  const char* const from = src + b * a.K * a.sr + o * a.so + at;
  char* const to = dst + b * a.N * a.dr + o * a.dout + at;
  U v[SLOTS];
#pragma unroll
  for (int j = 0; j < SLOTS; ++j) {
    const int q = __builtin_amdgcn_readlane(p, j);
    v[j] = *reinterpret_cast<const U*>(q >= 0 && mine ? from + q * a.sr : src);
  }
#pragma unroll
  for (int j = 0; j < SLOTS; ++j)
    if (__builtin_amdgcn_readlane(p, j) >= 0 && mine) *reinterpret_cast<U*>(to + j * a.dr) = v[j];
}

template <int SLOTS, class U>
static hipError_t launch_reorder_as(const ReorderArgs& a, hipStream_t s) {
  const int64_t units = a.inner / (int64_t)sizeof(U);
  const int64_t per = (a.outer * units + 255) / 256;
  hipLaunchKernelGGL((k_beam_reorder<SLOTS, U>), dim3((unsigned)(per * a.seqs * a.states)), dim3(256), 0, s,
                     a, (uint32_t)units, (uint32_t)per);
  return hipGetLastError();
}

template <class U>
static hipError_t launch_reorder_of(const ReorderArgs& a, hipStream_t s) {
  if (a.N <= 4) return launch_reorder_as<4, U>(a, s);
  if (a.N <= 8) return launch_reorder_as<8, U>(a, s);
  if (a.N <= 16) return launch_reorder_as<16, U>(a, s);
  if constexpr (sizeof(U) < 16) {   // the host takes smaller units for more slots
    if (a.N > 32) return launch_reorder_as<64, U>(a, s);
  }
  return launch_reorder_as<32, U>(a, s);
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
  if (a.states <= 0 || a.seqs <= 0 || a.outer <= 0 || a.inner <= 0) return hipSuccess;
  if (a.unit == 16) return launch_reorder_of<u32x4>(a, s);
  if (a.unit >= 4) return launch_reorder_of<uint32_t>(a, s);
  return launch_reorder_of<uint8_t>(a, s);
}

}  // namespace llp
