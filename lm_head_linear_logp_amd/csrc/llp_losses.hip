// llp_losses.hip -- losses on scored log-probabilities and their gradients: the clipped policy
// loss with a KL term, and the preference loss of paired responses.
//
// Both are bound by memory at many rows and by launches at few. A row's exponentials are fp32, its
// products and all sums fp64, in an order fixed by the sizes alone; there are no float atomics.
#include "llp_internal.h"

#include <hip/hip_runtime.h>
#include <math.h>

namespace llp {

constexpr int LOSS_THREADS = 256;

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

// Sum over a workgroup of NW waves, the same in every thread; sh: NW entries.
template <int NW, class T>
__device__ __forceinline__ T block_sum(T x, T* sh) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
  __syncthreads();
  T t = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) t += sh[w];
  __syncthreads();
  return t;
}

// The sequence holding row t: the last s in [lo, hi] with cu[s] <= t (lo when there is none).
// Any cu keeps the result in [lo, hi].
__device__ __forceinline__ int seq_of(const int32_t* cu, int64_t t, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The same for the whole wave (t uniform), 64 probes at a time: two rounds for 4096 sequences.
__device__ __forceinline__ int seq_of_wave(const int32_t* cu, int64_t t, int hi) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (lo < hi) {
    const int step = (hi - lo + 64) / 64;   // ceil((hi - lo + 1) / 64)
    const int at = lo + lane * step;
    const uint64_t below = __builtin_amdgcn_ballot_w64(at <= hi && (lane == 0 || cu[at <= hi ? at : hi] <= t));
    const int k = 63 - __builtin_clzll(below);
    lo += k * step;
    hi = lo + step - 1 < hi ? lo + step - 1 : hi;
  }
  return lo;
}

__device__ __forceinline__ bool cu_bad(const int32_t* cu, int S, int64_t T, int i) {
  const int c = cu[i];
  return (i == 0 && c != 0) || (i == S && (int64_t)c != T) || (i < S && cu[i + 1] < c);
}

// Whether the layout is malformed, found before anything reads the rows it names (layout_first), a
// slice of it per workgroup (us of a replayed call with and without: policy of 2^20 rows in 2^17
// sequences 149 and 139, preference 898 and 885).
__global__ __launch_bounds__(1024) void k_layout_first(const int32_t* cu, int S, int64_t T, int32_t* looks) {
  __shared__ int sh[16];
  int bad = 0;
#pragma unroll 4
  for (int i = blockIdx.x * 1024 + threadIdx.x; i <= S; i += LAYOUT_LOOKS * 1024) bad |= cu_bad(cu, S, T, i) ? 1 : 0;
  bad = block_sum<16>(bad, sh);
  if (threadIdx.x == 0) looks[blockIdx.x] = bad != 0 ? 1 : 0;
}
static_assert(LAYOUT_LOOKS == 64, "one flag per lane");
__device__ __forceinline__ bool layout_found_bad(const int32_t* looks) {
  return __builtin_amdgcn_ballot_w64(looks[threadIdx.x & 63] != 0) != 0;
}

// ------------------------------------------------------------------------------------
// Clipped policy loss. Up to POLICY_SOLO_ROWS rows one workgroup does it all in one launch.
// Beyond, launches: scored rows counted per block of POLICY_COUNT_ROWS (TOKEN_MEAN with a mask)
// or per sequence (SEQ_MEAN); the loss kernel, one pass over the rows; one workgroup that adds
// up its partial sums. With more than POLICY_SEQS sequences one more workgroup, after the count,
// finds the number of sequences with scored rows; up to that many every block of the loss kernel
// looks through the counts itself (2^20 rows, us of a replayed call, with the workgroup and
// without: 1024 sequences 21.2 and 20.1, 4096 24.7 and 25.9, 16384 36 and 46).
// The loss kernel reads 21 bytes a row and writes 8: 13.4 us for 2^20 rows that the caches hold,
// 2.3 TB/s, on which the sequence search, the transcendentals and the fp64 sums weigh as much as
// the memory; count and sum 5.9 and 3.9 us, little more than a launch each.
// ------------------------------------------------------------------------------------
constexpr int POLICY_SEQS = 2048;
constexpr int SOLO_THREADS = 1024;
static_assert(POLICY_BLOCK_ROWS == LOSS_THREADS * 4, "four rows per thread of the loss kernel");
static_assert(POLICY_SOLO_ROWS <= SOLO_THREADS * 4, "four rows per thread of the one workgroup");

// SEQ_MEAN counts carry a malformed cu_seqlens as -1. FIRST: the layout was looked over in front (a
// kernel of its own: tested at run time it cost 2^20 rows in 65536 sequences 85 us instead of 81).
template <bool FIRST>
__global__ __launch_bounds__(LOSS_THREADS) void k_policy_count(PolicyArgs a) {
  __shared__ int sh[LOSS_THREADS / 64];
  int64_t b, e;
  bool bad = false;
  if (FIRST && layout_found_bad(a.looks)) {
    if (threadIdx.x == 0) a.count[blockIdx.x] = -1;
    if (threadIdx.x == 0 && blockIdx.x == 0 && a.status) atomicOr(a.status, LLP_STATUS_LAYOUT_INVALID);
    return;
  }
  if (a.reduction == LLP_REDUCE_SEQ_MEAN) {
    bad = cu_bad(a.cu, a.S, a.T, blockIdx.x) || cu_bad(a.cu, a.S, a.T, blockIdx.x + 1);
    b = a.cu[blockIdx.x] > 0 ? a.cu[blockIdx.x] : 0;
    e = a.cu[blockIdx.x + 1] < a.T ? a.cu[blockIdx.x + 1] : a.T;
  } else {
    b = (int64_t)blockIdx.x * POLICY_COUNT_ROWS;
    e = b + POLICY_COUNT_ROWS < a.T ? b + POLICY_COUNT_ROWS : a.T;
  }
  int n = 0;
  if (a.mask == nullptr) {
    if (threadIdx.x == 0 && e > b) n = (int)(e - b);
  } else {
#pragma unroll 16
    for (int64_t t = b + threadIdx.x; t < e; t += LOSS_THREADS) n += a.mask[t] != 0 ? 1 : 0;
  }
  n = block_sum<LOSS_THREADS / 64>(n, sh);
  if (threadIdx.x == 0) {
    a.count[blockIdx.x] = bad ? -1 : n;
    if (bad && a.status) atomicOr(a.status, LLP_STATUS_LAYOUT_INVALID);
  }
}

// SEQ_MEAN: the number of sequences with scored rows, or -1 for a malformed cu_seqlens, from the
// counts (NW waves, the result in every thread).
template <int NW>
__device__ __forceinline__ int policy_seqs(const PolicyArgs& a, int* sh) {
  int n = 0, bad = 0;
  for (int i = threadIdx.x; i < a.S; i += 64 * NW) {
    const int c = a.count[i];
    n += c > 0 ? 1 : 0;
    bad += c < 0 ? 1 : 0;
  }
  n = block_sum<NW>(n, sh);
  bad = block_sum<NW>(bad, sh);
  return bad ? -1 : n;
}

__global__ __launch_bounds__(1024) void k_policy_seqs(PolicyArgs a) {
  __shared__ int sh[16];
  const int n = policy_seqs<16>(a, sh);
  if (threadIdx.x == 0) a.meta[0] = n;
}

// exp(y) - y - 1 without the cancellation near 0: below 0.5 its series, y^2 (1/2 + y/6 + ...).
__device__ __forceinline__ float exp_minus_linear(float y) {
  if (fabsf(y) >= 0.5f) return expm1f(y) - y;
  float p = 1.f / 3628800.f;
  p = fmaf(p, y, 1.f / 362880.f);
  p = fmaf(p, y, 1.f / 40320.f);
  p = fmaf(p, y, 1.f / 5040.f);
  p = fmaf(p, y, 1.f / 720.f);
  p = fmaf(p, y, 1.f / 120.f);
  p = fmaf(p, y, 1.f / 24.f);
  p = fmaf(p, y, 1.f / 6.f);
  p = fmaf(p, y, 0.5f);
  return p * y * y;
}

// Exponentials in fp32, the products after them in fp64: finite values of any size give finite
// terms, so that a term of weight or coefficient 0 adds 0.
struct PolicyRow {
  double pg, kl, grad;   // policy term, KL value, d (policy + kl_coef kl) / d logp
  float ratio;           // r
  bool clipped;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, float lp, float old, float adv,
                                                float ref) {
  PolicyRow o;
  // The difference of two floats is exact in fp64 up to 2^-53 of it: the borders decide alike
  // everywhere.
  const double d = (double)lp - (double)old;
  const float df = (float)d;
  const bool inside = fabs(d) <= (double)LLP_LOG_RATIO_MAX;
  o.ratio = expf(fminf(fmaxf(df, -(float)LLP_LOG_RATIO_MAX), (float)LLP_LOG_RATIO_MAX));
  float used = o.ratio;
  o.clipped = false;
  if (adv > 0.f && d > a.log_hi) {
    used = a.hi;
    o.clipped = true;
  } else if (adv < 0.f && d < a.log_lo) {
    used = a.lo;
    o.clipped = true;
  } else if (adv < 0.f && d > a.log_dual) {
    used = a.dual;
    o.clipped = true;
  }
  o.pg = -(double)adv * (double)used;
  o.grad = o.clipped || !inside ? 0.0 : -(double)adv * (double)o.ratio;
  o.kl = 0.0;
  if (a.ref != nullptr) {
    const double xd = (double)ref - (double)lp;
    double g;
    if (a.kl_kind == LLP_KL_K1) {
      o.kl = -xd;
      g = 1.0;
    } else if (a.kl_kind == LLP_KL_K2) {
      o.kl = 0.5 * xd * xd;
      g = -xd;
    } else {
      const float x = (float)xd;
      const float y = fminf(fmaxf(x, -(float)LLP_LOG_RATIO_MAX), (float)LLP_LOG_RATIO_MAX);
      o.kl = (double)exp_minus_linear(y);
      g = fabs(xd) <= (double)LLP_LOG_RATIO_MAX ? -(double)expm1f(x) : 0.0;
    }
    o.grad = fma(a.klc64, g, o.grad);
  }
  return o;
}

// One over the number n of rows (or sequences) that the loss is a mean of; 0 when there are none.
__device__ __forceinline__ double policy_norm(const PolicyArgs& a, int n) {
  if (a.reduction == LLP_REDUCE_SUM) return 1.0;
  const double d = a.denom != nullptr ? (double)a.denom[0] : (double)n;
  return d > 0.0 && d < INFINITY ? 1.0 / d : 0.0;
}

// Rows 4 per thread and pass: VEC (every array 16-byte aligned) with one load per array.
template <bool VEC>
__device__ __forceinline__ void load4(const float* p, int64_t t, int64_t T, float (&v)[4]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.f;
  } else if (VEC && t + 4 <= T) {
    const float4 x = *reinterpret_cast<const float4*>(p + t);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t + i < T ? p[t + i] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(float* p, int64_t t, int64_t T, const float (&v)[4]) {
  if (p == nullptr) return;
  if (VEC && t + 4 <= T) {
    *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < T) p[t + i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void mask4(const uint8_t* p, int64_t t, int64_t T, bool (&m)[4]) {
  if (VEC && p != nullptr && t + 4 <= T) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p + t);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = ((x >> (8 * i)) & 0xFFu) != 0;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = t + i < T && (p == nullptr || p[t + i] != 0);
  }
}

// Four rows of one thread.
struct PolicyRows {
  float lp[4], old[4], adv[4], ref[4], ent[4];
  bool m[4];
};

template <bool VEC>
__device__ __forceinline__ void policy_load(const PolicyArgs& a, int64_t t, PolicyRows& x) {
  mask4<VEC>(a.mask, t, a.T, x.m);
  load4<VEC>(a.logp, t, a.T, x.lp);
  load4<VEC>(a.old, t, a.T, x.old);
  load4<VEC>(a.adv, t, a.T, x.adv);
  load4<VEC>(a.ref, t, a.T, x.ref);
  load4<VEC>(a.ent, t, a.T, x.ent);
}

constexpr int POLICY_SUMS = LLP_POLICY_STATS - 1;   // after the loss

// Their terms into `sum` and their gradients out. by_seq: w = norm / the sequence's count, its
// sequence looked for in [s_lo, s_hi].
template <bool VEC>
__device__ __forceinline__ void policy_rows(const PolicyArgs& a, int64_t t, const PolicyRows& x, double norm,
                                            double up, bool by_seq, const int* count, int s_lo, int s_hi,
                                            double (&sum)[POLICY_SUMS], int& status) {
  float dl[4], de[4];
  int s = -1, s_end = 0;   // this thread's sequence and its end
  double w = norm;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dl[i] = de[i] = 0.f;
    if (!x.m[i]) continue;
    if (by_seq && (s < 0 || t + i >= s_end)) {
      s = seq_of(a.cu, t + i, s < 0 ? s_lo : s, s_hi);
      s_end = a.cu[s + 1];
      w = norm / (double)count[s];
    }
    sum[6] += 1.0;
    const bool fine = fabsf(x.lp[i]) < INFINITY && fabsf(x.old[i]) < INFINITY &&
                      fabsf(x.adv[i]) < INFINITY && fabsf(x.ref[i]) < INFINITY &&
                      fabsf(x.ent[i]) < INFINITY;
    if (!fine) {
      status |= LLP_STATUS_VALUE_NOT_FINITE;
      continue;
    }
    const PolicyRow r = policy_row(a, x.lp[i], x.old[i], x.adv[i], x.ref[i]);
    sum[0] += w * r.pg;
    sum[1] += w * r.kl;
    sum[2] += w * (double)x.ent[i];
    sum[3] += r.clipped ? w : 0.0;
    sum[4] += w * (double)r.ratio;
    sum[5] += w * ((double)x.old[i] - (double)x.lp[i]);
    dl[i] = (float)(up * w * r.grad);
    de[i] = (float)(up * w * -a.entc64);
  }
  store4<VEC>(a.dlogp, t, a.T, dl);
  store4<VEC>(a.dent, t, a.T, de);
}

// The threads' sums over a workgroup of NW waves: sum k in thread k (k < POLICY_SUMS).
template <int NW>
__device__ __forceinline__ double policy_total(const double (&sum)[POLICY_SUMS], double (*sh)[POLICY_SUMS]) {
#pragma unroll
  for (int k = 0; k < POLICY_SUMS; ++k) {
    const double x = wave_sum(sum[k]);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6][k] = x;
  }
  __syncthreads();
  double x = 0.0;
  if (threadIdx.x < POLICY_SUMS)
    for (int w = 0; w < NW; ++w) x += sh[w][threadIdx.x];
  return x;
}

// The finished sums (sum k in thread k) to loss and statistics; sh: POLICY_SUMS entries.
__device__ __forceinline__ void policy_finish(const PolicyArgs& a, double x, double* sh) {
  if (threadIdx.x < POLICY_SUMS) {
    sh[threadIdx.x] = x;
    if (a.stats) a.stats[1 + threadIdx.x] = (float)x;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const double loss = sh[0] + a.klc64 * sh[1] - a.entc64 * sh[2];
    a.loss[0] = (float)loss;
    if (a.stats) a.stats[0] = (float)loss;
  }
}

template <bool VEC>
__global__ __launch_bounds__(LOSS_THREADS) void k_policy(PolicyArgs a) {
  constexpr int NW = LOSS_THREADS / 64;
  __shared__ double shd[NW][POLICY_SUMS];
  __shared__ int shi[NW], ends[2];
  const int64_t step = (int64_t)gridDim.x * LOSS_THREADS * 4;
  int64_t t0 = (int64_t)blockIdx.x * LOSS_THREADS * 4;
  PolicyRows x;
  policy_load<VEC>(a, t0 + threadIdx.x * 4, x);   // in flight while the weights are found
  const bool by_seq = a.reduction == LLP_REDUCE_SEQ_MEAN;
  int n = 0;
  if (by_seq) {
    n = a.S <= POLICY_SEQS ? policy_seqs<NW>(a, shi) : a.meta[0];
  } else if (a.ncount > 0) {
    for (int i = threadIdx.x; i < a.ncount; i += LOSS_THREADS) n += a.count[i];
    n = block_sum<NW>(n, shi);
  } else {
    n = (int)a.T;   // no mask (or a denominator, or a sum)
  }
  const bool void_layout = by_seq && n < 0;
  const double norm = policy_norm(a, n);
  const double up = a.dloss != nullptr ? (double)a.dloss[0] : 1.0;
  double sum[POLICY_SUMS] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  int status = 0;
  if (!by_seq && a.cu != nullptr && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.S; i += LOSS_THREADS)
      if (cu_bad(a.cu, a.S, a.T, i)) status |= LLP_STATUS_LAYOUT_INVALID;
  for (;;) {
    const int64_t t = t0 + threadIdx.x * 4;
    if (by_seq && !void_layout) {
      // The sequences of the block's first and last rows bound every thread's search.
      const int w = threadIdx.x >> 6;
      if (w < 2) {
        const int64_t last = t0 + LOSS_THREADS * 4 - 1 < a.T - 1 ? t0 + LOSS_THREADS * 4 - 1 : a.T - 1;
        const int s = seq_of_wave(a.cu, w == 0 ? t0 : last, a.S - 1);
        if ((threadIdx.x & 63) == 0) ends[w] = s;
      }
      __syncthreads();
    }
    if (void_layout) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x.m[i] = false;
    }
    policy_rows<VEC>(a, t, x, norm, up, by_seq, a.count, by_seq ? ends[0] : 0, by_seq ? ends[1] : 0, sum, status);
    t0 += step;
    if (t0 >= a.T) break;
    __syncthreads();   // `ends` is read by all before the next search writes it
    policy_load<VEC>(a, t0 + threadIdx.x * 4, x);
  }
  if (status && a.status) atomicOr(a.status, status);
  const double total = policy_total<NW>(sum, shd);
  if (threadIdx.x < POLICY_SUMS) a.part[(int64_t)blockIdx.x * LLP_POLICY_STATS + threadIdx.x] = total;
}

__global__ __launch_bounds__(LOSS_THREADS) void k_policy_sum(PolicyArgs a) {
  constexpr int NW = LOSS_THREADS / 64;
  __shared__ double shd[NW][POLICY_SUMS], fin[POLICY_SUMS];
  double sum[POLICY_SUMS] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int b = threadIdx.x; b < a.nblocks; b += LOSS_THREADS)
#pragma unroll
    for (int k = 0; k < POLICY_SUMS; ++k) sum[k] += a.part[(int64_t)b * LLP_POLICY_STATS + k];
  policy_finish(a, policy_total<NW>(sum, shd), fin);
}

// Few rows, and few sequences: everything in one workgroup.
template <bool VEC>
__global__ __launch_bounds__(SOLO_THREADS) void k_policy_solo(PolicyArgs a) {
  constexpr int NW = SOLO_THREADS / 64;
  __shared__ double shd[NW][POLICY_SUMS], fin[POLICY_SUMS];
  __shared__ int shi[NW], count[POLICY_SOLO_SEQS];
  const bool by_seq = a.reduction == LLP_REDUCE_SEQ_MEAN;
  int status = 0, n = 0;
  PolicyRows x;
  const int64_t t = threadIdx.x * 4;   // four rows a thread: all of them
  policy_load<VEC>(a, t, x);
  bool bad = false;
  if (a.cu != nullptr)
    for (int i = threadIdx.x; i <= a.S; i += SOLO_THREADS) bad |= cu_bad(a.cu, a.S, a.T, i);
  if (bad) status |= LLP_STATUS_LAYOUT_INVALID;
  bool void_layout = false;
  if (by_seq) {
    for (int i = threadIdx.x; i < a.S; i += SOLO_THREADS) count[i] = 0;
    void_layout = block_sum<NW>(bad ? 1 : 0, shi) != 0;
    if (!void_layout) {
      // Whole numbers: the order of the additions is free. A run of rows of one sequence is one.
      int s = -1, s_end = 0, run = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!x.m[i]) continue;
        if (s < 0 || t + i >= s_end) {
          if (run) atomicAdd(count + s, run);
          s = seq_of(a.cu, t + i, s < 0 ? 0 : s, a.S - 1);
          s_end = a.cu[s + 1];
          run = 0;
        }
        ++run;
      }
      if (run) atomicAdd(count + s, run);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.S; i += SOLO_THREADS) n += count[i] > 0 ? 1 : 0;
  } else if (a.reduction == LLP_REDUCE_TOKEN_MEAN && a.denom == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) n += x.m[i] ? 1 : 0;
  }
  n = block_sum<NW>(n, shi);
  const double norm = policy_norm(a, n);
  const double up = a.dloss != nullptr ? (double)a.dloss[0] : 1.0;
  double sum[POLICY_SUMS] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  if (void_layout) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.m[i] = false;
  }
  policy_rows<VEC>(a, t, x, norm, up, by_seq, count, 0, a.S - 1, sum, status);
  if (status && a.status) atomicOr(a.status, status);
  policy_finish(a, policy_total<NW>(sum, shd), fin);
}

static bool all_aligned(std::initializer_list<const void*> ps, size_t n) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % n != 0) return false;
  return true;
}

hipError_t launch_policy(const PolicyArgs& a, hipStream_t s) {
  const dim3 block(LOSS_THREADS);
  const bool vec = all_aligned({a.logp, a.old, a.adv, a.ref, a.ent, a.dlogp, a.dent}, 16) &&
                   all_aligned({a.mask}, 4);
  if (a.nblocks == 0) {
    if (vec) hipLaunchKernelGGL(k_policy_solo<true>, dim3(1), dim3(SOLO_THREADS), 0, s, a);
    else hipLaunchKernelGGL(k_policy_solo<false>, dim3(1), dim3(SOLO_THREADS), 0, s, a);
    return hipGetLastError();
  }
  if (a.first) {
    hipLaunchKernelGGL(k_layout_first, dim3(LAYOUT_LOOKS), dim3(1024), 0, s, a.cu, a.S, a.T, a.looks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.ncount > 0) {
    if (a.first) hipLaunchKernelGGL(k_policy_count<true>, dim3((unsigned)a.ncount), block, 0, s, a);
    else hipLaunchKernelGGL(k_policy_count<false>, dim3((unsigned)a.ncount), block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.reduction == LLP_REDUCE_SEQ_MEAN && a.S > POLICY_SEQS) {
    hipLaunchKernelGGL(k_policy_seqs, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (vec) hipLaunchKernelGGL(k_policy<true>, dim3((unsigned)a.nblocks), block, 0, s, a);
  else hipLaunchKernelGGL(k_policy<false>, dim3((unsigned)a.nblocks), block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_policy_sum, dim3(1), block, 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Preference loss. Few rows in few pairs: one workgroup, one launch. Else, first launch: the sum
// of logp - ref_logp over each sequence's scored rows; PREF_SPLIT workgroups share a sequence, workgroup y taking its chunks y, y + PREF_SPLIT, ... of
// PREF_CHUNK rows, so that a sum's order depends on its sequence alone. Second: the sums become each
// pair's loss and gradient coefficient, and the losses are added up. Third (with few pairs, in
// one launch with the second): the coefficients are spread over the scored rows. Bound by memory
// and launches: 512 pairs of 4128769 rows take 12.5 + 4.7 + 8.2 us (3.0 and 2.5 TB/s in the first
// and the third).
// ------------------------------------------------------------------------------------
// Sum of the scored rows' log ratios of the sequence [from, to), part y of PREF_SPLIT, by thread
// `tid` of LOSS_THREADS; n rows, `bad` when one of them is not finite.
// HELD: the rows are in LDS, and one at a time they cost least.
template <bool HELD>
__device__ __forceinline__ void pref_partial(const PrefArgs& a, int64_t from, int64_t to, int y, int tid,
                                             double& sum, int& n, int& bad) {
  const int64_t b = from > 0 ? from : 0;
  const int64_t e = to < a.T ? to : a.T;
  sum = 0.0;
  n = bad = 0;
  for (int64_t c = b + (int64_t)y * PREF_CHUNK; c < e; c += PREF_SPLIT * PREF_CHUNK) {
    const int64_t ce = c + PREF_CHUNK < e ? c + PREF_CHUNK : e;
    if constexpr (HELD) {
#pragma unroll 1
      for (int t = (int)c + tid; t < (int)ce; t += LOSS_THREADS) {
        if (a.mask[t] == 0) continue;
        const float lp = a.logp[t], rf = a.ref != nullptr ? a.ref[t] : 0.f;
        if (fabsf(lp) < INFINITY && fabsf(rf) < INFINITY) sum += (double)lp - (double)rf;
        else bad = 1;
        ++n;
      }
      continue;
    }
    constexpr int N = PREF_CHUNK / LOSS_THREADS;
    // A chunk's loads all in flight; the rows' order does not depend on their alignment.
    float lp[N], rf[N];
    bool m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = c + i * LOSS_THREADS + tid;
      const bool in = t < ce;
      m[i] = in && (a.mask == nullptr || a.mask[t] != 0);
      lp[i] = in ? a.logp[t] : 0.f;
      rf[i] = in && a.ref != nullptr ? a.ref[t] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!m[i]) continue;
      if (fabsf(lp[i]) < INFINITY && fabsf(rf[i]) < INFINITY) sum += (double)lp[i] - (double)rf[i];
      else bad = 1;
      ++n;
    }
  }
}

template <bool FIRST>
__global__ __launch_bounds__(LOSS_THREADS) void k_pref_sum(PrefArgs a) {
  __shared__ double shd[LOSS_THREADS / 64];
  __shared__ int shi[LOSS_THREADS / 64];
  double sum;
  int n, bad;
  if (FIRST && layout_found_bad(a.looks)) return;   // every output is 0, whatever the sums are
  pref_partial<false>(a, a.cu[blockIdx.x], a.cu[blockIdx.x + 1], blockIdx.y, threadIdx.x, sum, n, bad);
  sum = block_sum<LOSS_THREADS / 64>(sum, shd);
  n = block_sum<LOSS_THREADS / 64>(n, shi);
  bad = block_sum<LOSS_THREADS / 64>(bad, shi);
  if (threadIdx.x == 0) {
    const int64_t o = (int64_t)blockIdx.x * PREF_SPLIT + blockIdx.y;
    a.sum[o] = sum;
    a.cnt[o] = bad ? -1 : n;
  }
}

// softplus(x) = log(1 + exp(x)), without overflow.
__device__ __forceinline__ double softplus(double x) {
  return fmax(x, 0.0) + log1p(exp(-fabs(x)));
}
__device__ __forceinline__ double sigmoid(double x) {
  const double e = exp(-fabs(x));
  return x >= 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);
}

constexpr int PAIR_THREADS = 1024;

struct PairOut {
  double loss;       // weighted
  float coef[2];     // of the scored rows of the chosen and of the rejected response
  float l, chosen, rejected;
  bool unfit;        // a value that is not finite was met
};

// Pair p from its sums; `up` is the upstream gradient over the number of pairs (for the mean).
__device__ __forceinline__ PairOut pref_pair(const PrefArgs& a, int p, double up) {
  double R[2] = {0.0, 0.0}, per[2] = {1.0, 1.0};
  const float w = a.weight != nullptr ? a.weight[p] : 1.f;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int n = 0;
#pragma unroll
    for (int y = 0; y < PREF_SPLIT; ++y) {
      const int64_t o = ((int64_t)2 * p + k) * PREF_SPLIT + y;
      R[k] += a.sum[o];
      const int c = a.cnt[o];
      if (c < 0) odd = true;
      n += c;
    }
    if (a.average) {
      per[k] = n > 0 ? 1.0 / (double)n : 0.0;
      R[k] *= per[k];
    }
  }
  PairOut o;
  // A pair of weight 0 keeps its own loss and rewards; it adds nothing and is not reported.
  const bool fit = !odd && fabsf(w) < INFINITY, live = fit && w != 0.f;
  o.unfit = !fit && w != 0.f;
  const double h = R[0] - R[1], m = a.beta * h - a.gamma;
  double l, g;   // the pair's loss and its derivative by h
  if (a.kind == LLP_PREF_SIGMOID) {
    l = (1.0 - a.smooth) * softplus(-m) + a.smooth * softplus(m);
    g = a.beta * (a.smooth - sigmoid(-m));
  } else if (a.kind == LLP_PREF_HINGE) {
    l = fmax(0.0, 1.0 - m);
    g = m < 1.0 ? -a.beta : 0.0;
  } else {
    const double x = h - 0.5 / a.beta;
    l = x * x;
    g = 2.0 * x;
  }
  const double c = live ? up * (double)w * g : 0.0;
  o.coef[0] = (float)(c * per[0]);
  o.coef[1] = (float)(-c * per[1]);
  o.loss = live ? (double)w * l : 0.0;
  o.l = fit ? (float)l : 0.f;
  o.chosen = fit ? (float)(a.beta * R[0]) : 0.f;
  o.rejected = fit ? (float)(a.beta * R[1]) : 0.f;
  return o;
}

// All pairs, by a workgroup of NW waves: coefficients to `coef`, and, with `write`, the outputs. A
// malformed layout makes everything 0.
template <int NW>
__device__ __forceinline__ void pref_pairs(const PrefArgs& a, float* coef, bool write, double* shd, int* shi) {
  int bad = 0;
  for (int i = threadIdx.x; i <= 2 * a.P; i += 64 * NW) bad += cu_bad(a.cu, 2 * a.P, a.T, i) ? 1 : 0;
  const bool void_layout = block_sum<NW>(bad, shi) != 0;
  const double up = (a.dloss != nullptr ? (double)a.dloss[0] : 1.0) / (a.mean ? (double)a.P : 1.0);
  double total = 0.0;
  bool unfit = false;
  for (int p = threadIdx.x; p < a.P; p += 64 * NW) {
    PairOut o{};
    if (!void_layout) o = pref_pair(a, p, up);
    unfit |= o.unfit;
    total += o.loss;
    coef[2 * p] = o.coef[0];
    coef[2 * p + 1] = o.coef[1];
    if (write && a.pair_loss != nullptr) a.pair_loss[p] = o.l;
    if (write && a.chosen != nullptr) a.chosen[p] = o.chosen;
    if (write && a.rejected != nullptr) a.rejected[p] = o.rejected;
  }
  if (!write) return;
  total = block_sum<NW>(total, shd);
  if (unfit && a.status) atomicOr(a.status, LLP_STATUS_VALUE_NOT_FINITE);
  if (threadIdx.x == 0) {
    a.loss[0] = (float)(a.mean && a.P > 0 ? total / (double)a.P : total);
    if (void_layout && a.status) atomicOr(a.status, LLP_STATUS_LAYOUT_INVALID);
  }
}

__global__ __launch_bounds__(PAIR_THREADS) void k_pref_pairs(PrefArgs a) {
  __shared__ double shd[PAIR_THREADS / 64];
  __shared__ int shi[PAIR_THREADS / 64];
  pref_pairs<PAIR_THREADS / 64>(a, a.coef, true, shd, shi);
}

// Gradients of rows t .. t + 3: their sequence's coefficient where they are scored; the sequences
// are looked for in [lo, hi].
template <bool VEC>
__device__ __forceinline__ void pref_spread(const PrefArgs& a, int64_t t, const float* coef, int lo, int hi) {
  bool m[4];
  mask4<VEC>(a.mask, t, a.T, m);
  float g[4];
  int s = -1, s_end = 0;
  float c = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] = 0.f;
    if (!m[i]) continue;
    if (s < 0 || t + i >= s_end) {
      s = seq_of(a.cu, t + i, s < 0 ? lo : s, hi);
      s_end = a.cu[s + 1];
      c = coef[s];
    }
    g[i] = c;
  }
  store4<VEC>(a.dlogp, t, a.T, g);
}

// FEW (at most PREF_FEW pairs): every workgroup works the pairs out for itself, the first one
// writes them out, and the launch in between is saved (4000 rows a pair, us of a replayed call,
// with that launch and without: 128 pairs 11.3 and 10.2, 256 12.7 and 12.7, 512 18.0 and 27.1).
constexpr int PREF_FEW = 128;

template <bool VEC, bool FEW>
__global__ __launch_bounds__(LOSS_THREADS) void k_pref_grad(PrefArgs a) {
  constexpr int NW = LOSS_THREADS / 64;
  __shared__ int ends[2];
  __shared__ float own[FEW ? 2 * PREF_FEW : 1];
  const int64_t t0 = (int64_t)blockIdx.x * LOSS_THREADS * 4;
  // The sequences of the workgroup's first and last rows bound every thread's search.
  const int w = threadIdx.x >> 6;
  if (w < 2 && t0 < a.T) {
    const int64_t last = t0 + LOSS_THREADS * 4 - 1 < a.T - 1 ? t0 + LOSS_THREADS * 4 - 1 : a.T - 1;
    const int s = seq_of_wave(a.cu, w == 0 ? t0 : last, 2 * a.P - 1);
    if ((threadIdx.x & 63) == 0) ends[w] = s;
  }
  if constexpr (FEW) {
    __shared__ double shd[NW];
    __shared__ int shi[NW];
    pref_pairs<NW>(a, own, blockIdx.x == 0, shd, shi);
  }
  __syncthreads();
  const int64_t t = t0 + threadIdx.x * 4;
  if (t >= a.T || a.dlogp == nullptr) return;
  const int lo = ends[0], hi = ends[1] > lo ? ends[1] : lo;
  pref_spread<VEC>(a, t, FEW ? own : a.coef, lo, hi);
}

// Few rows in few pairs: everything in one workgroup, each group of 256 threads summing whole
// sequences exactly as k_pref_sum's workgroups do (a sum's bits do not depend on the batch).
constexpr int PREF_SOLO_SEQS = 2 * PREF_SOLO_PAIRS;

template <bool VEC>
__global__ __launch_bounds__(PAIR_THREADS) void k_pref_solo(PrefArgs a) {
  constexpr int NW = PAIR_THREADS / 64, GROUPS = PAIR_THREADS / LOSS_THREADS, GW = LOSS_THREADS / 64;
  __shared__ double wsum[PREF_SOLO_SEQS][PREF_SPLIT][GW], sums[PREF_SOLO_SEQS][PREF_SPLIT], shd[NW];
  __shared__ int wcnt[PREF_SOLO_SEQS][PREF_SPLIT][GW], cnts[PREF_SOLO_SEQS][PREF_SPLIT], shi[NW];
  __shared__ float coef[PREF_SOLO_SEQS];
  __shared__ int cu[PREF_SOLO_SEQS + 1];
  // All rows, read at once: a group's sequences follow one another without waiting for memory.
  __shared__ float lp[PREF_SOLO_ROWS], rf[PREF_SOLO_ROWS];
  __shared__ __attribute__((aligned(16))) uint8_t on[PREF_SOLO_ROWS];
  const int group = threadIdx.x / LOSS_THREADS, tid = threadIdx.x % LOSS_THREADS;
  for (int i = threadIdx.x; i <= 2 * a.P; i += PAIR_THREADS) cu[i] = a.cu[i];
  {
    constexpr int N = PREF_SOLO_ROWS / PAIR_THREADS;
    float l[N], r[N];
    uint8_t m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = i * PAIR_THREADS + threadIdx.x;
      const bool in = t < a.T;
      l[i] = in ? a.logp[t] : 0.f;
      r[i] = in && a.ref != nullptr ? a.ref[t] : 0.f;
      m[i] = in && (a.mask == nullptr || a.mask[t] != 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = i * PAIR_THREADS + threadIdx.x;
      lp[t] = l[i];
      rf[t] = r[i];
      on[t] = m[i];
    }
  }
  __syncthreads();
  PrefArgs own = a;
  own.cu = cu;
  own.logp = lp;
  own.ref = rf;
  own.mask = on;
  own.sum = &sums[0][0];
  own.cnt = &cnts[0][0];
  for (int s = group; s < 2 * a.P; s += GROUPS)
    for (int y = 0; y < PREF_SPLIT; ++y) {
      double sum = 0.0;
      int n = 0, bad = 0;
      // Most responses end before their later parts begin.
      if ((int64_t)cu[s + 1] - cu[s] > (int64_t)y * PREF_CHUNK) {
        pref_partial<true>(own, cu[s], cu[s + 1], y, tid, sum, n, bad);
        sum = wave_sum(sum);
        static_assert(PREF_SOLO_ROWS < 1 << 16, "count and flags share a word");
        n = wave_sum(n + (bad << 16));
        bad = n >> 16;
        n &= 0xFFFF;
      }
      if ((tid & 63) == 0) {
        wsum[s][y][tid >> 6] = sum;
        wcnt[s][y][tid >> 6] = bad ? -1 : n;
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.P * PREF_SPLIT; i += PAIR_THREADS) {
    const int s = i / PREF_SPLIT, y = i % PREF_SPLIT;
    double t = 0;
    int n = 0;
    bool bad = false;
#pragma unroll
    for (int w = 0; w < GW; ++w) {
      t += wsum[s][y][w];
      bad |= wcnt[s][y][w] < 0;
      n += wcnt[s][y][w];
    }
    sums[s][y] = t;
    cnts[s][y] = bad ? -1 : n;
  }
  __syncthreads();
  pref_pairs<NW>(own, coef, true, shd, shi);
  __syncthreads();
  if (a.dlogp == nullptr) return;
  for (int64_t t = threadIdx.x * 4; t < a.T; t += PAIR_THREADS * 4) pref_spread<VEC>(own, t, coef, 0, 2 * a.P - 1);
}

template <bool FEW>
static void launch_pref_grad(const PrefArgs& a, hipStream_t s) {
  const int64_t n = a.dlogp != nullptr && a.T > 0 ? (a.T + LOSS_THREADS * 4 - 1) / (LOSS_THREADS * 4) : 1;
  const dim3 grid((unsigned)n), block(LOSS_THREADS);
  if (all_aligned({a.dlogp}, 16) && all_aligned({a.mask}, 4))
    hipLaunchKernelGGL((k_pref_grad<true, FEW>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_pref_grad<false, FEW>), grid, block, 0, s, a);
}

hipError_t launch_preference(const PrefArgs& a, hipStream_t s) {
  if (a.solo) {
    if (all_aligned({a.dlogp}, 16) && all_aligned({a.mask}, 4))
      hipLaunchKernelGGL(k_pref_solo<true>, dim3(1), dim3(PAIR_THREADS), 0, s, a);
    else
      hipLaunchKernelGGL(k_pref_solo<false>, dim3(1), dim3(PAIR_THREADS), 0, s, a);
    return hipGetLastError();
  }
  if (a.first) {
    hipLaunchKernelGGL(k_layout_first, dim3(LAYOUT_LOOKS), dim3(1024), 0, s, a.cu, 2 * a.P, a.T, a.looks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.P > 0) {
    const dim3 grid((unsigned)(2 * a.P), PREF_SPLIT);
    if (a.first) hipLaunchKernelGGL(k_pref_sum<true>, grid, dim3(LOSS_THREADS), 0, s, a);
    else hipLaunchKernelGGL(k_pref_sum<false>, grid, dim3(LOSS_THREADS), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.P <= PREF_FEW) {
    launch_pref_grad<true>(a, s);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_pref_pairs, dim3(1), dim3(PAIR_THREADS), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.dlogp == nullptr || a.T == 0) return e;
  launch_pref_grad<false>(a, s);
  return hipGetLastError();
}

}  // namespace llp
