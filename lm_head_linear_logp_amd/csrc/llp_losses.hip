// llp_losses.hip -- losses on scored log-probabilities and their gradients: the clipped policy
// loss with a KL term, and the preference loss of paired responses.
//
// Both are bound by memory at many rows and by launches at few. Per-row arithmetic is fp32, sums
// are fp64, in an order fixed by the sizes alone; there are no float atomics.
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

__device__ __forceinline__ bool cu_bad(const int32_t* cu, int S, int64_t T, int i) {
  const int c = cu[i];
  return (i == 0 && c != 0) || (i == S && (int64_t)c != T) || (i < S && cu[i + 1] < c);
}

// ------------------------------------------------------------------------------------
// Clipped policy loss. Launches: scored rows counted per block of POLICY_COUNT_ROWS (TOKEN_MEAN
// with a mask) or per sequence (SEQ_MEAN, then one workgroup that counts the sequences with
// scored rows and checks cu_seqlens); the loss kernel, one pass over the rows; one workgroup
// that adds up its partial sums.
// ------------------------------------------------------------------------------------
constexpr int POLICY_COUNT_ROWS = 16384;

__global__ __launch_bounds__(LOSS_THREADS) void k_policy_count(PolicyArgs a) {
  __shared__ int sh[LOSS_THREADS / 64];
  int64_t b, e;
  if (a.reduction == LLP_REDUCE_SEQ_MEAN) {
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
#pragma unroll 8
    for (int64_t t = b + threadIdx.x; t < e; t += LOSS_THREADS) n += a.mask[t] != 0 ? 1 : 0;
  }
  n = block_sum<LOSS_THREADS / 64>(n, sh);
  if (threadIdx.x == 0) a.count[blockIdx.x] = n;
}

// SEQ_MEAN: meta[0] = sequences with scored rows, meta[1] = 1 for a malformed cu_seqlens.
__global__ __launch_bounds__(1024) void k_policy_seqs(PolicyArgs a) {
  __shared__ int sh[16];
  int n = 0, bad = 0;
  for (int i = threadIdx.x; i <= a.S; i += 1024) {
    if (i < a.S) n += a.count[i] > 0 ? 1 : 0;
    bad += cu_bad(a.cu, a.S, a.T, i) ? 1 : 0;
  }
  n = block_sum<16>(n, sh);
  bad = block_sum<16>(bad, sh);
  if (threadIdx.x == 0) {
    a.meta[0] = n;
    a.meta[1] = bad ? 1 : 0;
    if (bad && a.status) atomicOr(a.status, LLP_STATUS_LAYOUT_INVALID);
  }
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

struct PolicyRow {
  float pg, kl, ratio, grad;   // policy term, KL value, r, d (policy + kl_coef kl) / d logp
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
  o.pg = -adv * used;
  o.grad = o.clipped || !inside ? 0.f : -adv * o.ratio;
  o.kl = 0.f;
  if (a.ref != nullptr) {
    const double xd = (double)ref - (double)lp;
    const float x = (float)xd;
    float g;
    if (a.kl_kind == LLP_KL_K1) {
      o.kl = -x;
      g = 1.f;
    } else if (a.kl_kind == LLP_KL_K2) {
      o.kl = 0.5f * x * x;
      g = -x;
    } else {
      const float y = fminf(fmaxf(x, -(float)LLP_LOG_RATIO_MAX), (float)LLP_LOG_RATIO_MAX);
      o.kl = exp_minus_linear(y);
      g = fabs(xd) <= (double)LLP_LOG_RATIO_MAX ? -expm1f(x) : 0.f;
    }
    o.grad = fmaf(a.klc, g, o.grad);
  }
  return o;
}

// One over the number of rows (or sequences) that the loss is a mean of; 0 when there are none.
__device__ __forceinline__ double policy_norm(const PolicyArgs& a, int* sh) {
  if (a.reduction == LLP_REDUCE_SUM) return 1.0;
  double n;
  if (a.denom != nullptr) {
    n = (double)a.denom[0];
  } else if (a.reduction == LLP_REDUCE_SEQ_MEAN) {
    n = (double)a.meta[0];
  } else if (a.mask == nullptr) {
    n = (double)a.T;
  } else {
    int c = 0;
    for (int i = threadIdx.x; i < a.ncount; i += LOSS_THREADS) c += a.count[i];
    n = (double)block_sum<LOSS_THREADS / 64>(c, sh);
  }
  return n > 0.0 && n < INFINITY ? 1.0 / n : 0.0;
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

template <bool VEC>
__global__ __launch_bounds__(LOSS_THREADS) void k_policy(PolicyArgs a) {
  __shared__ double shd[LOSS_THREADS / 64];
  __shared__ int shi[LOSS_THREADS / 64];
  const bool by_seq = a.reduction == LLP_REDUCE_SEQ_MEAN;
  const bool void_layout = by_seq && a.meta[1] != 0;
  const double norm = void_layout ? 0.0 : policy_norm(a, shi);
  const double up = a.dloss != nullptr ? (double)a.dloss[0] : 1.0;
  double sum[LLP_POLICY_STATS - 1] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};   // after the loss
  int status = 0;
  if (!by_seq && a.cu != nullptr && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.S; i += LOSS_THREADS)
      if (cu_bad(a.cu, a.S, a.T, i)) status |= LLP_STATUS_LAYOUT_INVALID;
  const int64_t step = (int64_t)gridDim.x * LOSS_THREADS * 4;
  for (int64_t t0 = (int64_t)blockIdx.x * LOSS_THREADS * 4; t0 < a.T; t0 += step) {
    const int64_t t = t0 + threadIdx.x * 4;
    float lp[4], old[4], adv[4], ref[4], ent[4], dl[4], de[4];
    bool m[4];
    mask4<VEC>(a.mask, t, a.T, m);
    load4<VEC>(a.logp, t, a.T, lp);
    load4<VEC>(a.old, t, a.T, old);
    load4<VEC>(a.adv, t, a.T, adv);
    load4<VEC>(a.ref, t, a.T, ref);
    load4<VEC>(a.ent, t, a.T, ent);
    int s = -1, s_end = 0;   // this thread's sequence and its end
    double w_seq = norm;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dl[i] = de[i] = 0.f;
      if (!m[i] || void_layout) continue;
      if (by_seq && (s < 0 || t + i >= s_end)) {
        s = seq_of(a.cu, t + i, s < 0 ? 0 : s, a.S - 1);
        s_end = a.cu[s + 1];
        w_seq = norm / (double)a.count[s];
      }
      sum[6] += 1.0;
      const bool fine = fabsf(lp[i]) < INFINITY && fabsf(old[i]) < INFINITY &&
                        fabsf(adv[i]) < INFINITY && fabsf(ref[i]) < INFINITY &&
                        fabsf(ent[i]) < INFINITY;
      if (!fine) {
        status |= LLP_STATUS_VALUE_NOT_FINITE;
        continue;
      }
      const PolicyRow r = policy_row(a, lp[i], old[i], adv[i], ref[i]);
      sum[0] += w_seq * (double)r.pg;
      sum[1] += w_seq * (double)r.kl;
      sum[2] += w_seq * (double)ent[i];
      sum[3] += r.clipped ? w_seq : 0.0;
      sum[4] += w_seq * (double)r.ratio;
      sum[5] += w_seq * ((double)old[i] - (double)lp[i]);
      dl[i] = (float)(up * w_seq * (double)r.grad);
      de[i] = (float)(up * w_seq * -a.entc64);
    }
    store4<VEC>(a.dlogp, t, a.T, dl);
    store4<VEC>(a.dent, t, a.T, de);
  }
  if (status && a.status) atomicOr(a.status, status);
#pragma unroll
  for (int k = 0; k < LLP_POLICY_STATS - 1; ++k) {
    const double x = block_sum<LOSS_THREADS / 64>(sum[k], shd);
    if (threadIdx.x == 0) a.part[(int64_t)blockIdx.x * LLP_POLICY_STATS + 1 + k] = x;
  }
}

__global__ __launch_bounds__(LOSS_THREADS) void k_policy_sum(PolicyArgs a) {
  __shared__ double shd[LOSS_THREADS / 64];
  double sum[LLP_POLICY_STATS - 1] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  for (int b = threadIdx.x; b < a.nblocks; b += LOSS_THREADS)
#pragma unroll
    for (int k = 0; k < LLP_POLICY_STATS - 1; ++k) sum[k] += a.part[(int64_t)b * LLP_POLICY_STATS + 1 + k];
#pragma unroll
  for (int k = 0; k < LLP_POLICY_STATS - 1; ++k) sum[k] = block_sum<LOSS_THREADS / 64>(sum[k], shd);
  if (threadIdx.x != 0) return;
  const double loss = sum[0] + a.klc64 * sum[1] - a.entc64 * sum[2];
  a.loss[0] = (float)loss;
  if (a.stats == nullptr) return;
  a.stats[0] = (float)loss;
#pragma unroll
  for (int k = 0; k < LLP_POLICY_STATS - 1; ++k) a.stats[1 + k] = (float)sum[k];
}

static bool all_aligned(std::initializer_list<const void*> ps, size_t n) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % n != 0) return false;
  return true;
}

hipError_t launch_policy(const PolicyArgs& a, hipStream_t s) {
  const dim3 block(LOSS_THREADS);
  if (a.ncount > 0) {
    hipLaunchKernelGGL(k_policy_count, dim3((unsigned)a.ncount), block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.reduction == LLP_REDUCE_SEQ_MEAN) {
    hipLaunchKernelGGL(k_policy_seqs, dim3(1), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool vec = all_aligned({a.logp, a.old, a.adv, a.ref, a.ent, a.dlogp, a.dent}, 16) &&
                   all_aligned({a.mask}, 4);
  if (vec) hipLaunchKernelGGL(k_policy<true>, dim3((unsigned)a.nblocks), block, 0, s, a);
  else hipLaunchKernelGGL(k_policy<false>, dim3((unsigned)a.nblocks), block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_policy_sum, dim3(1), block, 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Preference loss. First launch: the sum of logp - ref_logp over each sequence's scored rows;
// PREF_SPLIT workgroups share a sequence, workgroup y taking its chunks y, y + PREF_SPLIT, ... of
// PREF_CHUNK rows, so that a sum's order depends on its sequence alone. Second: one workgroup turns
// the sums into each pair's loss and gradient coefficient and adds up the losses. Third: the
// coefficients are spread over the scored rows.
// ------------------------------------------------------------------------------------
__global__ __launch_bounds__(LOSS_THREADS) void k_pref_sum(PrefArgs a) {
  __shared__ double shd[LOSS_THREADS / 64];
  __shared__ int shi[LOSS_THREADS / 64];
  const int s = blockIdx.x;
  const int64_t b = a.cu[s] > 0 ? a.cu[s] : 0;
  const int64_t e = a.cu[s + 1] < a.T ? a.cu[s + 1] : a.T;
  double sum = 0.0;
  int n = 0, bad = 0;
  for (int64_t c = b + (int64_t)blockIdx.y * PREF_CHUNK; c < e; c += PREF_SPLIT * PREF_CHUNK) {
    const int64_t ce = c + PREF_CHUNK < e ? c + PREF_CHUNK : e;
#pragma unroll 8
    for (int64_t t = c + threadIdx.x; t < ce; t += LOSS_THREADS) {
      if (a.mask != nullptr && a.mask[t] == 0) continue;
      const float lp = a.logp[t], rf = a.ref != nullptr ? a.ref[t] : 0.f;
      if (fabsf(lp) < INFINITY && fabsf(rf) < INFINITY) sum += (double)lp - (double)rf;
      else bad = 1;
      ++n;
    }
  }
  sum = block_sum<LOSS_THREADS / 64>(sum, shd);
  n = block_sum<LOSS_THREADS / 64>(n, shi);
  bad = block_sum<LOSS_THREADS / 64>(bad, shi);
  if (threadIdx.x == 0) {
    a.sum[(int64_t)s * PREF_SPLIT + blockIdx.y] = sum;
    a.cnt[(int64_t)s * PREF_SPLIT + blockIdx.y] = bad ? -1 : n;
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

__global__ __launch_bounds__(PAIR_THREADS) void k_pref_pairs(PrefArgs a) {
  __shared__ double shd[PAIR_THREADS / 64];
  __shared__ int shi[PAIR_THREADS / 64];
  int bad = 0;
  for (int i = threadIdx.x; i <= 2 * a.P; i += PAIR_THREADS) bad += cu_bad(a.cu, 2 * a.P, a.T, i) ? 1 : 0;
  const bool void_layout = block_sum<PAIR_THREADS / 64>(bad, shi) != 0;
  const double up = (a.dloss != nullptr ? (double)a.dloss[0] : 1.0) / (a.mean ? (double)a.P : 1.0);
  double total = 0.0;
  bool unfit = false;
  for (int p = threadIdx.x; p < a.P; p += PAIR_THREADS) {
    double R[2] = {0.0, 0.0}, per[2] = {1.0, 1.0};
    bool ok = !void_layout;
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
    if (w == 0.f) ok = false;
    else if (odd || !(fabsf(w) < INFINITY)) {
      if (ok) unfit = true;
      ok = false;
    }
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
    const double c = ok ? up * (double)w * g : 0.0;
    a.coef[2 * p] = (float)(c * per[0]);
    a.coef[2 * p + 1] = (float)(-c * per[1]);
    if (ok) total += (double)w * l;
    if (a.pair_loss != nullptr) a.pair_loss[p] = ok ? (float)l : 0.f;
    if (a.chosen != nullptr) a.chosen[p] = ok ? (float)(a.beta * R[0]) : 0.f;
    if (a.rejected != nullptr) a.rejected[p] = ok ? (float)(a.beta * R[1]) : 0.f;
  }
  total = block_sum<PAIR_THREADS / 64>(total, shd);
  if (unfit && a.status) atomicOr(a.status, LLP_STATUS_VALUE_NOT_FINITE);
  if (threadIdx.x == 0) {
    a.loss[0] = (float)(a.mean && a.P > 0 ? total / (double)a.P : total);
    if (void_layout && a.status) atomicOr(a.status, LLP_STATUS_LAYOUT_INVALID);
  }
}

template <bool VEC>
__global__ __launch_bounds__(LOSS_THREADS) void k_pref_grad(PrefArgs a) {
  const int64_t t0 = (int64_t)blockIdx.x * LOSS_THREADS * 4;
  __shared__ int ends[2];
  // The sequences this workgroup's rows lie in bound every thread's search.
  if (threadIdx.x < 2) {
    const int64_t t = threadIdx.x == 0 ? t0 : (t0 + LOSS_THREADS * 4 - 1 < a.T - 1 ? t0 + LOSS_THREADS * 4 - 1 : a.T - 1);
    ends[threadIdx.x] = seq_of(a.cu, t, 0, 2 * a.P - 1);
  }
  __syncthreads();
  const int64_t t = t0 + threadIdx.x * 4;
  if (t >= a.T) return;
  bool m[4];
  float g[4];
  mask4<VEC>(a.mask, t, a.T, m);
  int s = -1, s_end = 0;
  float c = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] = 0.f;
    if (!m[i]) continue;
    if (s < 0 || t + i >= s_end) {
      s = seq_of(a.cu, t + i, s < 0 ? ends[0] : s, ends[1] > ends[0] ? ends[1] : ends[0]);
      s_end = a.cu[s + 1];
      c = a.coef[s];
    }
    g[i] = c;
  }
  store4<VEC>(a.dlogp, t, a.T, g);
}

hipError_t launch_preference(const PrefArgs& a, hipStream_t s) {
  if (a.P > 0) {
    hipLaunchKernelGGL(k_pref_sum, dim3((unsigned)(2 * a.P), PREF_SPLIT), dim3(LOSS_THREADS), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_pref_pairs, dim3(1), dim3(PAIR_THREADS), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.dlogp == nullptr || a.T == 0) return e;
  const dim3 grid((unsigned)((a.T + LOSS_THREADS * 4 - 1) / (LOSS_THREADS * 4))), block(LOSS_THREADS);
  if (all_aligned({a.dlogp}, 16) && all_aligned({a.mask}, 4)) hipLaunchKernelGGL(k_pref_grad<true>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_pref_grad<false>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace llp
