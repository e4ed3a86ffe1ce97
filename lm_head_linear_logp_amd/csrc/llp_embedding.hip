// llp_embedding.hip -- token embedding of a vocabulary-partitioned table and its gradient.
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

// Local row of token t, or -1 (masked, another shard's, or out of range: then *status).
template <class Args>
__device__ __forceinline__ int emb_local(const Args& a, int64_t t, int& status) {
  if (a.mask != nullptr && a.mask[t] == 0) return -1;
  const int64_t id = a.ids[t];
  if (id < 0 || id >= a.real_vocab) {
    status |= LLP_STATUS_TOKEN_OUT_OF_RANGE;
    return -1;
  }
  const int64_t loc = id - a.offset;
  return loc >= 0 && loc < a.n_real ? (int)loc : -1;
}

// ------------------------------------------------------------------------------------
// Lookup: out[t] = scale * weight[local row of t], in fp32, rounded once to the weight's type; a
// row of zeros where there is none. A wave copies one row, or one of the pieces a row is cut
// into when there are few rows. Bound by memory.
// ------------------------------------------------------------------------------------
constexpr int EMB_WAVES = 4;
constexpr int EMB_PIECE = 8;   // most 16-byte chunks a lane holds

template <bool BF16>
__device__ __forceinline__ u32x4 emb_scale(u32x4 x, float s) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = pack_bf16x2(__builtin_bit_cast(float, x[i] << 16) * s,
                         __builtin_bit_cast(float, x[i] & 0xFFFF0000u) * s);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // A copy first: bit_cast of a vector's element reads the vector's first one.
      const uint32_t u = x[i];
      x[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) * s);
    }
  }
  return x;
}

template <bool BF16>
__global__ __launch_bounds__(64 * EMB_WAVES) void k_embed(EmbArgs a, int chunks, int per) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * EMB_WAVES + (threadIdx.x >> 6);
  if (t >= a.T) return;
  int status = 0;
  const int loc = emb_local(a, t, status);
  if (status && lane == 0 && blockIdx.y == 0 && a.status) atomicOr(a.status, status);
  constexpr int ES = BF16 ? 2 : 4;
  const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.W) + (int64_t)(loc < 0 ? 0 : loc) * a.ldw * ES);
  u32x4* dst = reinterpret_cast<u32x4*>(static_cast<char*>(a.out) + t * a.ldo * ES);
  const int end = min(chunks, ((int)blockIdx.y + 1) * per);
  for (int c0 = blockIdx.y * per; c0 < end; c0 += EMB_PIECE * 64) {
    u32x4 v[EMB_PIECE];
#pragma unroll
    for (int i = 0; i < EMB_PIECE; ++i) {
      const int c = c0 + i * 64 + lane;
      v[i] = u32x4{0, 0, 0, 0};
      if (loc >= 0 && c < end) v[i] = src[c];
    }
#pragma unroll
    for (int i = 0; i < EMB_PIECE; ++i) {
      const int c = c0 + i * 64 + lane;
      if (c < end) dst[c] = loc >= 0 ? emb_scale<BF16>(v[i], a.scale) : v[i];
    }
  }
}

hipError_t launch_embedding(const EmbArgs& a, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const int chunks = a.H / (a.bf16 ? 8 : 4);
  // Pieces of 64 .. 512 chunks per wave: enough waves to cover the compute units with few rows.
  int per = EMB_PIECE * 64;
  while (per > 64 && a.T * ((chunks + per - 1) / per) < 2048) per /= 2;
  const dim3 grid((unsigned)((a.T + EMB_WAVES - 1) / EMB_WAVES), (unsigned)((chunks + per - 1) / per));
  if (a.bf16) hipLaunchKernelGGL(k_embed<true>, grid, dim3(64 * EMB_WAVES), 0, s, a, chunks, per);
  else hipLaunchKernelGGL(k_embed<false>, grid, dim3(64 * EMB_WAVES), 0, s, a, chunks, per);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Gradient, first launch: a stable counting sort of the rows by token. Workgroup g owns the local
// rows [g R, (g + 1) R), at most EMB_ROWS_MAX of them, and reads every token id twice: each of
// its 16 waves counts its own contiguous part of the tokens into LDS counters of its own, a
// scan over (row, wave) turns them into positions, and the second pass hands out the positions
// in token order (lanes with the same row are ranked by ballot). The tokens of lower rows,
// counted in the first pass, give the group's first position, so no group waits for another.
// No atomic decides an order: the counters only count. Reading the ids once per group costs
// 2 x 9 bytes x groups per token from L2, against 2 H bytes of its gradient row from memory.
// ------------------------------------------------------------------------------------
constexpr int SORT_WAVES = 16, SORT_UNROLL = 8;

__global__ __launch_bounds__(64 * SORT_WAVES) void k_embed_sort(EmbBwdArgs a) {
  __shared__ int cnt[SORT_WAVES * EMB_ROWS_MAX];   // [wave][row]
  __shared__ int wtot[SORT_WAVES], wbelow[SORT_WAVES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int R = a.rows_per_group;
  const int64_t lo64 = (int64_t)blockIdx.x * R;
  const int lo = (int)lo64;
  const int nr = (int)(a.n_real - lo64 < R ? a.n_real - lo64 : R);
  const int64_t part = (((a.T + SORT_WAVES - 1) / SORT_WAVES) + 63) / 64 * 64;
  const int64_t tb = w * part, te = tb + part < a.T ? tb + part : a.T;
  int* const mine = cnt + w * R;
  for (int i = lane; i < nr; i += 64) mine[i] = 0;
  __builtin_amdgcn_wave_barrier();
  int below = 0, status = 0;
  for (int64_t t0 = tb; t0 < te; t0 += 64 * SORT_UNROLL) {
    int loc[SORT_UNROLL];
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      const int64_t t = t0 + u * 64 + lane;
      loc[u] = t < te ? emb_local(a, t, status) : -1;
    }
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      const int r = loc[u] - lo;
      below += loc[u] >= 0 && r < 0 ? 1 : 0;
      if (loc[u] >= 0 && r >= 0 && r < nr) atomicAdd(mine + r, 1);
    }
  }
  if (blockIdx.x == 0 && status && a.status) atomicOr(a.status, status);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off);
  if (lane == 0) wbelow[w] = below;
  __syncthreads();
  // Exclusive scan of the rows' totals; thread i takes rows 2i and 2i + 1.
  const int r0 = 2 * threadIdx.x;
  int tot[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (r0 + k < nr)
      for (int v = 0; v < SORT_WAVES; ++v) tot[k] += cnt[v * R + r0 + k];
  int incl = tot[0] + tot[1];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 63) wtot[w] = incl;
  __syncthreads();
  int run = incl - tot[0] - tot[1];
  for (int v = 0; v < SORT_WAVES; ++v) {
    run += wbelow[v];
    if (v < w) run += wtot[v];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (r0 + k < nr) {
      a.start[lo + r0 + k] = run;
      for (int v = 0; v < SORT_WAVES; ++v) {
        const int c = cnt[v * R + r0 + k];
        cnt[v * R + r0 + k] = run;
        run += c;
      }
      if (lo + r0 + k == a.n_real - 1) a.start[a.n_real] = run;
    }
  __syncthreads();
  volatile int* const next = mine;
  for (int64_t t0 = tb; t0 < te; t0 += 64 * SORT_UNROLL) {
    int loc[SORT_UNROLL];
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      const int64_t t = t0 + u * 64 + lane;
      loc[u] = t < te ? emb_local(a, t, status) : -1;
    }
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      const int r = loc[u] >= 0 ? loc[u] - lo : -1;
      const bool in = r >= 0 && r < nr;
      uint64_t left = __builtin_amdgcn_ballot_w64(in);
      while (left != 0) {
        const int leader = __builtin_ctzll(left);
        const int rr = __builtin_amdgcn_readlane(r, leader);
        const uint64_t same = __builtin_amdgcn_ballot_w64(in && r == rr);
        const int first = next[rr];
        if (in && r == rr) {
          const int pos = first + __popcll(same & ((1ull << lane) - 1));
          a.order[pos] = (int)(t0 + u * 64 + lane);
          a.row[pos] = lo + rr;
        }
        __builtin_amdgcn_wave_barrier();
        if (lane == leader) next[rr] = first + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        left &= ~same;
      }
    }
  }
}

hipError_t launch_embedding_sort(const EmbBwdArgs& a, hipStream_t s) {
  // A shard without real rows still reports ids out of range (one group with no rows).
  const int64_t groups = a.n_real > 0 ? (a.n_real + a.rows_per_group - 1) / a.rows_per_group : 1;
  if (a.T > 0)
    hipLaunchKernelGGL(k_embed_sort, dim3((unsigned)groups), dim3(64 * SORT_WAVES), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// Second launch: the sorted rows are cut into units of EMB_UNIT, whatever tokens they hold, so a
// token that fills half the batch costs no more than any other. A unit adds up its rows in
// order, 8 columns per thread in fp32, and writes each token's sum when the token changes; the
// sums of a token whose rows reach into another unit go to `part` (slot 0: it began in an earlier
// unit; slot 1: it begins here) and the third launch adds those up in unit order. Behind the
// units, when the gradient is overwritten, workgroups write the rows that no token names as 0.
// Bound by memory: one read of dout, one write (or read and write) of the touched rows.
// ------------------------------------------------------------------------------------
constexpr int EMB_ZERO_ROWS = 16;

template <bool BF16>
__device__ __forceinline__ void emb_load8(const void* base, int64_t off, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, u[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
    }
  } else {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + off + 4);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
}

__device__ __forceinline__ void emb_store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// dweight row of a finished sum: scale * sum, added to what is there or not.
__device__ __forceinline__ void emb_finish(const EmbBwdArgs& a, int row, int c, float (&v)[8]) {
  float* p = a.dW + (int64_t)row * a.ldw + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= a.scale;
  if (!a.overwrite) {
    float o[8];
    emb_load8<false>(p, 0, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += o[i];
  }
  emb_store8(p, v);
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_embed_sum(EmbBwdArgs a, int units) {
  const int c = ((int)blockIdx.y * (int)blockDim.x + (int)threadIdx.x) * 8;
  if ((int)blockIdx.x >= units) {
    // Rows without a token (and padding rows) become 0.
    if (c >= a.H) return;
    const int64_t v0 = ((int64_t)blockIdx.x - units) * EMB_ZERO_ROWS;
    for (int64_t v = v0; v < v0 + EMB_ZERO_ROWS && v < a.local_size; ++v) {
      if (v < a.n_real && a.T > 0 && a.start[v + 1] != a.start[v]) continue;
      const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      emb_store8(a.dW + v * a.ldw + c, z);
    }
    return;
  }
  const int N = a.start[a.n_real];
  const int u = blockIdx.x, s0 = u * EMB_UNIT;
  if (s0 >= N || c >= a.H) return;
  const int s1 = s0 + EMB_UNIT < N ? s0 + EMB_UNIT : N;
  const bool began = s0 > 0 && a.row[s0 - 1] == a.row[s0];
  const bool goes_on = s1 < N && a.row[s1 - 1] == a.row[s1];
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool first = true;
  constexpr int B = BF16 ? 8 : 4;   // rows in flight
  for (int s = s0; s < s1; s += B) {
    float v[B][8];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int k = s + i < s1 ? s + i : s1 - 1;
      emb_load8<BF16>(a.dout, (int64_t)a.order[k] * a.ldo + c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int k = s + i;
      if (k >= s1) break;
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] += v[i][x];
      const int r = a.row[k];
      if (k + 1 == s1 || a.row[k + 1] != r) {
        if (first && began) emb_store8(a.part + ((int64_t)u * 2) * a.H + c, acc);
        else if (k + 1 == s1 && goes_on) emb_store8(a.part + ((int64_t)u * 2 + 1) * a.H + c, acc);
        else emb_finish(a, r, c, acc);
        first = false;
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] = 0.f;
      }
    }
  }
}

// Third launch: the workgroup of the unit where a token shared by several units begins adds its
// partial sums: 8 waves take consecutive eighths of the units, then their sums are added in order.
constexpr int FIX_WAVES = 8;

__global__ __launch_bounds__(64 * FIX_WAVES) void k_embed_fix(EmbBwdArgs a) {
  __shared__ float sh[FIX_WAVES][64][8];
  const int N = a.start[a.n_real];
  const int u = blockIdx.x, s0 = u * EMB_UNIT, s1 = s0 + EMB_UNIT;
  if (s1 >= N) return;
  const int r = a.row[s1];
  if (a.row[s1 - 1] != r || a.start[r] < s0) return;
  const int last = (a.start[r + 1] - 1) / EMB_UNIT;
  const int n = last - u;   // units after this one
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int b = u + 1 + (int)((int64_t)n * w / FIX_WAVES), e = u + 1 + (int)((int64_t)n * (w + 1) / FIX_WAVES);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.H) {
    if (w == 0) emb_load8<false>(a.part, ((int64_t)u * 2 + 1) * a.H + c, acc);
#pragma unroll 4
    for (int k = b; k < e; ++k) {
      float v[8];
      emb_load8<false>(a.part, (int64_t)k * 2 * a.H + c, v);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] += v[x];
    }
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) sh[w][lane][x] = acc[x];
  __syncthreads();
  if (w != 0 || c >= a.H) return;
  for (int k = 1; k < FIX_WAVES; ++k)
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] += sh[k][lane][x];
  emb_finish(a, r, c, acc);
}

hipError_t launch_embedding_sum(const EmbBwdArgs& a, hipStream_t s) {
  const int units = a.n_real > 0 ? (int)((a.T + EMB_UNIT - 1) / EMB_UNIT) : 0;
  const int64_t zero = a.overwrite ? (a.local_size + EMB_ZERO_ROWS - 1) / EMB_ZERO_ROWS : 0;
  if (units + zero == 0) return hipGetLastError();
  const int threads = a.H / 8 >= 256 ? 256 : (a.H / 8 + 63) / 64 * 64;
  const dim3 grid((unsigned)(units + zero), (unsigned)((a.H / 8 + threads - 1) / threads));
  if (a.bf16) hipLaunchKernelGGL(k_embed_sum<true>, grid, dim3(threads), 0, s, a, units);
  else hipLaunchKernelGGL(k_embed_sum<false>, grid, dim3(threads), 0, s, a, units);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || units <= 1) return e;
  hipLaunchKernelGGL(k_embed_fix, dim3((unsigned)units - 1, (unsigned)((a.H / 8 + 63) / 64)),
                     dim3(64 * FIX_WAVES), 0, s, a);
  return hipGetLastError();
}

}  // namespace llp
