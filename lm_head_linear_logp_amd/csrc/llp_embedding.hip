// llp_embedding.hip -- token embedding of a vocabulary-partitioned table and its gradient.
#include "llp_internal.h"
#include "llp_tile.hpp"

#include <math.h>

namespace llp {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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
// into when there are few rows. Bound by memory: 119 us a call for 56583 x 4096 bf16, 3.9 TB/s of
// rows written and 3.9 read, many of them again from the caches.
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
      // Past the caches, which hold the rows that other tokens read again (129 -> 119 us for 56583
      // tokens of 4096 columns).
      if (c < end) __builtin_nontemporal_store(loc >= 0 ? emb_scale<BF16>(v[i], a.scale) : v[i], dst + c);
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
// Gradient. Launches: k_embed_ids (ids to int32 local rows), k_embed_sort (a stable counting sort
// of the rows by token), k_embed_sum (the sums, and the rows without a token), k_embed_fix (the
// sums of tokens that several units share).
//
// The sort: workgroup g owns the local rows [g R, (g + 1) R), at most EMB_ROWS_MAX of them, and
// reads every token's local row. Each of its 16 waves counts its own contiguous part of the
// tokens into LDS counters of its own and keeps the ones it found in an LDS list; a scan over
// (row, wave) turns the counters into positions; then the list (and, past its end, the tokens
// again) is walked in order to hand them out, lanes with the same row ranked by ballot. The
// tokens of lower rows, counted on the way, give the group's first position, so no group waits
// for another. No atomic decides an order: the counters only count. Every group reads 4 bytes
// per token from L2, a kilobyte per token in all, against 2 H bytes of its gradient row from
// memory; read as the caller's int64 ids, twice, it was bound by the vector ALUs (64.6 us at
// 56583 tokens).
// ------------------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_embed_ids(EmbBwdArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.T) return;
  int status = 0;
  a.loc[t] = emb_local(a, t, status);
  if (status && a.status) atomicOr(a.status, status);
}

constexpr int SORT_WAVES = 16, SORT_UNROLL = 16, SORT_LIST = 256;

// Hands out positions, in lane order, to the lanes with `in` (local row r of the group, token t).
__device__ __forceinline__ void sort_place(const EmbBwdArgs& a, volatile int* next, int lo, bool in,
                                           int r, int t, int lane) {
  uint64_t left = __builtin_amdgcn_ballot_w64(in);
  while (left != 0) {
    const int leader = __builtin_ctzll(left);
    const int rr = __builtin_amdgcn_readlane(r, leader);
    const uint64_t same = __builtin_amdgcn_ballot_w64(in && r == rr);
    const int first = next[rr];
    if (in && r == rr) {
      const int pos = first + __popcll(same & ((1ull << lane) - 1));
      a.order[pos] = t;
      a.row[pos] = lo + rr;
    }
    __builtin_amdgcn_wave_barrier();
    if (lane == leader) next[rr] = first + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    left &= ~same;
  }
}

// RAW: from the caller's ids (few tokens: one launch less); else from k_embed_ids.
template <bool RAW>
__global__ __launch_bounds__(64 * SORT_WAVES) void k_embed_sort(EmbBwdArgs a) {
  __shared__ int cnt[SORT_WAVES * EMB_ROWS_MAX];   // [wave][row]
  __shared__ int2 list[SORT_WAVES][SORT_LIST];     // token, row
  __shared__ int wtot[SORT_WAVES], wbelow[SORT_WAVES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int R = a.rows_per_group, T = (int)a.T;
  const int lo = (int)(blockIdx.x * (int64_t)R);
  const int nr = (int)(a.n_real - lo < R ? a.n_real - lo : R);
  const int part = ((T + SORT_WAVES - 1) / SORT_WAVES + 63) / 64 * 64;
  const int tb = w * part < T ? w * part : T, te = tb + part < T ? tb + part : T;
  int* const mine = cnt + w * R;
  for (int i = lane; i < nr; i += 64) mine[i] = 0;
  __builtin_amdgcn_wave_barrier();
  int status = 0;
  auto local = [&](int t) { return RAW ? emb_local(a, t, status) : a.loc[t]; };
  int below = 0, found = 0, resume = te;   // resume: the tokens from here on are not in the list
  for (int t0 = tb; t0 < te; t0 += 64 * SORT_UNROLL) {
    int loc[SORT_UNROLL];
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      const int t = t0 + u * 64 + lane;
      loc[u] = t < te ? local(t) : -1;
    }
#pragma unroll
    for (int u = 0; u < SORT_UNROLL; ++u) {
      // Unsigned, -1 is past every row.
      below += (uint32_t)loc[u] < (uint32_t)lo ? 1 : 0;
      const uint32_t r = (uint32_t)loc[u] - (uint32_t)lo;
      const bool in = loc[u] >= 0 && r < (uint32_t)nr;
      const uint64_t hits = __builtin_amdgcn_ballot_w64(in);
      if (hits != 0) {
        if (in) atomicAdd(mine + r, 1);
        const int n = __popcll(hits);
        if (resume == te && found + n <= SORT_LIST) {
          if (in) list[w][found + __popcll(hits & ((1ull << lane) - 1))] = make_int2(t0 + u * 64 + lane, (int)r);
          found += n;
        } else if (resume == te) {
          resume = t0 + u * 64;
        }
      }
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off);
  if (lane == 0) wbelow[w] = below;
  if (RAW && blockIdx.x == 0 && status && a.status) atomicOr(a.status, status);
  __syncthreads();
  // Exclusive scan of the rows' totals, one row per thread.
  static_assert(EMB_ROWS_MAX <= 64 * SORT_WAVES, "one row per thread");
  const int r = threadIdx.x;
  int tot = 0;
  if (r < nr)
    for (int v = 0; v < SORT_WAVES; ++v) tot += cnt[v * R + r];
  int incl = tot;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 63) wtot[w] = incl;
  __syncthreads();
  int run = incl - tot;
  for (int v = 0; v < SORT_WAVES; ++v) {
    run += wbelow[v];
    if (v < w) run += wtot[v];
  }
  if (r < nr) {
    a.start[lo + r] = run;
    for (int v = 0; v < SORT_WAVES; ++v) {
      const int c = cnt[v * R + r];
      cnt[v * R + r] = run;
      run += c;
    }
    if (lo + r == a.n_real - 1) a.start[a.n_real] = run;
  }
  __syncthreads();
  for (int i = 0; i < found; i += 64) {
    const bool in = i + lane < found;
    const int2 e = in ? list[w][i + lane] : make_int2(0, 0);
    sort_place(a, mine, lo, in, e.y, e.x, lane);
  }
  for (int t0 = resume; t0 < te; t0 += 64) {
    const int t = t0 + lane;
    const int loc = t < te ? local(t) : -1;
    const uint32_t q = (uint32_t)loc - (uint32_t)lo;
    sort_place(a, mine, lo, loc >= 0 && q < (uint32_t)nr, (int)q, t, lane);
  }
}

// Up to this many the ids are read raw: one launch less (37984 rows, us of a replayed call, raw and
// not: 4096 tokens 20.8 and 21.1, 8192 28.0 and 29.5, 16384 33.5 and 32.7).
constexpr int64_t SORT_RAW_TOKENS = 8192;

hipError_t launch_embedding_sort(const EmbBwdArgs& a, hipStream_t s) {
  if (a.T <= 0) return hipGetLastError();
  const int64_t groups = (a.n_real + a.rows_per_group - 1) / a.rows_per_group;
  const dim3 block(64 * SORT_WAVES);
  if (a.T <= SORT_RAW_TOKENS) {
    // A shard without real rows still reports ids out of range (a group with no rows).
    hipLaunchKernelGGL(k_embed_sort<true>, dim3((unsigned)(groups > 0 ? groups : 1)), block, 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_embed_ids, dim3((unsigned)((a.T + 255) / 256)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 0) return e;
  hipLaunchKernelGGL(k_embed_sort<false>, dim3((unsigned)groups), block, 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------
// The sums: the sorted rows are cut into units of a.unit, whatever tokens they hold, so a token
// that fills half the batch costs no more than any other. A unit adds up its rows in order, 8
// columns per thread in fp32, and writes each token's sum when the token changes; the sums of a
// token whose rows reach into another unit go to `part` (slot 0: it began in an earlier unit;
// slot 1: it begins here), and the unit where such a token begins notes in `span` how many units
// follow. When the gradient is overwritten, the rows that no token names are written as 0, by
// workgroups behind the units. Bound by memory: one read of dout, one write (or read and write) of
// the touched rows, the zeros (us a call, and the bytes over them: 485 for 56583 x 4096 bf16 onto
// 151936 rows, 6.1 TB/s; 100 for 4096 x 4096 onto 37984 rows, 6.6 TB/s).
// ------------------------------------------------------------------------------------
// Zeros are written in a launch of their own where dout is larger than this: beside many units
// they keep the units' reads waiting (151936 x 4096, us a call, apart and beside: 407 and 495 for
// 16000 tokens, 559 and 697 for 56583; 376 and 370 for 8000, 361 and 349 for 64; 37984 x 4096: 160
// and 168 for 16000, 124 and 118 for 8000; 4096 x 256: 25 and 20 for 4096).
constexpr int64_t EMB_APART_BYTES = int64_t(96) << 20;

// NT (bf16): read once, not kept in the caches.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void emb_load8(const void* base, int64_t off, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off);
    const u32x4 u = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, u[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + off);
    const f32x4 x = p[0], y = p[1];   // half lines each: the caches put them together
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = x[i];
      v[4 + i] = y[i];
    }
  }
}

__device__ __forceinline__ void emb_store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// dweight row of a finished sum: scale * sum, added to what is there or not. (Past the caches
// these half-line stores were slow, 145 us a call for 4096 tokens over 37984 rows against 130;
// swapped between lanes so that each took 1 KB in a row, they ran no faster than this.)
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

// Rows without a token become 0: one 16-byte store per thread and step, whole cache lines per
// wave, past the caches; workgroup b of `step` takes the pieces b, b + step, ... of all rows, so
// that what is written at one time lies together. (Sixteen rows of one workgroup written in a loop
// reached 5.4 TB/s instead of 7.1: 460 us instead of 348 for 151936 x 4096.)
__device__ __forceinline__ void emb_zero(const EmbBwdArgs& a, int64_t b, int64_t step, int64_t blocks, int pieces) {
  for (; b < blocks; b += step) {
    const int64_t v = b / pieces;
    const int c = ((int)(b - v * pieces) * (int)blockDim.x + (int)threadIdx.x) * 4;
    if (v < a.n_real && a.T > 0 && a.start[v + 1] != a.start[v]) continue;
    if (c < a.H)
      __builtin_nontemporal_store(f32x4{0.f, 0.f, 0.f, 0.f}, reinterpret_cast<f32x4*>(a.dW + v * a.ldw + c));
  }
}

__global__ __launch_bounds__(256) void k_embed_zero(EmbBwdArgs a, int64_t blocks, int pieces) {
  emb_zero(a, blockIdx.x, gridDim.x, blocks, pieces);
}

// NT: dout is larger than the 256 MB of the last-level cache, so nothing of it is still there from
// its producer, and what else is there is worth keeping (56583 x 4096 bf16: 487 us a call, 506
// without; 4096 x 4096, which the cache holds, lost 5 % by it).
template <bool BF16, bool NT>
__global__ __launch_bounds__(256) void k_embed_sum(EmbBwdArgs a, int units, int ny, int64_t blocks, int pieces) {
  if ((int)blockIdx.x >= units * ny) {
    emb_zero(a, (int64_t)blockIdx.x - units * ny, gridDim.x - units * ny, blocks, pieces);
    return;
  }
  const int by = (int)blockIdx.x / units;
  const int c = (by * (int)blockDim.x + (int)threadIdx.x) * 8;
  const int N = a.start[a.n_real];
  const int u = (int)blockIdx.x - by * units, s0 = u * a.unit;
  const int s1 = s0 + a.unit < N ? s0 + a.unit : N;
  const bool began = s0 < N && s0 > 0 && a.row[s0 - 1] == a.row[s0];
  const bool goes_on = s0 < N && s1 < N && a.row[s1 - 1] == a.row[s1];
  if (by == 0 && threadIdx.x == 0) {
    int n = 0;
    if (goes_on) {
      const int r = a.row[s1];
      if (a.start[r] >= s0) n = (a.start[r + 1] - 1) / a.unit - u;
    }
    a.span[u] = n;
  }
  if (s0 >= N || c >= a.H) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool first = true;
  constexpr int B = BF16 ? 8 : 4;   // rows in flight
  for (int s = s0; s < s1; s += B) {
    float v[B][8];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int k = s + i < s1 ? s + i : s1 - 1;
      emb_load8<BF16, NT>(a.dout, (int64_t)a.order[k] * a.ldo + c, v[i]);
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

// Tokens shared by several units: a workgroup looks through FIX_UNITS units and, where such a
// token begins, adds its partial sums: 8 waves take consecutive eighths of the units, then their
// sums are added in order.
constexpr int FIX_WAVES = 8, FIX_UNITS = 2;

__global__ __launch_bounds__(64 * FIX_WAVES) void k_embed_fix(EmbBwdArgs a, int units) {
  __shared__ float sh[FIX_WAVES][64][8];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const int u0 = blockIdx.x * FIX_UNITS;
  const int span = lane < FIX_UNITS && u0 + lane < units ? a.span[u0 + lane] : 0;
  uint64_t begins = __builtin_amdgcn_ballot_w64(span > 0);
  while (begins != 0) {
    const int i = __builtin_ctzll(begins);
    begins &= begins - 1;
    const int u = u0 + i, n = __builtin_amdgcn_readlane(span, i);   // n units after this one
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
    if (w == 0 && c < a.H) {
      for (int k = 1; k < FIX_WAVES; ++k)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] += sh[k][lane][x];
      emb_finish(a, a.row[(u + 1) * a.unit], c, acc);
    }
    __syncthreads();
  }
}

hipError_t launch_embedding_sum(const EmbBwdArgs& a, hipStream_t s) {
  const int units = a.n_real > 0 ? (int)((a.T + a.unit - 1) / a.unit) : 0;
  const int threads = a.H / 8 >= 256 ? 256 : (a.H / 8 + 63) / 64 * 64;
  const int ny = (a.H / 8 + threads - 1) / threads;
  const int pieces = (a.H / 4 + threads - 1) / threads;
  int64_t blocks = a.overwrite ? a.local_size * pieces : 0;
  if (units + blocks == 0) return hipGetLastError();
  int wgs = (int)(blocks < 1 << 22 ? blocks : 1 << 22);
  const int64_t bytes = a.T * a.H * (a.bf16 ? 2 : 4);
  if (wgs > 0 && units > 0 && bytes > EMB_APART_BYTES) {
    hipLaunchKernelGGL(k_embed_zero, dim3((unsigned)wgs), dim3(threads), 0, s, a, blocks, pieces);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    blocks = wgs = 0;
  }
  const dim3 grid((unsigned)(units * ny + wgs));
  const bool nt = bytes > (int64_t(256) << 20);
  if (a.bf16 && nt) hipLaunchKernelGGL((k_embed_sum<true, true>), grid, dim3(threads), 0, s, a, units, ny, blocks, pieces);
  else if (a.bf16) hipLaunchKernelGGL((k_embed_sum<true, false>), grid, dim3(threads), 0, s, a, units, ny, blocks, pieces);
  else hipLaunchKernelGGL((k_embed_sum<false, false>), grid, dim3(threads), 0, s, a, units, ny, blocks, pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || units <= 1) return e;
  hipLaunchKernelGGL(k_embed_fix, dim3((unsigned)((units + FIX_UNITS - 1) / FIX_UNITS), (unsigned)((a.H / 8 + 63) / 64)),
                     dim3(64 * FIX_WAVES), 0, s, a, units);
  return hipGetLastError();
}

}  // namespace llp
