// llp_internal.h -- kernel argument blocks and launchers shared by the C-ABI host code and
// the HIP kernels. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "llp.h"

namespace llp {

// Number of fixed K (vocabulary) ranges the dhidden product is split into. Fixed, so that a
// row's summation order never depends on the batch.
constexpr int DH_SPLITS = 2;
constexpr int TILE = 256;  // BM = BN of every GEMM tile
// Static device scratch of llp_forward_noalloc: the forward workspace of up to this many bytes
// (T = 4096 rows over a 151936-column vocabulary need 29.2 MB).
constexpr size_t SCRATCH_BYTES = size_t(32) << 20;
constexpr int MAX_DEVICES = 64;
constexpr int KSTEP = 64;  // K depth of one pipelined GEMM step
constexpr int QCTR_INTS = 16;  // tile-queue counters per GEMM kernel launch (llp_tile.hpp)
// Vocabulary tiles per slab of G with LLP_FLAG_G_SLABS (LLP_G_SLAB_COLUMNS / TILE).
constexpr int G_SLAB_TILES = LLP_G_SLAB_COLUMNS / 256;
// Rows per workgroup of the layout scan when it takes several; up to that many rows one
// workgroup scans them all.
constexpr int64_t LAYOUT_BLOCK_ROWS = 16384;
inline int64_t layout_blocks(int64_t T) {
  return T > LAYOUT_BLOCK_ROWS ? (T + LAYOUT_BLOCK_ROWS - 1) / LAYOUT_BLOCK_ROWS : 1;
}

// Rows up to which a forward is one of few rows.
constexpr int64_t FEW_ROWS = 64;

struct LayoutArgs {
  int64_t T;
  const uint8_t* mask;
  const int32_t* cu_seqlens;
  int32_t num_seqs;
  int32_t world;
  const int64_t* targets;
  int64_t offset, n_real, real_vocab;
  int32_t* count;   // [1 + layout_blocks(T)]: scored rows, then per layout block (if several)
  int32_t* scored;  // [T] compact index -> row
  int32_t* pos;     // [T] row -> compact index or -1
  int32_t* tloc;    // [T] compact index -> local target column or -1
  float* out_t;     // zero outputs of unscored rows (any may be null)
  uint8_t* out_f;
  float* out_l;
  float* out_e;
  float* out_p;
  int32_t* status;
  int32_t* qctr;    // tile-queue counters of the GEMM kernels of this call, zeroed here
  int32_t nqctr;
};

struct FwdArgs {
  const uint16_t* W;
  int64_t ldw;
  const uint16_t* h;
  int64_t ldh;
  const void* bias;
  int32_t bias_f32;
  int32_t H;
  int64_t n_real;
  int32_t nvt, ntb;
  float c1;
  const int32_t* count;
  const int32_t* scored;
  const int32_t* tloc;
  float* pm;
  float* ps;
  float* pq;
  float* tz;
  int64_t pstride;  // row capacity of the partial arrays (ntb * 256)
  int32_t* qctr;    // tile-queue counters (QCTR_INTS), zero at launch
  int32_t workers;  // host side: persistent workers to launch (the device's compute units)
};

struct CombineArgs {
  int32_t nvt;
  int64_t rows;     // host side: the call's rows (scored or not)
  int64_t pstride;
  const int32_t* count;
  const int32_t* scored;
  const int32_t* tloc;
  const float* pm;
  const float* ps;
  const float* pq;
  const float* tz;
  float* out_t;
  uint8_t* out_f;
  float* out_l;
  float* out_e;
  float* out_p;
};

struct MergeArgs {
  int64_t T;
  int32_t world;
  const uint8_t* mask;
  const float* tl[LLP_MAX_WORLD];
  const uint8_t* flag[LLP_MAX_WORLD];
  const float* lse[LLP_MAX_WORLD];
  const float* ent[LLP_MAX_WORLD];
  float* out_p;
  float* out_l;
  float* out_e;
  int32_t* status;
};

struct ToppArgs {
  int64_t T;
  const void* logits;
  int32_t bf16;
  int32_t K;
  int64_t lstride;
  const int64_t* ids;
  int64_t ids_stride;
  const int64_t* targets;
  const uint8_t* mask;
  int64_t offset, n_real, real_vocab;
  float c1;
  float* out_t;
  uint8_t* out_f;
  float* out_l;
  float* out_p;
  int32_t* status;
};

struct LogitsArgs {
  int64_t T;
  const void* logits;
  int32_t bf16;
  int64_t ld;
  int64_t offset, n_real, real_vocab;
  int32_t world;
  const uint8_t* mask;
  const int32_t* cu_seqlens;
  int32_t num_seqs;
  const int64_t* targets;
  float c1;
  float* out_t;
  uint8_t* out_f;
  float* out_l;
  float* out_e;
  float* out_p;
  int32_t* status;
};

struct KeepArgs {
  int64_t T;
  const void* logits;
  int32_t bf16;
  int64_t lstride;
  const uint8_t* keep;
  int64_t kstride;
  int64_t offset, n_real, real_vocab;
  const uint8_t* mask;
  const int64_t* targets;
  float c1;
  float* out_t;
  uint8_t* out_f;
  float* out_l;
  float* out_p;
  int32_t* status;
};

struct GradArgs {
  const uint16_t* W;
  int64_t ldw;
  const uint16_t* h;
  int64_t ldh;
  const void* bias;
  int32_t bias_f32;
  int32_t H;
  int64_t n_real;
  int32_t nvt, ntb;
  float c1;
  const int32_t* count;
  const int32_t* scored;
  const int32_t* tloc;
  int32_t toff;     // local column of the weight's first row (a vocabulary slab's first column)
  const float* lse;
  const float* dlogp;
  const float* dent;
  const float* ent;
  uint16_t* G;
  int64_t ldg;
  int32_t* qctr;    // tile-queue counters (QCTR_INTS), zero at launch
  float* dbp;       // bias-gradient partials [token block][ldg] (column sums of each G tile),
                    // or null when the request has no bias
};

struct DhArgs {
  const uint16_t* G;
  int64_t ldg;
  const uint16_t* W;  // the shard's weight rows (K-major operand of dhidden = G W)
  int64_t ldw;
  int64_t n_real;
  int32_t H;
  int32_t ntm, ntn, nsplit, nks;
  const int32_t* count;
  float* P;
  int64_t pstride;  // rows per split
  int32_t accumulate;  // 0: P = the product; 1: P += the product (later vocabulary slabs)
  int32_t* qctr;    // tile-queue counters (QCTR_INTS), zero at launch
};

struct DhReduceArgs {
  int64_t T;
  int32_t H;
  int32_t nsplit;
  const int32_t* pos;
  const float* P;
  int64_t pstride;
  uint16_t* dH;
  int64_t ldd;
};

struct DwArgs {
  const uint16_t* G;  // [scored row][local vocabulary], K-major operand of dweight = G^T hg
  int64_t ldg;
  const uint16_t* hgT;
  int64_t ldk;  // row stride of hgT (the scored-row capacity)
  int32_t H;
  int32_t ntm, ntn;
  int64_t n_real;
  const int32_t* count;
  float* dW;
  int64_t lddw;
  int32_t overwrite;  // 1: dW = the product (no read of dW); 0: dW += the product
  int32_t* qctr;    // tile-queue counters (QCTR_INTS), zero at launch
};

struct ZeroArgs {
  float* p;
  int64_t ld;
  int64_t r0, r1;  // rows [r0, r1)
  int64_t cols;
};

struct TransposeArgs {
  const uint16_t* in;
  int64_t ldi;
  const int32_t* idx;    // row gather list or null
  const int32_t* count;  // number of valid rows on the device, or null (use nvalid)
  int64_t nvalid;
  int32_t cols;          // columns of `in` read (multiple of 64)
  uint16_t* out;
  int64_t ldo;
};

struct DbArgs {
  const float* dbp;  // [token block][ldp] partials of the gradient tiles
  int64_t ldp;
  int64_t n_real;
  const int32_t* count;
  float* db;
  int32_t overwrite;  // 1: db = the sum; 0: db += the sum
};

struct QuantArgs {
  const void* x;
  int32_t bf16;
  int64_t ldx;
  int64_t rows;
  int32_t cols, colsp;  // columns, and rounded up to LLP_INT8_COLUMNS
  int8_t* q;
  int64_t ldq;
  float* scale;
};

// The fused forward on int8 operands: `f` holds the rows as 16-bit elements (W, ldw, h, ldh and H
// count pairs of columns).
struct Fwd8Args {
  FwdArgs f;
  LayoutArgs la;    // few rows: the layout, which the kernels work out themselves
  CombineArgs ca;   // few rows: the outputs
  const float* hs;  // [T] scale of each hidden row
  const float* ws;  // [local vocabulary] scale of each weight row
};

struct EmbArgs {
  const int64_t* ids;
  const uint8_t* mask;
  int64_t T;
  int64_t offset, n_real, real_vocab;
  int32_t H;
  float scale;
  const void* W;
  int32_t bf16;
  int64_t ldw;
  void* out;
  int64_t ldo;
  int32_t* status;
};

// Embedding gradient: rows are sorted by token in groups of EMB_ROWS_MAX local ids at most, and
// summed in units of emb_unit(T) consecutive sorted rows: small ones spread few tokens over the
// compute units, large ones leave fewer tokens shared between units.
constexpr int EMB_ROWS_MAX = 1024;
inline int emb_unit(int64_t T) { return T <= 4096 ? 16 : 32; }
struct EmbBwdArgs {
  const int64_t* ids;
  const uint8_t* mask;
  int64_t T;
  int64_t offset, n_real, real_vocab, local_size;
  int32_t H;
  int32_t rows_per_group;
  int32_t unit;     // emb_unit(T)
  float scale;
  int32_t overwrite;
  const void* dout;
  int32_t bf16;
  int64_t ldo;
  float* dW;
  int64_t ldw;
  int32_t* loc;     // [T] local row of each token, or -1
  int32_t* start;   // [n_real + 1] first sorted position of each local row
  int32_t* order;   // [T] sorted position -> row of dout
  int32_t* row;     // [T] sorted position -> local row
  int32_t* span;    // [units] units after this one that share the token beginning here
  float* part;      // [units][2][H] sums of a unit's first and last segment (rows shared by units)
  int32_t* status;
};

// The losses read each sequence's rows where cu_seqlens says they are: T rows in all, but a malformed
// one may name all of them again for every other sequence, hours of work at the largest sizes. Where
// sequences x rows pass this, a launch in front looks the layout over and a malformed one's rows are
// not read; below, 2^36 rows at most are (about 0.3 s), and that launch is saved.
constexpr int64_t LAYOUT_FIRST = int64_t(1) << 37;
constexpr int LAYOUT_LOOKS = 64;   // its workgroups
inline bool layout_first(const llp_token_layout& l) {
  return (int64_t)l.num_seqs * l.num_tokens > LAYOUT_FIRST;
}

// Rows and sequences up to which one workgroup computes a policy loss in one launch (us of a
// replayed call, one launch and three: 4096 rows 9.9 and 12.5, by sequence 15.0 and 16.5; 8192
// rows 13.4 and 12.8, by sequence 23.1 and 16.3).
constexpr int64_t POLICY_SOLO_ROWS = 4096;
constexpr int POLICY_SOLO_SEQS = 1024;
// Beyond: rows per workgroup of the count and per workgroup and pass of the loss kernel, and the
// latter's most workgroups.
constexpr int64_t POLICY_COUNT_ROWS = 16384, POLICY_BLOCK_ROWS = 1024, POLICY_BLOCKS = 1024;
struct PolicyArgs {
  int64_t T;
  const float* logp;
  const float* old;
  const float* adv;
  const float* ref;
  const float* ent;
  const uint8_t* mask;
  const int32_t* cu;
  int32_t S;
  double log_lo, log_hi, log_dual;     // borders of d = logp - old_logp
  float lo, hi, dual;                  // the clipped ratios
  int32_t kl_kind, reduction;
  const float* denom;
  int32_t nblocks;                     // blocks of the loss kernel; 0: one workgroup does it all
  int32_t ncount;                      // blocks of the count kernel (0: nothing to count)
  int32_t* count;                      // [ncount] scored rows, or [S] for SEQ_MEAN
  int32_t* meta;                       // [1] sequences with scored rows, -1: malformed cu_seqlens
  int32_t first;                       // the layout is looked over in front (layout_first)
  int32_t* looks;                      // [LAYOUT_LOOKS] what that found (1: malformed)
  double* part;                        // [nblocks][LLP_POLICY_STATS]
  float* loss;
  float* stats;
  const float* dloss;
  float* dlogp;
  float* dent;
  double klc64, entc64;
  int32_t* status;
};

// Workgroups that share one sequence's sum of a preference loss (fixed: the sum's order depends on
// the sequence alone).
constexpr int PREF_SPLIT = 4;
constexpr int PREF_CHUNK = 4096;
// Rows and pairs up to which one workgroup computes a preference loss in one launch: a launch
// costs the host more than the device. One launch and two, us a call and replayed from a graph:
//   1 pair of 64 rows       14.7 and 19.2,   7.1 and  8.3
//   4 pairs of 2300 rows    14.6 and 19.1,   9.4 and  8.9
//   8 pairs of 4607 rows    14.6 and 19.1,  13.0 and  9.1
//   9 pairs of 4607 rows    14.6 and 19.0,  13.4 and  9.1
//   16 pairs of 8192 rows   17.4 and 19.0,  17.9 and  8.7
//   32 pairs of 8192 rows   27.6 and 19.2,  28.2 and  8.8
// The border weighs the two: a stream that waits for the host gains 4.5 us by it up to 8 pairs, a
// graph or a busy stream loses up to 4 from 5 pairs on (and gains 1 at one pair). Past it a call's
// gain shrinks and a replay's loss grows.
constexpr int64_t PREF_SOLO_ROWS = 8192;
constexpr int PREF_SOLO_PAIRS = 8;
struct PrefArgs {
  int64_t T;
  const float* logp;
  const float* ref;
  const float* weight;
  const uint8_t* mask;
  const int32_t* cu;
  int32_t P;
  double beta, gamma, smooth;
  int32_t kind, average, mean;
  int32_t solo;      // one workgroup does it all, without the workspace
  double* sum;       // [2 P][PREF_SPLIT]
  int32_t* cnt;      // [2 P][PREF_SPLIT], scored rows; -1 when one of them is not finite
  float* coef;       // [2 P] d loss / d logp of a scored row of the sequence
  int32_t first;     // the layout is looked over in front (layout_first)
  int32_t* looks;    // [LAYOUT_LOOKS] what that found (1: malformed)
  float* loss;
  float* pair_loss;
  float* chosen;
  float* rejected;
  const float* dloss;
  float* dlogp;
  int32_t* status;
};

// Quantisation in blocks of 128 (llp_fp8.hip).
struct Quant8Args {
  const void* x;
  int32_t bf16;
  int64_t ldx;
  int64_t rows, cols;
  int32_t block, transpose;
  uint8_t* q;
  int64_t ldq;
  float* scale;
  int64_t lds;
};

// A product of operands in e4m3 (llp_fp8.hip): out[t][v], or with `grad` out[v][t].
struct Linear8Args {
  const uint8_t* x;      // [T] rows, scales by group: xs[g * ldxs + t]
  int64_t ldx;
  const float* xs;
  int64_t ldxs;
  const uint8_t* W;      // [V] rows, scales by block: ws[(v / 128) * ldws + g]
  int64_t ldw;
  const float* ws;
  int64_t ldws;
  const void* bias;
  int32_t bias_f32;
  int32_t out_bf16;
  void* out;
  int64_t ldo;
  int64_t T, V;
  int32_t steps;         // groups of 128
  int32_t grad;          // the weight gradient's layout of out
  int32_t accumulate;    // grad: out += the product
  int32_t vec;           // rows of out are 16-byte aligned
  int32_t nvt, ntb;      // tiles of the launch
};

// Beam search (llp_beam.hip). A wave takes BEAM_BLOCK columns of a row at a time.
constexpr int BEAM_BLOCK = 2048;
struct BeamArgs {
  const void* logits;
  int32_t bf16;
  int64_t ld;
  int64_t rows, n_real, offset;
  int32_t num;
  int32_t blocks;        // blocks of BEAM_BLOCK columns per row
  float c1;
  float* value;
  int64_t* token;
  float* max;
  double* sum;
  int32_t* status;
};

struct BeamSelectArgs {
  int32_t world, num, K, num_out;
  int64_t seqs;
  const float* value[LLP_MAX_WORLD];
  const int64_t* token[LLP_MAX_WORLD];
  const float* max[LLP_MAX_WORLD];
  const double* sum[LLP_MAX_WORLD];
  const float* scores;
  const uint8_t* finished;
  int64_t end_id;
  float c1;
  int64_t* out_token;
  int32_t* out_parent;
  float* out_score;
  int32_t* status;
};

constexpr int REORDER_STATES = 64;   // states per launch
struct ReorderArgs {
  const void* src[REORDER_STATES];
  void* dst[REORDER_STATES];
  int32_t states, K, N;              // K source beams, N slots per sequence
  int32_t unit;                      // bytes per load: 16, 4 or 1
  int64_t seqs, outer, inner;
  int64_t sr, so, dr, dout;          // row and outer strides of src and dst, bytes
  const int32_t* parents;
  int32_t* status;
};

hipError_t launch_layout(const LayoutArgs& a, hipStream_t s);
hipError_t launch_fwd(const FwdArgs& a, hipStream_t s);
hipError_t launch_combine(const CombineArgs& a, int64_t T_cap, hipStream_t s);
hipError_t launch_merge(const MergeArgs& a, hipStream_t s);
hipError_t launch_topp(const ToppArgs& a, hipStream_t s);
hipError_t launch_grad(const GradArgs& a, hipStream_t s);
hipError_t launch_dh(const DhArgs& a, hipStream_t s);
hipError_t launch_dh_reduce(const DhReduceArgs& a, hipStream_t s);
hipError_t launch_dw(const DwArgs& a, hipStream_t s);
hipError_t launch_transpose(const TransposeArgs& a, int64_t rows, hipStream_t s);
hipError_t launch_dbias(const DbArgs& a, hipStream_t s);
hipError_t launch_zero_rows(const ZeroArgs& a, hipStream_t s);
hipError_t launch_logits(const LogitsArgs& a, hipStream_t s);
hipError_t launch_keep(const KeepArgs& a, hipStream_t s);
hipError_t launch_quant(const QuantArgs& a, hipStream_t s);
hipError_t launch_fwd8(const Fwd8Args& a, hipStream_t s);
hipError_t launch_fwd8_few(const Fwd8Args& a, hipStream_t s);
hipError_t launch_embedding(const EmbArgs& a, hipStream_t s);
hipError_t launch_embedding_sort(const EmbBwdArgs& a, hipStream_t s);
hipError_t launch_embedding_sum(const EmbBwdArgs& a, hipStream_t s);
hipError_t launch_policy(const PolicyArgs& a, hipStream_t s);
hipError_t launch_preference(const PrefArgs& a, hipStream_t s);
hipError_t launch_quant8(const Quant8Args& a, hipStream_t s);
hipError_t launch_quant8_both(const Quant8Args& a, const Quant8Args& t, hipStream_t s);   // one x
hipError_t launch_linear8(const Linear8Args& a, hipStream_t s);
hipError_t launch_beam_candidates(const BeamArgs& a, hipStream_t s);
hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t s);
hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s);
hipError_t probe_kernels();
// Looks up this device's copy of the static scratch (the current device must be `device`);
// idempotent. Called under the library's open lock.
hipError_t scratch_init(int device);
// The device address of that copy, or null before scratch_init succeeded on the device.
void* scratch_address(int device);

}  // namespace llp
