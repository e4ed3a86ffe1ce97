// llp_api_gen.cpp -- C-ABI entry points of the operators that decode and train with a head in 8-bit
// floating point: block quantisation, products of such operands, and one step of a beam search.
// As in llp_api.cpp, validation runs before any HIP call.
#include <hip/hip_runtime_api.h>
#include <math.h>

#include "llp.h"
#include "llp_host.h"
#include "llp_internal.h"

using namespace llp;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 23) - 256;
constexpr int64_t kMaxTiles = int64_t(1) << 23;   // a launch holds fewer than 2^32 threads
constexpr int64_t kMaxStride = int64_t(1) << 40;

int64_t blocks_of(int64_t n) { return round_up(n, LLP_FP8_BLOCK) / LLP_FP8_BLOCK; }

bool dtype_ok(int32_t d) { return d == LLP_DTYPE_BF16 || d == LLP_DTYPE_F32; }
size_t size_of(int32_t d) { return d == LLP_DTYPE_F32 ? 4 : 2; }

// An e4m3 operand of a product: rows, strides, alignment (its pointers may be NULL without rows or
// depth).
llp_status check_operand(const char* name, const uint8_t* p, int64_t stride, const float* scale,
                         int64_t rows, int64_t depth) {
  LLP_CHECK(rows >= 0, LLP_ERR_INVALID_ARGUMENT, "%s has %lld rows", name, (long long)rows);
  LLP_CHECK(rows <= kMaxRows, LLP_ERR_UNSUPPORTED, "%s: %lld rows exceed 2^23 - 256", name, (long long)rows);
  LLP_CHECK(stride >= depth && stride % 16 == 0, LLP_ERR_INVALID_ARGUMENT,
            "%s stride %lld must be >= depth and a multiple of 16", name, (long long)stride);
  // Tile rows are addressed with 32-bit byte offsets: 319 rows and the depth.
  LLP_CHECK(stride <= (int64_t(1) << 23), LLP_ERR_UNSUPPORTED, "%s stride must be <= 2^23", name);
  LLP_CHECK(aligned(scale, 4), LLP_ERR_INVALID_ARGUMENT, "%s scale not aligned to fp32", name);
  if (rows > 0 && depth > 0) {
    LLP_CHECK(p && scale, LLP_ERR_INVALID_ARGUMENT, "%s and its scale are required", name);
    LLP_CHECK(aligned(p, 16), LLP_ERR_INVALID_ARGUMENT, "%s not 16-byte aligned", name);
  }
  return LLP_OK;
}

// A quantisation's checks and what its kernel takes.
llp_status check_quant(const llp_fp8_quant_request* req, Quant8Args* args) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  const llp_fp8_quant_request& p = *req;
  LLP_CHECK(p.rows >= 0 && p.rows < (int64_t(1) << 31) && p.cols >= 0 && p.cols < (int64_t(1) << 31),
            LLP_ERR_INVALID_ARGUMENT, "x of %lld x %lld is out of range", (long long)p.rows, (long long)p.cols);
  LLP_CHECK(dtype_ok(p.x_dtype), LLP_ERR_INVALID_ARGUMENT, "x_dtype %d is not BF16 or F32", p.x_dtype);
  LLP_CHECK(p.block_rows == 1 || p.block_rows == LLP_FP8_BLOCK, LLP_ERR_INVALID_ARGUMENT,
            "block_rows %d is not 1 or %d", p.block_rows, LLP_FP8_BLOCK);
  LLP_CHECK(p.x_stride >= p.cols && p.x_stride < kMaxStride, LLP_ERR_INVALID_ARGUMENT,
            "x_stride %lld must be >= cols", (long long)p.x_stride);
  const int64_t M = p.transpose ? p.cols : p.rows, K = p.transpose ? p.rows : p.cols;
  LLP_CHECK(p.q_stride >= round_up(K, LLP_FP8_BLOCK) && p.q_stride % 16 == 0 && p.q_stride < kMaxStride,
            LLP_ERR_INVALID_ARGUMENT, "q_stride %lld must be >= %lld and a multiple of 16", (long long)p.q_stride,
            (long long)round_up(K, LLP_FP8_BLOCK));
  LLP_CHECK(p.scale_stride >= (p.block_rows == 1 ? M : blocks_of(K)) && p.scale_stride < kMaxStride,
            LLP_ERR_INVALID_ARGUMENT, "scale_stride %lld is too small", (long long)p.scale_stride);
  LLP_CHECK(blocks_of(p.rows) * blocks_of(p.cols) < kMaxTiles, LLP_ERR_UNSUPPORTED,
            "x of %lld x %lld holds too many blocks", (long long)p.rows, (long long)p.cols);
  if (M > 0 && K > 0) {
    LLP_CHECK(p.x && p.q && p.scale, LLP_ERR_INVALID_ARGUMENT, "x, q and scale are required");
    LLP_CHECK(aligned(p.x, size_of(p.x_dtype)), LLP_ERR_INVALID_ARGUMENT, "x not aligned to its element type");
    LLP_CHECK(aligned(p.q, 16) && aligned(p.scale, 4), LLP_ERR_INVALID_ARGUMENT,
              "q must be 16-byte aligned, scale aligned to fp32");
  }
  Quant8Args& a = *args;
  a.x = p.x;
  a.bf16 = p.x_dtype == LLP_DTYPE_BF16;
  a.ldx = p.x_stride;
  a.rows = p.rows;
  a.cols = p.cols;
  a.block = p.block_rows != 1;
  a.transpose = p.transpose != 0;
  a.q = p.q;
  a.ldq = p.q_stride;
  a.scale = p.scale;
  a.lds = p.scale_stride;
  return LLP_OK;
}

llp_status run_linear(const llp_fp8_linear_request* req, bool grad, void* stream) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  const llp_fp8_linear_request& p = *req;
  LLP_CHECK(p.depth >= 0 && p.depth % LLP_FP8_BLOCK == 0, LLP_ERR_INVALID_ARGUMENT,
            "depth %lld is not a multiple of %d", (long long)p.depth, LLP_FP8_BLOCK);
  LLP_CHECK(p.depth <= (int64_t(1) << 23), LLP_ERR_UNSUPPORTED, "depth %lld exceeds 2^23", (long long)p.depth);
  llp_status st = check_operand("x", p.x, p.x_stride, p.x_scale, p.rows, p.depth);
  if (st != LLP_OK) return st;
  st = check_operand("weight", p.weight, p.weight_stride, p.weight_scale, p.cols, p.depth);
  if (st != LLP_OK) return st;
  LLP_CHECK(p.x_scale_stride >= p.rows && p.x_scale_stride < kMaxStride, LLP_ERR_INVALID_ARGUMENT,
            "x_scale_stride %lld must be >= rows", (long long)p.x_scale_stride);
  LLP_CHECK(p.weight_scale_stride >= p.depth / LLP_FP8_BLOCK && p.weight_scale_stride < kMaxStride,
            LLP_ERR_INVALID_ARGUMENT, "weight_scale_stride %lld must be >= depth / %d",
            (long long)p.weight_scale_stride, LLP_FP8_BLOCK);
  LLP_CHECK((round_up(p.rows, 32) / 32) * blocks_of(p.cols) < kMaxTiles, LLP_ERR_UNSUPPORTED,
            "%lld x %lld outputs are too many tiles", (long long)p.rows, (long long)p.cols);
  LLP_CHECK(dtype_ok(p.out_dtype), LLP_ERR_INVALID_ARGUMENT, "out_dtype %d is not BF16 or F32", p.out_dtype);
  const bool overwrite = (p.flags & LLP_FLAG_OVERWRITE_GRADS) != 0;
  LLP_CHECK((p.flags & ~uint32_t(grad ? LLP_FLAG_OVERWRITE_GRADS : 0)) == 0, LLP_ERR_INVALID_ARGUMENT,
            "unknown flags 0x%x", p.flags);
  if (grad) {
    LLP_CHECK(p.bias == nullptr, LLP_ERR_INVALID_ARGUMENT, "a weight gradient takes no bias");
    LLP_CHECK(overwrite || p.out_dtype == LLP_DTYPE_F32, LLP_ERR_INVALID_ARGUMENT,
              "a gradient that is added to must be fp32");
  } else if (p.bias != nullptr) {
    LLP_CHECK(dtype_ok(p.bias_dtype), LLP_ERR_INVALID_ARGUMENT, "bias_dtype %d is not BF16 or F32", p.bias_dtype);
    LLP_CHECK(aligned(p.bias, size_of(p.bias_dtype)), LLP_ERR_INVALID_ARGUMENT,
              "bias not aligned to its element type");
  }
  const int64_t orows = grad ? p.cols : p.rows, ocols = grad ? p.rows : p.cols;
  const size_t es = size_of(p.out_dtype);
  LLP_CHECK(p.out_stride >= ocols && p.out_stride < kMaxStride, LLP_ERR_INVALID_ARGUMENT,
            "out_stride %lld must be >= %lld", (long long)p.out_stride, (long long)ocols);
  // 32 rows of an fp32 gradient are addressed with 32-bit byte offsets.
  LLP_CHECK(!grad || p.out_dtype != LLP_DTYPE_F32 || p.out_stride < (int64_t(1) << 24), LLP_ERR_UNSUPPORTED,
            "an fp32 gradient's out_stride must be < 2^24");
  if (orows > 0 && ocols > 0) {
    LLP_CHECK(p.out != nullptr, LLP_ERR_INVALID_ARGUMENT, "out is NULL");
    LLP_CHECK(aligned(p.out, es), LLP_ERR_INVALID_ARGUMENT, "out not aligned to its element type");
  }
  st = check_device();
  if (st != LLP_OK) return st;
  if (orows == 0 || ocols == 0 || (grad && p.depth == 0 && !overwrite)) return LLP_OK;
  Linear8Args a{};
  a.x = p.x;
  a.ldx = p.x_stride;
  a.xs = p.x_scale;
  a.ldxs = p.x_scale_stride;
  a.W = p.weight;
  a.ldw = p.weight_stride;
  a.ws = p.weight_scale;
  a.ldws = p.weight_scale_stride;
  a.bias = p.bias;
  a.bias_f32 = p.bias_dtype == LLP_DTYPE_F32;
  a.out_bf16 = p.out_dtype == LLP_DTYPE_BF16;
  a.out = p.out;
  a.ldo = p.out_stride;
  a.T = p.rows;
  a.V = p.cols;
  a.steps = (int32_t)(p.depth / LLP_FP8_BLOCK);
  a.grad = grad;
  a.accumulate = grad && !overwrite;
  a.vec = aligned(p.out, 16) && p.out_stride * (int64_t)es % 16 == 0;
  LLP_HIP(launch_linear8(a, static_cast<hipStream_t>(stream)), "fp8 product kernel launch");
  return LLP_OK;
}

// ---- Beam search ----------------------------------------------------------------------------
// c1 = 1 / temperature within what the kernels' exponents hold.
llp_status check_beam_temperature(float temperature, float* c1) {
  *c1 = (float)(1.0 / (double)temperature);
  LLP_CHECK(temperature > 0.f && *c1 >= 0x1p-64f && *c1 <= 0x1p64f, LLP_ERR_INVALID_ARGUMENT,
            "temperature must be in [2^-64, 2^64]");
  return LLP_OK;
}

llp_status check_beam(const llp_beam_request* req, float* c1) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  llp_status st = check_partition(req->vocab);
  if (st != LLP_OK) return st;
  LLP_CHECK(req->num_rows >= 0 && req->num_rows < (int64_t(1) << 22), LLP_ERR_INVALID_ARGUMENT,
            "num_rows %lld outside [0, 2^22)", (long long)req->num_rows);
  // A workgroup keeps 32 bytes of LDS for every 2048 columns.
  LLP_CHECK(req->vocab.local_size <= (int64_t(1) << 21), LLP_ERR_UNSUPPORTED,
            "local_size %lld exceeds 2^21", (long long)req->vocab.local_size);
  LLP_CHECK(req->vocab.padded_vocab < kMaxStride, LLP_ERR_UNSUPPORTED, "padded_vocab must be < 2^40");
  LLP_CHECK(req->num >= 1 && req->num <= LLP_MAX_BEAMS, LLP_ERR_INVALID_ARGUMENT,
            "num %d outside [1, %d]", req->num, LLP_MAX_BEAMS);
  LLP_CHECK(dtype_ok(req->logits_dtype), LLP_ERR_INVALID_ARGUMENT, "logits_dtype %d is not BF16 or F32",
            req->logits_dtype);
  const int64_t es = (int64_t)size_of(req->logits_dtype);
  LLP_CHECK(req->logits_stride >= req->vocab.local_size && req->logits_stride < kMaxStride,
            LLP_ERR_INVALID_ARGUMENT, "logits_stride %lld must be >= local_size", (long long)req->logits_stride);
  if (req->num_rows > 0 && local_real(req->vocab) > 0) {
    LLP_CHECK(req->logits != nullptr && aligned(req->logits, 16), LLP_ERR_INVALID_ARGUMENT,
              "logits must be non-NULL and 16-byte aligned");
    LLP_CHECK(req->num_rows == 1 || req->logits_stride * es % 16 == 0, LLP_ERR_INVALID_ARGUMENT,
              "rows of logits must be 16-byte aligned");
  }
  return check_beam_temperature(req->temperature, c1);
}

// Whether `rows` x `outer` pieces of `inner` bytes at these strides are apart: the smaller stride
// holds a piece, the larger all pieces of the smaller.
bool apart(int64_t rows, int64_t outer, int64_t inner, int64_t rs, int64_t os) {
  if (rows <= 1 && outer <= 1) return true;
  if (outer <= 1) return rs >= inner;
  if (rows <= 1) return os >= inner;
  if (rs <= os) return rs >= inner && os >= (rows - 1) * rs + inner;
  return os >= inner && rs >= (outer - 1) * os + inner;
}

}  // namespace

extern "C" {

LLP_API llp_status llp_quantize_blocks(const llp_fp8_quant_request* req, void* stream) {
  Quant8Args a{};
  llp_status st = check_quant(req, &a);
  if (st != LLP_OK) return st;
  st = check_device();
  if (st != LLP_OK) return st;
  LLP_HIP(launch_quant8(a, static_cast<hipStream_t>(stream)), "fp8 quantise kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_quantize_both(const llp_fp8_quant_request* groups, const llp_fp8_quant_request* blocks,
                                     void* stream) {
  Quant8Args a{}, t{};
  llp_status st = check_quant(groups, &a);
  if (st != LLP_OK) return st;
  st = check_quant(blocks, &t);
  if (st != LLP_OK) return st;
  LLP_CHECK(a.x == t.x && a.bf16 == t.bf16 && a.ldx == t.ldx && a.rows == t.rows && a.cols == t.cols,
            LLP_ERR_INVALID_ARGUMENT, "the two requests name different x");
  LLP_CHECK(!a.block && !a.transpose && t.block && t.transpose, LLP_ERR_INVALID_ARGUMENT,
            "the first request is by group, the second in blocks and transposed");
  st = check_device();
  if (st != LLP_OK) return st;
  LLP_HIP(launch_quant8_both(a, t, static_cast<hipStream_t>(stream)), "fp8 quantise kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_linear_fp8(const llp_fp8_linear_request* req, void* stream) {
  return run_linear(req, false, stream);
}

LLP_API llp_status llp_dweight_fp8(const llp_fp8_linear_request* req, void* stream) {
  return run_linear(req, true, stream);
}

LLP_API llp_status llp_beam_candidates(const llp_beam_request* req, const llp_beam_parts* out, void* stream) {
  float c1;
  llp_status st = check_beam(req, &c1);
  if (st != LLP_OK) return st;
  LLP_CHECK(out != nullptr, LLP_ERR_INVALID_ARGUMENT, "out is NULL");
  if (req->num_rows > 0)
    LLP_CHECK(out->value && out->token && out->max && out->sum, LLP_ERR_INVALID_ARGUMENT,
              "out.value, out.token, out.max and out.sum are required");
  st = check_device();
  if (st != LLP_OK) return st;
  BeamArgs a{};
  a.logits = req->logits;
  a.bf16 = req->logits_dtype == LLP_DTYPE_BF16;
  a.ld = req->logits_stride;
  a.rows = req->num_rows;
  a.n_real = local_real(req->vocab);
  a.offset = req->vocab.offset;
  a.num = req->num;
  a.blocks = (int32_t)(round_up(a.n_real, BEAM_BLOCK) / BEAM_BLOCK);
  a.c1 = c1;
  a.value = out->value;
  a.token = out->token;
  a.max = out->max;
  a.sum = out->sum;
  a.status = req->status_word;
  LLP_HIP(launch_beam_candidates(a, static_cast<hipStream_t>(stream)), "beam candidates kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_beam_select(const llp_beam_select_request* req, const llp_beam_out* out,
                                   void* stream) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  LLP_CHECK(req->world >= 1 && req->world <= LLP_MAX_WORLD, LLP_ERR_INVALID_ARGUMENT,
            "world %d outside [1, %d]", req->world, LLP_MAX_WORLD);
  LLP_CHECK(req->num_beams >= 1 && req->num_beams <= LLP_MAX_BEAMS, LLP_ERR_INVALID_ARGUMENT,
            "num_beams %d outside [1, %d]", req->num_beams, LLP_MAX_BEAMS);
  LLP_CHECK(req->num >= 1 && req->num <= LLP_MAX_BEAMS && req->num_out >= 1 && req->num_out <= LLP_MAX_BEAMS,
            LLP_ERR_INVALID_ARGUMENT, "num %d and num_out %d must be in [1, %d]", req->num, req->num_out,
            LLP_MAX_BEAMS);
  LLP_CHECK(req->num >= req->num_out, LLP_ERR_INVALID_ARGUMENT, "%d candidates a row for num_out %d", req->num,
            req->num_out);
  LLP_CHECK(req->num_seqs >= 0 && req->num_seqs < (int64_t(1) << 22), LLP_ERR_INVALID_ARGUMENT,
            "num_seqs %lld outside [0, 2^22)", (long long)req->num_seqs);
  float c1;
  llp_status st = check_beam_temperature(req->temperature, &c1);
  if (st != LLP_OK) return st;
  LLP_CHECK(req->parts != nullptr && out != nullptr, LLP_ERR_INVALID_ARGUMENT, "parts and out are required");
  BeamSelectArgs a{};
  if (req->num_seqs > 0) {
    LLP_CHECK(req->scores != nullptr, LLP_ERR_INVALID_ARGUMENT, "scores is NULL");
    LLP_CHECK(out->token && out->parent && out->score, LLP_ERR_INVALID_ARGUMENT,
              "out.token, out.parent and out.score are required");
    for (int32_t r = 0; r < req->world; ++r) {
      const llp_beam_parts& p = req->parts[r];
      LLP_CHECK(p.value && p.token && p.max && p.sum, LLP_ERR_INVALID_ARGUMENT,
                "parts[%d]: value, token, max and sum are required", r);
      a.value[r] = p.value;
      a.token[r] = p.token;
      a.max[r] = p.max;
      a.sum[r] = p.sum;
    }
  }
  st = check_device();
  if (st != LLP_OK) return st;
  a.world = req->world;
  a.num = req->num;
  a.K = req->num_beams;
  a.num_out = req->num_out;
  a.seqs = req->num_seqs;
  a.scores = req->scores;
  a.finished = req->finished;
  a.end_id = req->end_id;
  a.c1 = c1;
  a.out_token = out->token;
  a.out_parent = out->parent;
  a.out_score = out->score;
  a.status = req->status_word;
  LLP_HIP(launch_beam_select(a, static_cast<hipStream_t>(stream)), "beam select kernel launch");
  return LLP_OK;
}

LLP_API llp_status llp_beam_reorder(const llp_beam_reorder_request* req, void* stream) {
  LLP_CHECK(req != nullptr, LLP_ERR_INVALID_ARGUMENT, "request is NULL");
  const llp_beam_reorder_request& p = *req;
  LLP_CHECK(p.num_states >= 0 && p.num_seqs >= 0 && p.outer >= 0 && p.inner >= 0, LLP_ERR_INVALID_ARGUMENT,
            "a negative size");
  LLP_CHECK(p.num_src >= 1 && p.num_src <= LLP_MAX_BEAMS && p.num_out >= 1 && p.num_out <= LLP_MAX_BEAMS,
            LLP_ERR_INVALID_ARGUMENT, "num_src %d and num_out %d must be in [1, %d]", p.num_src, p.num_out,
            LLP_MAX_BEAMS);
  LLP_CHECK(p.num_seqs < (int64_t(1) << 22) && p.outer < kMaxStride && p.inner < kMaxStride,
            LLP_ERR_INVALID_ARGUMENT, "num_seqs, outer or inner out of range");
  for (int64_t s : {p.src_row_stride, p.src_outer_stride, p.dst_row_stride, p.dst_outer_stride})
    LLP_CHECK(s >= 0 && s < kMaxStride, LLP_ERR_INVALID_ARGUMENT, "stride %lld out of range", (long long)s);
  const bool work = p.num_states > 0 && p.num_seqs > 0 && p.outer > 0 && p.inner > 0;
  // Bytes per load: whatever every piece's start and length is a multiple of. (Slots past 32 would
  // not fit the registers 16 bytes at a time.)
  int64_t unit = p.num_out > 32 ? 4 : 16;
  if (work) {
    LLP_CHECK(p.src && p.dst && p.parents, LLP_ERR_INVALID_ARGUMENT, "src, dst and parents are required");
    LLP_CHECK(apart(p.num_seqs * p.num_out, p.outer, p.inner, p.dst_row_stride, p.dst_outer_stride),
              LLP_ERR_INVALID_ARGUMENT, "pieces of a state overlap");
    int64_t all = p.inner;
    if (p.num_seqs * p.num_src > 1) all |= p.src_row_stride;
    if (p.num_seqs * p.num_out > 1) all |= p.dst_row_stride;
    if (p.outer > 1) all |= p.src_outer_stride | p.dst_outer_stride;
    for (int32_t i = 0; i < p.num_states; ++i) {
      LLP_CHECK(p.src[i] && p.dst[i], LLP_ERR_INVALID_ARGUMENT, "state %d is NULL", i);
      LLP_CHECK((p.src[i] == p.dst[i]) == (p.src[0] == p.dst[0]), LLP_ERR_INVALID_ARGUMENT,
                "all states are reordered in place, or none");
      LLP_CHECK(p.src[i] != p.dst[i] || (p.num_src == p.num_out && p.src_row_stride == p.dst_row_stride &&
                                         p.src_outer_stride == p.dst_outer_stride),
                LLP_ERR_INVALID_ARGUMENT, "a reordering in place keeps number, strides and places of the slots");
      for (int32_t k = 0; k < i; ++k)
        LLP_CHECK(p.dst[k] != p.dst[i], LLP_ERR_INVALID_ARGUMENT, "states %d and %d are the same", k, i);
      all |= (int64_t)(reinterpret_cast<uintptr_t>(p.src[i]) | reinterpret_cast<uintptr_t>(p.dst[i]));
    }
    while (all % unit != 0) unit /= 2;
    if (unit == 8) unit = 4;
    if (unit == 2) unit = 1;
    // A launch holds fewer than 2^24 workgroups of 256 threads.
    const int64_t pieces = p.inner / unit;
    LLP_CHECK(pieces < kMaxStride / p.outer &&
                  (p.outer * pieces + 255) / 256 < (int64_t(1) << 24) / p.num_seqs,
              LLP_ERR_UNSUPPORTED, "a state of %lld pieces of %lld bytes for %lld sequences is too large",
              (long long)p.outer, (long long)p.inner, (long long)p.num_seqs);
  }
  llp_status st = check_device();
  if (st != LLP_OK) return st;
  if (!work) return LLP_OK;
  const int64_t per = (p.outer * (p.inner / unit) + 255) / 256 * p.num_seqs;
  int64_t most = ((int64_t(1) << 24) - 1) / per;   // states of one launch, within that limit
  if (most > REORDER_STATES) most = REORDER_STATES;
  for (int32_t i = 0; i < p.num_states; i += (int32_t)most) {
    ReorderArgs a{};
    a.states = (int32_t)(p.num_states - i < most ? p.num_states - i : most);
    for (int32_t k = 0; k < a.states; ++k) {
      a.src[k] = p.src[i + k];
      a.dst[k] = p.dst[i + k];
    }
    a.K = p.num_src;
    a.N = p.num_out;
    a.unit = (int32_t)unit;
    a.seqs = p.num_seqs;
    a.outer = p.outer;
    a.inner = p.inner;
    a.sr = p.src_row_stride;
    a.so = p.src_outer_stride;
    a.dr = p.dst_row_stride;
    a.dout = p.dst_outer_stride;
    a.parents = p.parents;
    a.status = p.status_word;
    LLP_HIP(launch_beam_reorder(a, static_cast<hipStream_t>(stream)), "beam reorder kernel launch");
  }
  return LLP_OK;
}

}  // extern "C"
