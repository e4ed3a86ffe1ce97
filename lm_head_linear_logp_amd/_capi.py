"""ctypes mirror of include/llp.h (structs, constants, function signatures)."""
from __future__ import annotations

import ctypes as C
import os

LLP_OK = 0
LLP_ERR_UNAVAILABLE = 1
LLP_ERR_INVALID_ARGUMENT = 2
LLP_ERR_UNSUPPORTED = 3
LLP_ERR_HIP = 4
LLP_ERR_INTERNAL = 5
STATUS_NAMES = {0: "OK", 1: "UNAVAILABLE", 2: "INVALID_ARGUMENT", 3: "UNSUPPORTED", 4: "HIP",
                5: "INTERNAL"}

LLP_STATUS_TARGET_OUT_OF_RANGE = 1
LLP_STATUS_TARGET_NOT_FOUND = 2
LLP_STATUS_REPLAY_ID_INVALID = 4
LLP_STATUS_LAYOUT_INVALID = 8
LLP_STATUS_TOKEN_OUT_OF_RANGE = 16
LLP_STATUS_VALUE_NOT_FINITE = 32
LLP_STATUS_PARENT_INVALID = 64

LLP_DTYPE_BF16 = 1
LLP_DTYPE_F32 = 2
LLP_OP_FORWARD = 1
LLP_OP_BACKWARD = 2
LLP_FLAG_WANT_ENTROPY = 1
LLP_FLAG_OVERWRITE_GRADS = 2
LLP_FLAG_G_SLABS = 4
LLP_G_SLAB_COLUMNS = 32768
LLP_MAX_REPLAY_IDS = 64
LLP_MAX_WORLD = 64
LLP_INT8_COLUMNS = 128
LLP_FP8_BLOCK = 128
LLP_MAX_BEAMS = 64
LLP_KL_K1, LLP_KL_K2, LLP_KL_K3 = 1, 2, 3
LLP_REDUCE_TOKEN_MEAN, LLP_REDUCE_SEQ_MEAN, LLP_REDUCE_SUM = 1, 2, 3
LLP_LOG_RATIO_MAX = 20
LLP_POLICY_STATS = 8
LLP_PREF_SIGMOID, LLP_PREF_HINGE, LLP_PREF_IPO = 1, 2, 3

vp = C.c_void_p


class llp_info(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("version", C.c_char * 16), ("arch", C.c_char * 32),
                ("route", C.c_char * 128), ("max_replay_ids", C.c_int32),
                ("num_cus", C.c_int32), ("device", C.c_int32), ("reserved", C.c_int32)]


class llp_projection(C.Structure):
    _fields_ = [("hidden", vp), ("hidden_stride", C.c_int64), ("weight", vp),
                ("weight_stride", C.c_int64), ("bias", vp), ("bias_dtype", C.c_int32),
                ("reserved", C.c_int32), ("hidden_size", C.c_int64)]


class llp_vocab_partition(C.Structure):
    _fields_ = [("offset", C.c_int64), ("local_size", C.c_int64), ("real_vocab", C.c_int64),
                ("padded_vocab", C.c_int64), ("rank", C.c_int32), ("world", C.c_int32)]


class llp_token_layout(C.Structure):
    _fields_ = [("num_tokens", C.c_int64), ("num_seqs", C.c_int32), ("reserved", C.c_int32),
                ("cu_seqlens", vp), ("loss_mask", vp)]


class llp_request(C.Structure):
    _fields_ = [("proj", llp_projection), ("vocab", llp_vocab_partition),
                ("layout", llp_token_layout), ("target_ids", vp), ("temperature", C.c_float),
                ("flags", C.c_uint32), ("status_word", vp)]


class llp_partials(C.Structure):
    _fields_ = [("target_logit", vp), ("in_range", vp), ("lse", vp), ("entropy", vp),
                ("logp", vp)]


class llp_final_out(C.Structure):
    _fields_ = [("logp", vp), ("lse", vp), ("entropy", vp)]


class llp_bwd_in(C.Structure):
    _fields_ = [("lse", vp), ("dlogp", vp), ("dentropy", vp), ("entropy", vp)]


class llp_bwd_out(C.Structure):
    _fields_ = [("dhidden", vp), ("dhidden_stride", C.c_int64), ("dweight", vp),
                ("dweight_stride", C.c_int64), ("dbias", vp)]


class llp_topp_request(C.Structure):
    _fields_ = [("logits", vp), ("logits_dtype", C.c_int32), ("num_replay", C.c_int32),
                ("logits_stride", C.c_int64), ("num_tokens", C.c_int64),
                ("vocab", llp_vocab_partition), ("replay_ids", vp), ("replay_stride", C.c_int64),
                ("target_ids", vp), ("loss_mask", vp), ("temperature", C.c_float),
                ("processed_logprobs", C.c_int32), ("status_word", vp)]


class llp_logits_request(C.Structure):
    _fields_ = [("logits", vp), ("logits_dtype", C.c_int32), ("reserved", C.c_int32),
                ("logits_stride", C.c_int64), ("vocab", llp_vocab_partition),
                ("layout", llp_token_layout), ("target_ids", vp), ("temperature", C.c_float),
                ("flags", C.c_uint32), ("status_word", vp)]


class llp_keep_mask_request(C.Structure):
    _fields_ = [("logits", vp), ("logits_dtype", C.c_int32), ("processed_logprobs", C.c_int32),
                ("logits_stride", C.c_int64), ("keep_mask", vp), ("keep_stride", C.c_int64),
                ("num_tokens", C.c_int64), ("vocab", llp_vocab_partition), ("target_ids", vp),
                ("loss_mask", vp), ("temperature", C.c_float), ("reserved", C.c_int32),
                ("status_word", vp)]


class llp_quant_request(C.Structure):
    _fields_ = [("x", vp), ("x_dtype", C.c_int32), ("reserved", C.c_int32),
                ("x_stride", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64), ("q", vp),
                ("q_stride", C.c_int64), ("scale", vp)]


class llp_int8_request(C.Structure):
    _fields_ = [("hidden", vp), ("hidden_stride", C.c_int64), ("hidden_scale", vp),
                ("weight", vp), ("weight_stride", C.c_int64), ("weight_scale", vp),
                ("bias", vp), ("bias_dtype", C.c_int32), ("flags", C.c_uint32),
                ("hidden_size", C.c_int64), ("vocab", llp_vocab_partition),
                ("layout", llp_token_layout), ("target_ids", vp), ("temperature", C.c_float),
                ("reserved", C.c_int32), ("status_word", vp)]


class llp_policy_request(C.Structure):
    _fields_ = [("logp", vp), ("old_logp", vp), ("advantages", vp), ("ref_logp", vp),
                ("entropy", vp), ("layout", llp_token_layout), ("clip_low", C.c_double),
                ("clip_high", C.c_double), ("dual_clip", C.c_double), ("kl_coef", C.c_double),
                ("entropy_coef", C.c_double), ("kl_kind", C.c_int32), ("reduction", C.c_int32),
                ("denominator", vp), ("status_word", vp)]


class llp_policy_out(C.Structure):
    _fields_ = [("loss", vp), ("stats", vp), ("dloss", vp), ("dlogp", vp), ("dentropy", vp)]


class llp_pref_request(C.Structure):
    _fields_ = [("logp", vp), ("ref_logp", vp), ("pair_weight", vp),
                ("layout", llp_token_layout), ("beta", C.c_double), ("gamma", C.c_double),
                ("label_smoothing", C.c_double), ("kind", C.c_int32), ("average", C.c_int32),
                ("reduction", C.c_int32), ("reserved", C.c_int32), ("status_word", vp)]


class llp_pref_out(C.Structure):
    _fields_ = [("loss", vp), ("pair_loss", vp), ("chosen", vp), ("rejected", vp),
                ("dloss", vp), ("dlogp", vp)]


class llp_embedding_request(C.Structure):
    _fields_ = [("token_ids", vp), ("token_mask", vp), ("num_tokens", C.c_int64),
                ("vocab", llp_vocab_partition), ("hidden_size", C.c_int64),
                ("scale", C.c_float), ("flags", C.c_uint32), ("status_word", vp)]


class llp_fp8_quant_request(C.Structure):
    _fields_ = [("x", vp), ("x_dtype", C.c_int32), ("block_rows", C.c_int32),
                ("x_stride", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("transpose", C.c_int32), ("reserved", C.c_int32), ("q", vp),
                ("q_stride", C.c_int64), ("scale", vp), ("scale_stride", C.c_int64)]


class llp_fp8_linear_request(C.Structure):
    _fields_ = [("x", vp), ("x_stride", C.c_int64), ("x_scale", vp), ("x_scale_stride", C.c_int64),
                ("weight", vp), ("weight_stride", C.c_int64), ("weight_scale", vp),
                ("weight_scale_stride", C.c_int64), ("bias", vp), ("bias_dtype", C.c_int32),
                ("out_dtype", C.c_int32), ("out", vp), ("out_stride", C.c_int64),
                ("rows", C.c_int64), ("cols", C.c_int64), ("depth", C.c_int64),
                ("flags", C.c_uint32), ("reserved", C.c_int32)]


class llp_beam_request(C.Structure):
    _fields_ = [("logits", vp), ("logits_dtype", C.c_int32), ("num", C.c_int32),
                ("logits_stride", C.c_int64), ("num_rows", C.c_int64),
                ("vocab", llp_vocab_partition), ("temperature", C.c_float),
                ("reserved", C.c_int32), ("status_word", vp)]


class llp_beam_parts(C.Structure):
    _fields_ = [("value", vp), ("token", vp), ("max", vp), ("sum", vp)]


class llp_beam_select_request(C.Structure):
    _fields_ = [("world", C.c_int32), ("num", C.c_int32), ("parts", C.POINTER(llp_beam_parts)),
                ("num_seqs", C.c_int64), ("num_beams", C.c_int32), ("num_out", C.c_int32),
                ("scores", vp), ("finished", vp), ("end_id", C.c_int64),
                ("temperature", C.c_float), ("reserved", C.c_int32), ("status_word", vp)]


class llp_beam_out(C.Structure):
    _fields_ = [("token", vp), ("parent", vp), ("score", vp)]


class llp_beam_reorder_request(C.Structure):
    _fields_ = [("src", C.POINTER(vp)), ("dst", C.POINTER(vp)), ("num_states", C.c_int32),
                ("num_src", C.c_int32), ("num_out", C.c_int32), ("reserved", C.c_int32),
                ("num_seqs", C.c_int64), ("outer", C.c_int64), ("inner", C.c_int64),
                ("src_row_stride", C.c_int64), ("src_outer_stride", C.c_int64),
                ("dst_row_stride", C.c_int64), ("dst_outer_stride", C.c_int64), ("parents", vp),
                ("status_word", vp)]


SIGNATURES = {
    "llp_open": (C.c_int, [C.c_int32, C.POINTER(llp_info)]),
    "llp_workspace_bytes": (C.c_int, [C.POINTER(llp_request), C.c_int32, C.POINTER(C.c_size_t)]),
    "llp_forward": (C.c_int, [C.POINTER(llp_request), C.POINTER(llp_partials), vp, C.c_size_t, vp]),
    "llp_forward_noalloc": (C.c_int, [C.POINTER(llp_request), C.POINTER(llp_partials), vp]),
    "llp_merge": (C.c_int, [C.c_int32, C.POINTER(llp_partials), C.c_int64, vp,
                            C.POINTER(llp_final_out), vp, vp]),
    "llp_backward": (C.c_int, [C.POINTER(llp_request), C.POINTER(llp_bwd_in),
                               C.POINTER(llp_bwd_out), vp, C.c_size_t, vp]),
    "llp_top_p_replay": (C.c_int, [C.POINTER(llp_topp_request), C.POINTER(llp_partials), vp]),
    "llp_forward_logits": (C.c_int, [C.POINTER(llp_logits_request), C.POINTER(llp_partials), vp]),
    "llp_keep_mask_replay": (C.c_int, [C.POINTER(llp_keep_mask_request), C.POINTER(llp_partials),
                                       vp]),
    "llp_quantize_rows": (C.c_int, [C.POINTER(llp_quant_request), vp]),
    "llp_int8_workspace_bytes": (C.c_int, [C.POINTER(llp_int8_request), C.POINTER(C.c_size_t)]),
    "llp_forward_int8": (C.c_int, [C.POINTER(llp_int8_request), C.POINTER(llp_partials), vp,
                                   C.c_size_t, vp]),
    "llp_policy_workspace_bytes": (C.c_int, [C.POINTER(llp_policy_request),
                                             C.POINTER(C.c_size_t)]),
    "llp_policy_loss": (C.c_int, [C.POINTER(llp_policy_request), C.POINTER(llp_policy_out), vp,
                                  C.c_size_t, vp]),
    "llp_preference_workspace_bytes": (C.c_int, [C.POINTER(llp_pref_request),
                                                 C.POINTER(C.c_size_t)]),
    "llp_preference_loss": (C.c_int, [C.POINTER(llp_pref_request), C.POINTER(llp_pref_out), vp,
                                      C.c_size_t, vp]),
    "llp_embedding": (C.c_int, [C.POINTER(llp_embedding_request), vp, C.c_int32, C.c_int64, vp,
                                C.c_int64, vp]),
    "llp_embedding_workspace_bytes": (C.c_int, [C.POINTER(llp_embedding_request),
                                                C.POINTER(C.c_size_t)]),
    "llp_embedding_backward": (C.c_int, [C.POINTER(llp_embedding_request), vp, C.c_int32,
                                         C.c_int64, vp, C.c_int64, vp, C.c_size_t, vp]),
    "llp_quantize_blocks": (C.c_int, [C.POINTER(llp_fp8_quant_request), vp]),
    "llp_quantize_both": (C.c_int, [C.POINTER(llp_fp8_quant_request), C.POINTER(llp_fp8_quant_request), vp]),
    "llp_linear_fp8": (C.c_int, [C.POINTER(llp_fp8_linear_request), vp]),
    "llp_dweight_fp8": (C.c_int, [C.POINTER(llp_fp8_linear_request), vp]),
    "llp_beam_candidates": (C.c_int, [C.POINTER(llp_beam_request), C.POINTER(llp_beam_parts), vp]),
    "llp_beam_select": (C.c_int, [C.POINTER(llp_beam_select_request), C.POINTER(llp_beam_out),
                                  vp]),
    "llp_beam_reorder": (C.c_int, [C.POINTER(llp_beam_reorder_request), vp]),
    "llp_last_error": (C.c_char_p, []),
}

# The in-tree build; LLP_LIBRARY may name another build of the same sources.
LIB_PATH = os.environ.get("LLP_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libllp.so")
_lib = None


def load() -> C.CDLL:
    """Load the in-tree HIP library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                           "(python -m lm_head_linear_logp_amd.build)")
    lib = C.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
