"""Operators that decode and train with a head in 8-bit floating point (include/llp.h): block
quantisation, products of such operands with their gradients, and one step of a beam search.
Argument marshalling, as in ops.py: every tensor is checked here, every step runs in libllp.so on the
tensors' own device and that device's current stream. fp8_linear alone records a gradient: the other calls read and
write tensors as they are, and a caller's tensor that one writes counts as changed in place, so that a
backward pass which saved it before is refused."""
from __future__ import annotations

import ctypes as C
import functools
from typing import NamedTuple, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version as _changed

from . import _capi as A
from . import _need, _ptr, _status, _vocab
from .ops import _DTYPE, _F32, _I32, _I64, _U8, _at, _call, _ready, _tensor

_F8, _F64 = torch.float8_e4m3fn, torch.float64
_BLOCK = A.LLP_FP8_BLOCK


def _stride(t, rows, width):
    """Row stride of a matrix (its own width where it holds no second row, or nothing)."""
    return t.stride(0) if rows > 1 and width > 0 else width


def _blocks(n):
    return -(-n // _BLOCK)


def _rows(t, name):
    """A bf16 or fp32 matrix whose rows are contiguous and apart."""
    _tensor(t, name)
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be a bf16 or fp32 tensor, got {t.dtype}")
    dev = t.device
    if not (t.dim() == 2 and t.is_contiguous()):
        _need(t, name, t.dtype, 2, dev)
    return dev


# ---- Products in 8-bit floating point ----------------------------------------------------------
def _scale_stride(t, name, rows, depth, by_block, dev):
    """Stride of an operand's scales [rows or their blocks, depth / 128]: by group the rows are
    contiguous (as quantize_blocks lays them out), by block the groups are."""
    shape = (_blocks(rows) if by_block else rows, depth // _BLOCK)
    if not (type(t) is torch.Tensor and t.dtype is _F32 and t.device == dev and t.shape == shape):
        _tensor(t, name)
        if t.dtype != _F32 or t.device != dev:
            raise TypeError(f"{name} must be an fp32 tensor on {dev}, got {t.dtype} on {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    n, groups = shape
    inner, outer = (1, 0) if by_block else (0, 1)
    if shape[inner] > 1 and t.stride(inner) != 1:
        raise ValueError(f"{name} must be contiguous along " + ("its groups" if by_block else
                         "its rows (quantize_blocks returns it so)"))
    return t.stride(outer) if shape[outer] > 1 else max(shape[inner], 1)


def quantize_blocks(x: torch.Tensor, *, rows: int = 1, transpose: bool = False,
                    out: Optional[tuple] = None) -> tuple:
    """llp_quantize_blocks: a bf16 or fp32 matrix (or, with transpose, its transpose) [M, K] in e4m3
    with an fp32 scale for each `rows` (1 or 128) by 128 values. Returns (q, scale): float8_e4m3fn
    [M, K rounded up to 128] (0 past K) and fp32 [M / rows rounded up, K / 128 rounded up], so that
    q[m, k] * scale[m // rows, k // 128] stands for the value. With rows = 1 the scale's storage is
    the other way round (a transposed view), which is how linear_fp8 reads it. `out`: the two tensors
    to write."""
    dev = _rows(x, "x")
    R, Cc = x.shape
    M, K = (Cc, R) if transpose else (R, Cc)
    if rows not in (1, _BLOCK):
        raise ValueError(f"rows must be 1 or {_BLOCK}, got {rows!r}")
    G = _blocks(K)
    if out is not None:
        q, scale = out
        _need(q, "out[0]", _F8, 2, dev, (M, G * _BLOCK))
        lds = _scale_stride(scale, "out[1]", M, G * _BLOCK, rows != 1, dev)
    _ready(dev)
    if out is None:
        q = torch.empty(M, G * _BLOCK, dtype=_F8, device=dev)
        if rows == 1:
            lds = max(M, 1)
            scale = torch.empty_strided((M, G), (1, lds), dtype=_F32, device=dev)
        else:
            scale, lds = torch.empty(_blocks(M), G, dtype=_F32, device=dev), max(G, 1)
    req = A.llp_fp8_quant_request(x.data_ptr(), _DTYPE[x.dtype], rows, _stride(x, R, Cc), R, Cc,
                                  1 if transpose else 0, 0, q.data_ptr(), _stride(q, M, G * _BLOCK),
                                  scale.data_ptr(), lds)
    _call(dev, "llp_quantize_blocks", C.byref(req))
    if out is not None:
        _changed((q, scale))
    return q, scale


def quantize_both(x: torch.Tensor) -> tuple:
    """llp_quantize_both: ``quantize_blocks(x)`` and ``quantize_blocks(x, rows=128, transpose=True)`` in one
    pass over x: what the input's and the weight's gradient take of an upstream gradient. Returns
    (q, scale, q_t, scale_t)."""
    dev = _rows(x, "x")
    R, Cc = x.shape
    _ready(dev)
    G, Gt = _blocks(Cc), _blocks(R)
    q = torch.empty(R, G * _BLOCK, dtype=_F8, device=dev)
    scale = torch.empty_strided((R, G), (1, max(R, 1)), dtype=_F32, device=dev)
    q_t = torch.empty(Cc, Gt * _BLOCK, dtype=_F8, device=dev)
    scale_t = torch.empty(G, Gt, dtype=_F32, device=dev)
    at, dt, ld = x.data_ptr(), _DTYPE[x.dtype], _stride(x, R, Cc)
    groups = A.llp_fp8_quant_request(at, dt, 1, ld, R, Cc, 0, 0, q.data_ptr(), G * _BLOCK,
                                     scale.data_ptr(), max(R, 1))
    blocks = A.llp_fp8_quant_request(at, dt, _BLOCK, ld, R, Cc, 1, 0, q_t.data_ptr(), Gt * _BLOCK,
                                     scale_t.data_ptr(), Gt)
    _call(dev, "llp_quantize_both", C.byref(groups), C.byref(blocks))
    return q, scale, q_t, scale_t


def _product(x, x_scale, weight, weight_scale, names):
    """The request of a product of two e4m3 operands."""
    dev = _tensor(x, names[0]).device
    if not (x.dtype is _F8 and x.dim() == 2 and x.is_contiguous()):
        _need(x, names[0], _F8, 2, dev)
    T, K = x.shape
    if not (type(weight) is torch.Tensor and weight.dtype is _F8 and weight.dim() == 2 and weight.device == dev
            and weight.shape[1] == K and weight.is_contiguous()):
        _need(weight, names[1], _F8, 2, dev, (None, K))
    V = weight.shape[0]
    if K % _BLOCK:
        raise ValueError(f"{names[0]} has {K} columns, not a multiple of {_BLOCK}")
    r = A.llp_fp8_linear_request()
    r.x, r.x_stride = x.data_ptr(), _stride(x, T, K)
    r.x_scale, r.x_scale_stride = _ptr(x_scale), _scale_stride(x_scale, names[0] + "_scale", T, K, False, dev)
    r.weight, r.weight_stride = weight.data_ptr(), _stride(weight, V, K)
    r.weight_scale, r.weight_scale_stride = _ptr(weight_scale), _scale_stride(
        weight_scale, names[1] + "_scale", V, K, True, dev)
    r.rows, r.cols, r.depth = T, V, K
    return r, dev, T, V


def linear_fp8(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor,
               weight_scale: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """llp_linear_fp8: x . weight^T + bias of operands as quantize_blocks gives them, x [T, K] with
    rows=1 and weight [V, K] with rows=128, summed in fp32 and rounded once to out_dtype (bf16 or
    fp32). Into bf16 the 8-bit matrix instructions add a group's products, with about 14 bits below the
    largest: results whose products nearly cancel keep fewer than bf16's bits. With the weight quantised
    transposed it is the input gradient. An allocated result has
    rows of a multiple of 16 bytes (a view [T, V] where V is not), as the calls that read logits
    take them."""
    r, dev, T, V = _product(x, x_scale, weight, weight_scale, ("x", "weight"))
    if out is not None:
        _rows(out, "out")
        _need(out, "out", out.dtype, 2, dev, (T, V))
        out_dtype = out.dtype
    elif out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype must be bf16 or fp32, got {out_dtype}")
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype not in _DTYPE:
            raise TypeError("bias must be a bf16 or fp32 tensor")
        r.bias, r.bias_dtype = _at(bias, "bias", bias.dtype, V, dev), _DTYPE[bias.dtype]
    _ready(dev)
    given = out is not None
    if not given:
        width = V + -V % (4 if out_dtype == _F32 else 8)
        out = torch.empty_strided((T, V), (width, 1), dtype=out_dtype, device=dev)
    r.out, r.out_dtype, r.out_stride = out.data_ptr(), _DTYPE[out_dtype], _stride(out, T, V)
    _call(dev, "llp_linear_fp8", C.byref(r))
    if given:
        _changed(out)
    return out


def dweight_fp8(dout_t: torch.Tensor, dout_scale: torch.Tensor, x_t: torch.Tensor,
                x_scale: torch.Tensor, *, dweight: Optional[torch.Tensor] = None,
                overwrite: bool = False, out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """llp_dweight_fp8: dweight (fp32 [V, H]) += dout^T . x with both operands quantised transposed,
    dout_t [V, T] in blocks (rows=128) and x_t [H, T] in groups (rows=1). overwrite=True writes
    instead, and then dweight may be bf16. A missing dweight is allocated in out_dtype.
    A block's largest entry sets the scale of 128 columns and 128 tokens of dout, so that of a softmax's
    gradient most small entries go to 0 beside the targets'. Where that matters
    ``linear_fp8(*quantize_blocks(dout, transpose=True), *quantize_blocks(x, rows=128, transpose=True))``
    is the same product with a scale for each column's 128 tokens of dout, and blocks along x."""
    r, dev, H, V = _product(x_t, x_scale, dout_t, dout_scale, ("x_t", "dout_t"))
    if dweight is None:
        overwrite = True
        if out_dtype not in _DTYPE:
            raise TypeError(f"out_dtype must be bf16 or fp32, got {out_dtype}")
    else:
        _rows(dweight, "dweight")
        _need(dweight, "dweight", dweight.dtype, 2, dev, (V, H))
        out_dtype = dweight.dtype
        if out_dtype != _F32 and not overwrite:
            raise TypeError("a dweight that is added to must be fp32")
    r.flags = A.LLP_FLAG_OVERWRITE_GRADS if overwrite else 0
    _ready(dev)
    given = dweight is not None
    if not given:
        dweight = torch.empty(V, H, dtype=out_dtype, device=dev)
    r.out, r.out_dtype, r.out_stride = dweight.data_ptr(), _DTYPE[out_dtype], _stride(dweight, V, H)
    _call(dev, "llp_dweight_fp8", C.byref(r))
    if given:
        _changed(dweight)
    return dweight


class _Fp8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, out_dtype):
        ctx.save_for_backward(x, weight)
        return linear_fp8(*quantize_blocks(x), *quantize_blocks(weight, rows=_BLOCK),
                          out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight = ctx.saved_tensors
        # An expanded or transposed upstream gradient.
        if dy.stride(1) != 1 or dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()
        dx = dw = None
        want_x, want_w = ctx.needs_input_grad[:2]
        if want_x and want_w:
            q, scale, q_t, scale_t = quantize_both(dy)
        elif want_x:
            q, scale = quantize_blocks(dy)
        else:
            q_t, scale_t = quantize_blocks(dy, rows=_BLOCK, transpose=True)
        if want_x:
            dx = linear_fp8(q, scale, *quantize_blocks(weight, rows=_BLOCK, transpose=True), out_dtype=x.dtype)
        if want_w:
            dw = dweight_fp8(q_t, scale_t, *quantize_blocks(x, transpose=True), out_dtype=weight.dtype)
        return dx, dw, None


def fp8_linear(x: torch.Tensor, weight: torch.Tensor, *,
               out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """x . weight^T as an autograd node whose three products run in 8-bit floating point: x of any
    shape [..., K] and weight [V, K], bf16 or fp32, quantised here (x, and the upstream gradient, in
    groups of 128; the weight in blocks of 128 x 128; along the tokens, for the weight gradient, the
    upstream gradient in blocks, see ``dweight_fp8`` for what that costs, and x in groups). Gradients
    are those of the product at the quantised operands, in x's and weight's own dtypes, summed as
    ``linear_fp8`` does."""
    _tensor(x, "x")
    dev = _rows(weight, "weight")
    if x.dtype not in _DTYPE:
        raise TypeError(f"x must be a bf16 or fp32 tensor, got {x.dtype}")
    if x.device != dev:
        raise ValueError(f"x is on {x.device}, weight on {dev}")
    if x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x is {tuple(x.shape)}, weight {tuple(weight.shape)}")
    if out_dtype is None:
        out_dtype = x.dtype
    flat = x.reshape(-1, x.shape[-1]) if x.shape[-1] else x.reshape(x.shape[:-1].numel(), 0)
    if flat.numel() and (flat.stride(1) != 1 or (flat.shape[0] > 1 and flat.stride(0) < flat.shape[1])):
        flat = flat.contiguous()
    return _Fp8Linear.apply(flat, weight, out_dtype).reshape(*x.shape[:-1], weight.shape[0])


# ---- Beam search -----------------------------------------------------------------------------
_PARTS = (("value", _F32), ("token", _I64), ("max", _F32), ("sum", _F64))


def _check_parts(p, name, rows, num, dev):
    v, i, m, s = p["value"], p["token"], p["max"], p["sum"]
    if (type(v) is type(i) is type(m) is type(s) is torch.Tensor
            and v.dtype is _F32 and i.dtype is _I64 and m.dtype is _F32 and s.dtype is _F64
            and v.shape == i.shape == (rows, num) and m.shape == s.shape == (rows,)
            and v.device == i.device == m.device == s.device == dev and v.is_contiguous()
            and i.is_contiguous() and m.is_contiguous() and s.is_contiguous()):
        return
    for k, dt in _PARTS:
        shape = (rows, num) if k in ("value", "token") else (rows,)
        _need(p[k], f"{name}['{k}']", dt, len(shape), dev, shape)
        if not p[k].is_contiguous():
            raise ValueError(f"{name}['{k}'] must be contiguous")


def _part_pointers(p):
    return A.llp_beam_parts(p["value"].data_ptr(), p["token"].data_ptr(), p["max"].data_ptr(),
                            p["sum"].data_ptr())


def _num(n, name):
    if not isinstance(n, int) or not 1 <= n <= A.LLP_MAX_BEAMS:
        raise ValueError(f"{name} must be a whole number in [1, {A.LLP_MAX_BEAMS}], got {n!r}")
    return n


def beam_candidates(logits: torch.Tensor, num: int, *, temperature: float = 1.0, offset: int = 0,
                    real_vocab: Optional[int] = None, padded_vocab: Optional[int] = None,
                    rank: int = 0, world: int = 1, status: Optional[torch.Tensor] = None,
                    out: Optional[dict] = None) -> dict:
    """llp_beam_candidates on one vocabulary shard: the `num` most likely tokens of each row of
    logits [rows, local_size] (bf16 or fp32, rows 16-byte aligned) and what normalises the row.
    Returns value (logits) and token (global ids) [rows, num], most likely first, ties to the lowest
    id, -inf and -1 past a row's last candidate; max fp32 and sum fp64 [rows]. For ``beam_select``,
    with the shards' results in rank order. A row that holds a NaN or +inf has no candidates, sum -1,
    and sets VALUE_NOT_FINITE in `status`."""
    dev = _rows(logits, "logits")
    R, V = logits.shape
    r = A.llp_beam_request()
    r.logits, r.logits_dtype, r.num = logits.data_ptr(), _DTYPE[logits.dtype], _num(num, "num")
    r.logits_stride, r.num_rows = _stride(logits, R, V), R
    _vocab(r.vocab, offset, V, real_vocab, padded_vocab, rank, world)
    r.temperature = float(temperature)
    _status(status, dev)
    r.status_word = _ptr(status)
    if out is not None:
        _check_parts(out, "out", R, num, dev)
    _ready(dev)
    given = out is not None
    if not given:
        out = dict(value=torch.empty(R, num, dtype=_F32, device=dev),
                   token=torch.empty(R, num, dtype=_I64, device=dev),
                   max=torch.empty(R, dtype=_F32, device=dev),
                   sum=torch.empty(R, dtype=_F64, device=dev))
    _call(dev, "llp_beam_candidates", C.byref(r), C.byref(_part_pointers(out)))
    if given:
        _changed(tuple(out[k] for k, _ in _PARTS))
    return out


def beam_select(parts: Sequence[dict], scores: torch.Tensor, num: Optional[int] = None, *,
                temperature: float = 1.0, finished: Optional[torch.Tensor] = None,
                end_id: Optional[int] = None, status: Optional[torch.Tensor] = None,
                out: Optional[dict] = None) -> dict:
    """llp_beam_select: for each of B sequences of K beams the `num` best continuations (K of them by
    default) over its beams and the vocabulary, from the ``beam_candidates`` of every shard (rank
    order; B * K rows, at least `num` candidates each, the same temperature). scores fp32 [B, K]:
    the beams' sums of log-probabilities so far (-inf: a beam that is not there, as all but the
    first are at the start). finished uint8 [B, K]: beams that ended; each goes on with `end_id` at
    its own score. Returns token int64, parent int32 (the beam continued) and score fp32, [B, num],
    best first, ties to the lowest beam and token; where too few candidates are there token and
    parent are -1 and the score is -inf."""
    if isinstance(parts, dict):
        raise TypeError("parts is a sequence: the shards' results of beam_candidates in rank order")
    world = len(parts)
    if not 1 <= world <= A.LLP_MAX_WORLD:
        raise ValueError(f"beam_select takes 1 to {A.LLP_MAX_WORLD} shards, got {world}")
    dev = _tensor(scores, "scores").device
    if not (scores.dtype is _F32 and scores.dim() == 2 and scores.is_contiguous()):
        _need(scores, "scores", _F32, 2, dev)
        raise ValueError("scores must be contiguous")
    B, K = scores.shape
    _num(K, "the number of beams")
    num = _num(K if num is None else num, "num")
    each = _tensor(parts[0]["value"], "parts[0]['value']").shape
    if len(each) != 2 or each[1] < num:
        raise ValueError(f"parts[0]['value'] has shape {tuple(each)}: {num} candidates a row are needed")
    arr = (A.llp_beam_parts * world)()
    for i, p in enumerate(parts):
        _check_parts(p, f"parts[{i}]", B * K, each[1], dev)
        arr[i] = _part_pointers(p)
    r = A.llp_beam_select_request()
    r.world, r.num, r.parts = world, _num(int(each[1]), "candidates a row"), arr
    r.num_seqs, r.num_beams, r.num_out = B, K, num
    r.scores = scores.data_ptr()
    if finished is not None:
        if end_id is None:
            raise ValueError("finished needs end_id")
        _need(finished, "finished", _U8, 2, dev, (B, K))
        if not finished.is_contiguous():
            raise ValueError("finished must be contiguous")
        r.finished, r.end_id = finished.data_ptr(), int(end_id)
    r.temperature = float(temperature)
    _status(status, dev)
    r.status_word = _ptr(status)
    if out is not None:
        for k, dt in (("token", _I64), ("parent", _I32), ("score", _F32)):
            _need(out[k], f"out['{k}']", dt, 2, dev, (B, num))
            if not out[k].is_contiguous():
                raise ValueError(f"out['{k}'] must be contiguous")
    _ready(dev)
    given = out is not None
    if not given:
        out = dict(token=torch.empty(B, num, dtype=_I64, device=dev),
                   parent=torch.empty(B, num, dtype=_I32, device=dev),
                   score=torch.empty(B, num, dtype=_F32, device=dev))
    o = A.llp_beam_out(out["token"].data_ptr(), out["parent"].data_ptr(), out["score"].data_ptr())
    _call(dev, "llp_beam_select", C.byref(r), C.byref(o))
    if given:
        _changed((out["token"], out["parent"], out["score"]))
    return out


def _pieces(shape, *strides):
    """A state's dims behind the first as (outer, inner, outer stride of each tensor), in elements;
    None where they are not pieces at one stride."""
    dims = []
    for i, n in enumerate(shape):
        if n == 1:
            continue
        here = tuple(s[i] for s in strides)
        if dims and all(d == s * n for d, s in zip(dims[-1][1], here)):
            dims[-1] = (dims[-1][0] * n, here)
        else:
            dims.append((n, here))
    one = (1,) * len(strides)
    if dims and dims[-1][1] == one:
        inner = dims.pop()[0]
    else:
        inner = 1
    if len(dims) > 1:
        return None
    return (dims[0][0], inner, dims[0][1]) if dims else (1, inner, (0,) * len(strides))


class _Layout(NamedTuple):
    """States' pieces: beams K of a sequence read, rows written, strides and lengths in bytes; `levels`:
    the strides written, largest first, each with the bytes of what lies within one step."""
    K: int
    rows: int
    outer: int
    inner: int
    sr: int
    so: int
    dr: int
    do: int
    extent: int
    src_extent: int
    levels: tuple


@functools.lru_cache(maxsize=1024)
def _reorder_layout(shape, stride, to_shape, to_stride, size, B, N, in_place):
    """The layout of a state and what it goes to, or None where there is nothing to move."""
    if len(shape) < 1 or shape[1:] != to_shape[1:]:
        raise ValueError("and what it goes to must be alike but for their rows")
    if to_shape[0] != B * N or (shape[0] % B if B else shape[0]):
        raise ValueError(f"has {shape[0]} rows, to be written {to_shape[0]}: {B} sequences of {N} "
                         "are expected")
    if 0 in to_shape:
        return None
    if shape[0] == 0:
        raise ValueError("holds no rows")
    p = _pieces(shape[1:], stride[1:], to_stride[1:])
    if p is None:
        raise ValueError(f"of strides {stride} is not rows of pieces at one stride")
    outer, inner, rows = p[0], p[1] * size, to_shape[0]
    so, do = (st * size for st in p[2])
    K = _num(shape[0] // B, "beams per sequence")
    dr = to_stride[0] * size if rows > 1 else 0
    sr = dr if in_place else stride[0] * size if shape[0] > 1 else 0
    reach, levels = inner, ()
    for st, n in sorted((st, n) for st, n in ((dr, rows), (do, outer)) if n > 1):
        if st < reach:
            raise ValueError("has rows to be written that overlap")
        levels = ((st, reach), *levels)
        reach += (n - 1) * st
    return _Layout(K, rows, outer, inner, sr, so, dr, do, reach, (shape[0] - 1) * sr + (outer - 1) * so + inner,
                   levels)


def beam_reorder(states, parents: torch.Tensor, *, out=None, status: Optional[torch.Tensor] = None):
    """llp_beam_reorder: what is kept per beam follows the beams that were chosen. states: a tensor
    or a sequence of them, of any dtype, [B * K, ...] with the beams of a sequence in consecutive
    rows; parents int32 [B, N] (``beam_select``'s). In place (N = K) row b * N + j takes row
    b * K + parents[b, j] as it was before the call; with `out` (the like of states, [B * N, ...], none
    between a state's first byte and its last) the rows go there. A parent of -1 leaves the row as it
    is; one past the beams does too and sets PARENT_INVALID in `status`. A state may be a view: its dims behind the first are
    contiguous, or pieces at one stride, as a cache [rows, heads, room, dim] cut to its length is.
    Returns the tensors written."""
    single = isinstance(states, torch.Tensor)
    src = [states] if single else list(states)
    dst = src if out is None else [out] if isinstance(out, torch.Tensor) else list(out)
    if len(dst) != len(src):
        raise ValueError(f"{len(src)} states and {len(dst)} tensors to write")
    dev = _tensor(parents, "parents").device
    _need(parents, "parents", _I32, 2, dev)
    B, N = parents.shape
    _num(N, "parents per sequence")
    if not parents.is_contiguous():
        raise ValueError("parents must be contiguous")
    _status(status, dev)
    calls, seen, last = {}, [], None   # states of one layout go together
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (isinstance(s, torch.Tensor) and isinstance(d, torch.Tensor)):
            raise TypeError(f"states[{i}] and what it goes to must be tensors")
        if s.device != dev or d.device != dev or s.dtype != d.dtype:
            raise ValueError(f"states[{i}] and what it goes to must be on {dev} and of one dtype")
        key = (s.shape, s.stride(), s.dtype, d.shape, d.stride(), d is s)
        if key != last:   # most are alike
            try:
                c = _reorder_layout(s.shape, s.stride(), d.shape, d.stride(), s.element_size(), B, N, d is s)
            except ValueError as e:
                raise ValueError(f"states[{i}] {e}") from None
            # In place or not is a call's own.
            src_at, dst_at = calls.setdefault((c, d is s), ([], []))
            last = key
        if c is None:
            continue
        at, to = s.data_ptr(), d.data_ptr()
        seen.append((to, to + c.extent, i, c))
        if d is not s and at < to + c.extent and to < at + c.src_extent:
            raise ValueError(f"out[{i}] overlaps states[{i}]")
        src_at.append(at)
        dst_at.append(to)
    _apart(seen, src if out is not None else [])
    if seen:
        _ready(dev)
    for (c, _), (src_at, dst_at) in calls.items():
        n = len(src_at)
        if n == 0:
            continue
        r = A.llp_beam_reorder_request(
            (C.c_void_p * n)(*src_at), (C.c_void_p * n)(*dst_at), n, c.K, N, 0, B, c.outer, c.inner, c.sr,
            c.so, c.dr, c.do, parents.data_ptr(), _ptr(status))
        _call(dev, "llp_beam_reorder", C.byref(r))
    if seen:
        _changed(dst)
    return states if out is None else out


def _apart(seen, sources):
    """Refuses states that share bytes: a call moves them all at once."""
    seen.sort(key=lambda t: t[:2])
    for i, a in enumerate(seen):
        for b in seen[i + 1:]:
            if b[0] >= a[1]:
                break
            if not _interleaved(a, b):
                raise ValueError(f"states {a[2]} and {b[2]} overlap")
    for s in sources:
        p = s.data_ptr()
        end = p + s.element_size() * (1 + sum((n - 1) * st for n, st in zip(s.shape, s.stride())))
        for d in seen:
            if s.numel() and p < d[1] and d[0] < end:
                raise ValueError(f"out[{d[2]}] overlaps a state")


def _interleaved(a, b):
    """Whether two states, the second no lower in memory, lie between each other's rows or pieces, as the
    keys and values of a cache [rows, 2, ...] do, or parts of one buffer's rows."""
    ca, cb = a[3], b[3]
    shift = b[0] - a[0]
    if shift >= ca.extent:
        return True
    for (s, in_a), (sb, in_b) in zip(ca.levels, cb.levels):
        if s != sb:
            return False
        shift %= s
        if shift + in_b > s:
            return False
        if shift >= in_a:
            return True
    return False
