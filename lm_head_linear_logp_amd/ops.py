"""Operators around the fused linear log-prob (include/llp.h): 8-bit scoring, the policy and
preference losses, the token embedding. Argument marshalling, as in the package itself: every
tensor is checked here, every step runs in libllp.so on the tensors' own device and that device's
current stream."""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _capi as A
from . import (_check, _need, _partials_alloc, _partials_out, _ptr, _status, _vec, _vocab, open)

_F32, _BF16, _U8, _I8, _I32, _I64 = (torch.float32, torch.bfloat16, torch.uint8, torch.int8,
                                     torch.int32, torch.int64)
_DTYPE = {torch.bfloat16: A.LLP_DTYPE_BF16, torch.float32: A.LLP_DTYPE_F32}
_KL = {"k1": A.LLP_KL_K1, "k2": A.LLP_KL_K2, "k3": A.LLP_KL_K3}
_REDUCE = {"token_mean": A.LLP_REDUCE_TOKEN_MEAN, "seq_mean": A.LLP_REDUCE_SEQ_MEAN,
           "sum": A.LLP_REDUCE_SUM}
_PREF = {"sigmoid": A.LLP_PREF_SIGMOID, "hinge": A.LLP_PREF_HINGE, "ipo": A.LLP_PREF_IPO}
_PREF_REDUCE = {"mean": A.LLP_REDUCE_TOKEN_MEAN, "sum": A.LLP_REDUCE_SUM}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _at(t, name, dtype, n, dev):
    """Pointer of a contiguous 1-d tensor of n elements (_vec, which words the refusal, is the
    slower test: these calls are short enough for it to show)."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.shape == (n,) and t.device == dev
            and t.is_contiguous()):
        _vec(t, name, dtype, n, dev)
    return t.data_ptr()


def _opt(t, name, dtype, n, dev):
    """The same of an optional tensor."""
    return None if t is None else _at(t, name, dtype, n, dev)


_ready_devices = set()


def _ready(dev):
    """The tensors' device, opened (the last check before the library is called)."""
    if dev in _ready_devices:
        return
    if dev.type != "cuda":
        raise RuntimeError(f"tensors are on {dev}: the kernels run on a gfx950 GPU only")
    open(dev.index)
    _ready_devices.add(dev)


_fns = {}
# The current stream's handle without the Stream object around it (1.8 us of a 10 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(A.load(), name)
    return f


def _call(dev, name, *args):
    """One execution call of the library on `dev`'s current stream, with `dev` current."""
    stream = (_raw_stream(dev.index) if _raw_stream is not None
              else torch.cuda.current_stream(dev).cuda_stream)
    if torch.cuda.current_device() == dev.index:
        st = _fn(name)(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = _fn(name)(*args, stream)
    if st != A.LLP_OK:
        _check(st, name)


def _space(name, req, dev, workspace):
    """Pointer and size of the call's workspace: the caller's when it is large enough, else a new
    one (which the caching allocator hands on in stream order), or none where none is needed."""
    n = C.c_size_t(0)
    st = _fn(name)(C.byref(req), C.byref(n))
    if st != A.LLP_OK:
        _check(st, name)
    if n.value == 0:
        return None, 0, None
    if workspace is None or workspace.numel() < n.value:
        workspace = torch.empty(n.value, dtype=_U8, device=dev)
    return workspace.data_ptr(), workspace.numel(), workspace


def _check_space(workspace, dev):
    if workspace is not None:
        _need(workspace, "workspace", _U8, 1, dev)


def _stride(t, rows, width):
    """Row stride of a matrix (its own width when there is no second row to step to)."""
    return t.stride(0) if rows > 1 else width


# ---- 8-bit scoring ---------------------------------------------------------------------------
def quantize_rows(x: torch.Tensor, *, out: Optional[tuple] = None) -> tuple:
    """llp_quantize_rows: symmetric 8-bit quantisation of the rows of a bf16 or fp32 matrix
    [R, K]. Returns (q, scale): int8 [R, K rounded up to 128] (the columns past K are 0) and
    fp32 [R], with x[r] ~ q[r] * scale[r]. `out`: the two tensors to write."""
    _tensor(x, "x")
    if x.dtype not in _DTYPE:
        raise TypeError(f"x must be a bf16 or fp32 tensor, got {x.dtype}")
    dev = x.device
    _need(x, "x", x.dtype, 2, dev)
    R, K = x.shape
    if K < 1:
        raise ValueError("x needs at least one column")
    Kp = -(-K // A.LLP_INT8_COLUMNS) * A.LLP_INT8_COLUMNS
    if out is not None:
        q, scale = out
        _need(q, "out[0]", _I8, 2, dev, (R, Kp))
        _vec(scale, "out[1]", _F32, R, dev)
    _ready(dev)
    if out is None:
        q = torch.empty((R, Kp), dtype=_I8, device=dev)
        scale = torch.empty(R, dtype=_F32, device=dev)
    req = A.llp_quant_request(x.data_ptr(), _DTYPE[x.dtype], 0, _stride(x, R, K), R, K,
                              q.data_ptr(), _stride(q, R, Kp), scale.data_ptr())
    _call(dev, "llp_quantize_rows", C.byref(req))
    return q, scale


def forward_int8(hidden: torch.Tensor, hidden_scale: torch.Tensor, weight: torch.Tensor,
                 weight_scale: torch.Tensor, target_ids: torch.Tensor, *, temperature: float,
                 bias: Optional[torch.Tensor] = None, loss_mask: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, offset: int = 0,
                 real_vocab: Optional[int] = None, padded_vocab: Optional[int] = None,
                 rank: int = 0, world: int = 1, want_entropy: bool = True,
                 status: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """llp_forward_int8: ``forward`` with hidden states and weight in 8-bit integers, as
    ``quantize_rows`` gives them (hidden [T, K] int8 with a scale per token, weight
    [local_size, K] int8 with a scale per vocabulary column, K a multiple of 128). Returns the
    partials of ``forward``; those of several shards go to ``merge``."""
    dev = _tensor(hidden, "hidden").device
    _need(hidden, "hidden", _I8, 2, dev)
    T, K = hidden.shape
    _need(weight, "weight", _I8, 2, dev, (None, K))
    V = weight.shape[0]
    r = A.llp_int8_request()
    r.hidden, r.hidden_stride = hidden.data_ptr(), _stride(hidden, T, K)
    r.hidden_scale = _at(hidden_scale, "hidden_scale", _F32, T, dev)
    r.weight, r.weight_stride = weight.data_ptr(), _stride(weight, V, K)
    r.weight_scale = _at(weight_scale, "weight_scale", _F32, V, dev)
    r.target_ids = _at(target_ids, "target_ids", _I64, T, dev)
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype not in _DTYPE:
            raise TypeError("bias must be a bf16 or fp32 tensor")
        r.bias, r.bias_dtype = _at(bias, "bias", bias.dtype, V, dev), _DTYPE[bias.dtype]
    r.flags = A.LLP_FLAG_WANT_ENTROPY if want_entropy else 0
    r.hidden_size = K
    _vocab(r.vocab, offset, V, real_vocab, padded_vocab, rank, world)
    r.layout = _layout(T, loss_mask, cu_seqlens, dev)
    r.temperature = float(temperature)
    _status(status, dev)
    r.status_word = _ptr(status)
    if out is not None:
        _partials_out(out, T, dev, want_entropy)
    _check_space(workspace, dev)
    _ready(dev)
    if out is None:
        out = _partials_alloc(T, dev, want_entropy)
    o = A.llp_partials(_ptr(out["target_logit"]), _ptr(out["in_range"]), _ptr(out["lse"]),
                       _ptr(out.get("entropy")), _ptr(out.get("logp")))
    ws, size, _keep = _space("llp_int8_workspace_bytes", r, dev, workspace)
    _call(dev, "llp_forward_int8", C.byref(r), C.byref(o), ws, size)
    return out


def _layout(T, loss_mask, cu_seqlens, dev):
    mask = _opt(loss_mask, "loss_mask", _U8, T, dev)
    if cu_seqlens is None:
        return A.llp_token_layout(T, 0, 0, None, mask)
    if not (type(cu_seqlens) is torch.Tensor and cu_seqlens.dtype is _I32 and cu_seqlens.dim() == 1
            and cu_seqlens.device == dev and cu_seqlens.is_contiguous()):
        _need(cu_seqlens, "cu_seqlens", _I32, 1, dev)
    n = cu_seqlens.shape[0]
    if n < 1:
        raise ValueError("cu_seqlens needs at least one entry")
    return A.llp_token_layout(T, n - 1, 0, cu_seqlens.data_ptr(), mask)


def _len(t, name, dtype):
    """Device and length of the 1-d tensor that sets a call's row count."""
    dev = _tensor(t, name).device
    if not (t.dtype is dtype and t.dim() == 1 and t.is_contiguous()):
        _need(t, name, dtype, 1, dev)
    return dev, t.shape[0]


# ---- Losses ----------------------------------------------------------------------------------
def policy_grads(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                 ref_logp: Optional[torch.Tensor] = None,
                 entropy: Optional[torch.Tensor] = None,
                 loss_mask: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                 clip_high: float = 0.2, dual_clip: float = 0.0, kl: str = "k3",
                 kl_coef: float = 0.0, entropy_coef: float = 0.0, reduction: str = "token_mean",
                 denominator: Optional[torch.Tensor] = None,
                 dloss: Optional[torch.Tensor] = None, want_grad: bool = True,
                 status: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """llp_policy_loss: the clipped policy loss with a KL term and an entropy bonus over T scored
    rows, and its gradients for ``backward``. All arrays fp32 [T]; loss_mask uint8 [T]; reduction
    "token_mean", "seq_mean" (needs cu_seqlens) or "sum"; kl "k1", "k2" or "k3". denominator:
    fp32 [1], the number of rows (token_mean) or sequences (seq_mean) of a batch spread over
    several processes. dloss: fp32 [1], the loss's upstream gradient (1 when None).
    Returns loss [1], stats [8] (loss, policy, kl, entropy, clipped, ratio, old_logp - logp as
    means, then the number of scored rows), dlogp [T] and dentropy [T] (None without `entropy`;
    both None unless want_grad)."""
    dev, T = _len(logp, "logp", _F32)
    if ref_logp is None and kl_coef:
        raise ValueError("kl_coef needs ref_logp")
    if entropy is None and entropy_coef:
        raise ValueError("entropy_coef needs entropy")
    if reduction == "seq_mean" and cu_seqlens is None:
        raise ValueError("reduction 'seq_mean' needs cu_seqlens")
    _status(status, dev)
    r = A.llp_policy_request(
        logp.data_ptr(), _at(old_logp, "old_logp", _F32, T, dev),
        _at(advantages, "advantages", _F32, T, dev), _opt(ref_logp, "ref_logp", _F32, T, dev),
        _opt(entropy, "entropy", _F32, T, dev), _layout(T, loss_mask, cu_seqlens, dev), clip_low,
        clip_high, dual_clip, kl_coef, entropy_coef, _choice(_KL, kl, "kl"),
        _choice(_REDUCE, reduction, "reduction"),
        _opt(denominator, "denominator", _F32, 1, dev), _ptr(status))
    dl = _opt(dloss, "dloss", _F32, 1, dev)
    has_ent = entropy is not None and want_grad
    if out is not None:
        _vec(out["loss"], "out['loss']", _F32, 1, dev)
        _vec(out["stats"], "out['stats']", _F32, A.LLP_POLICY_STATS, dev)
        if want_grad:
            _vec(out["dlogp"], "out['dlogp']", _F32, T, dev)
        if has_ent:
            _vec(out["dentropy"], "out['dentropy']", _F32, T, dev)
    _check_space(workspace, dev)
    _ready(dev)
    if out is None:
        new = logp.new_empty
        out = dict(loss=new(1), stats=new(A.LLP_POLICY_STATS), dlogp=new(T) if want_grad else None,
                   dentropy=new(T) if has_ent else None)
    o = A.llp_policy_out(out["loss"].data_ptr(), out["stats"].data_ptr(), dl,
                         out["dlogp"].data_ptr() if want_grad else None,
                         out["dentropy"].data_ptr() if has_ent else None)
    ws, size, _keep = _space("llp_policy_workspace_bytes", r, dev, workspace)
    _call(dev, "llp_policy_loss", C.byref(r), C.byref(o), ws, size)
    return out


def preference_grads(logp: torch.Tensor, cu_seqlens: torch.Tensor, *,
                     ref_logp: Optional[torch.Tensor] = None,
                     loss_mask: Optional[torch.Tensor] = None,
                     pair_weight: Optional[torch.Tensor] = None, beta: float = 0.1,
                     kind: str = "sigmoid", label_smoothing: float = 0.0, gamma: float = 0.0,
                     average: bool = False, reduction: str = "mean",
                     dloss: Optional[torch.Tensor] = None, want_grad: bool = True,
                     status: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     out: Optional[dict] = None) -> dict:
    """llp_preference_loss: the loss of P pairs of packed responses (cu_seqlens int32 [2P + 1];
    sequence 2i is pair i's chosen response, 2i + 1 the rejected one) and its gradient for
    ``backward``. kind "sigmoid", "hinge" or "ipo"; reduction "mean" (over pairs) or "sum";
    average: mean log ratio per response instead of the sum. Returns loss [1], pair_loss [P],
    chosen [P] and rejected [P] (beta times the responses' log ratios) and dlogp [T] (None
    unless want_grad). pair_weight weighs the pairs in the loss; a pair of weight 0 still gets its
    own pair_loss, chosen and rejected."""
    dev, T = _len(logp, "logp", _F32)
    layout = _layout(T, loss_mask, _tensor(cu_seqlens, "cu_seqlens"), dev)
    if layout.num_seqs % 2:
        raise ValueError(f"cu_seqlens has {layout.num_seqs + 1} entries; 2 * pairs + 1 expected")
    P = layout.num_seqs // 2
    if P == 0 and T > 0:
        raise ValueError("cu_seqlens holds no pair")
    _status(status, dev)
    r = A.llp_pref_request(
        logp.data_ptr(), _opt(ref_logp, "ref_logp", _F32, T, dev),
        _opt(pair_weight, "pair_weight", _F32, P, dev), layout, beta, gamma, label_smoothing,
        _choice(_PREF, kind, "kind"), 1 if average else 0,
        _choice(_PREF_REDUCE, reduction, "reduction"), 0, _ptr(status))
    dl = _opt(dloss, "dloss", _F32, 1, dev)
    if out is not None:
        _vec(out["loss"], "out['loss']", _F32, 1, dev)
        for k in ("pair_loss", "chosen", "rejected"):
            _vec(out[k], f"out['{k}']", _F32, P, dev)
        if want_grad:
            _vec(out["dlogp"], "out['dlogp']", _F32, T, dev)
    _check_space(workspace, dev)
    _ready(dev)
    if out is None:
        new = logp.new_empty
        out = dict(loss=new(1), pair_loss=new(P), chosen=new(P), rejected=new(P),
                   dlogp=new(T) if want_grad else None)
    o = A.llp_pref_out(out["loss"].data_ptr(), _ptr(out["pair_loss"]), _ptr(out["chosen"]),
                       _ptr(out["rejected"]), dl, out["dlogp"].data_ptr() if want_grad else None)
    ws, size, _keep = _space("llp_preference_workspace_bytes", r, dev, workspace)
    _call(dev, "llp_preference_loss", C.byref(r), C.byref(o), ws, size)
    return out


def _mask_u8(mask):
    return mask.to(_U8) if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool else mask


def _upstream(g):
    """A scalar's upstream gradient as the contiguous fp32 [1] the library reads."""
    return g.reshape(1).to(_F32).contiguous()


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, ref_logp, loss_mask, cu_seqlens,
                denominator, kw):
        o = policy_grads(logp, old_logp, advantages, ref_logp=ref_logp, entropy=entropy,
                         loss_mask=loss_mask, cu_seqlens=cu_seqlens, denominator=denominator,
                         want_grad=False, **kw)
        ctx.save_for_backward(logp, entropy, old_logp, advantages, ref_logp, loss_mask,
                              cu_seqlens, denominator)
        ctx.kw = dict(kw, status=None)
        ctx.mark_non_differentiable(o["stats"])
        return o["loss"].reshape(()), o["stats"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _dstats):
        logp, entropy, old_logp, advantages, ref_logp, mask, cu, denominator = ctx.saved_tensors
        g = policy_grads(logp, old_logp, advantages, ref_logp=ref_logp, entropy=entropy,
                         loss_mask=mask, cu_seqlens=cu, denominator=denominator,
                         dloss=_upstream(dloss), **ctx.kw)
        return (g["dlogp"] if ctx.needs_input_grad[0] else None,
                g["dentropy"] if ctx.needs_input_grad[1] else None,
                None, None, None, None, None, None, None)


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                ref_logp: Optional[torch.Tensor] = None, entropy: Optional[torch.Tensor] = None,
                loss_mask: Optional[torch.Tensor] = None,
                cu_seqlens: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                clip_high: float = 0.2, dual_clip: float = 0.0, kl: str = "k3",
                kl_coef: float = 0.0, entropy_coef: float = 0.0, reduction: str = "token_mean",
                denominator: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """The clipped policy loss as an autograd node on ``linear_logp``'s logp and entropy (the
    arguments of ``policy_grads``; old_logp, advantages and ref_logp are constants). Returns
    (loss, stats): a scalar with gradients to logp and entropy, and the statistics, without."""
    kw = dict(clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl=kl, kl_coef=kl_coef,
              entropy_coef=entropy_coef, reduction=reduction, status=status)
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, ref_logp, _mask_u8(loss_mask),
                             cu_seqlens, denominator, kw)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, cu_seqlens, ref_logp, loss_mask, pair_weight, kw):
        o = preference_grads(logp, cu_seqlens, ref_logp=ref_logp, loss_mask=loss_mask,
                             pair_weight=pair_weight, want_grad=False, **kw)
        ctx.save_for_backward(logp, cu_seqlens, ref_logp, loss_mask, pair_weight)
        ctx.kw = dict(kw, status=None)
        ctx.mark_non_differentiable(o["chosen"], o["rejected"])
        return o["loss"].reshape(()), o["chosen"], o["rejected"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _dc, _dr):
        logp, cu_seqlens, ref_logp, loss_mask, pair_weight = ctx.saved_tensors
        g = preference_grads(logp, cu_seqlens, ref_logp=ref_logp, loss_mask=loss_mask,
                             pair_weight=pair_weight, dloss=_upstream(dloss), **ctx.kw)
        return g["dlogp"], None, None, None, None, None


def preference_loss(logp: torch.Tensor, cu_seqlens: torch.Tensor, *,
                    ref_logp: Optional[torch.Tensor] = None,
                    loss_mask: Optional[torch.Tensor] = None,
                    pair_weight: Optional[torch.Tensor] = None, beta: float = 0.1,
                    kind: str = "sigmoid", label_smoothing: float = 0.0, gamma: float = 0.0,
                    average: bool = False, reduction: str = "mean",
                    status: Optional[torch.Tensor] = None):
    """The preference loss as an autograd node on ``linear_logp``'s logp (the arguments of
    ``preference_grads``; ref_logp and pair_weight are constants). Returns (loss, chosen,
    rejected); the rewards carry no gradient."""
    kw = dict(beta=beta, kind=kind, label_smoothing=label_smoothing, gamma=gamma,
              average=average, reduction=reduction, status=status)
    return _PreferenceLoss.apply(logp, cu_seqlens, ref_logp, _mask_u8(loss_mask), pair_weight, kw)


# ---- Token embedding -------------------------------------------------------------------------
def _embedding_request(token_ids, token_mask, T, H, local_size, scale, offset, real_vocab,
                       padded_vocab, rank, world, status, dev):
    r = A.llp_embedding_request()
    r.token_ids = token_ids.data_ptr()
    r.token_mask = _opt(token_mask, "token_mask", _U8, T, dev)
    r.num_tokens = T
    _vocab(r.vocab, offset, local_size, real_vocab, padded_vocab, rank, world)
    r.hidden_size = H
    r.scale = scale
    _status(status, dev)
    r.status_word = _ptr(status)
    return r


def embedding_forward(token_ids: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0,
                      token_mask: Optional[torch.Tensor] = None, offset: int = 0,
                      real_vocab: Optional[int] = None, padded_vocab: Optional[int] = None,
                      rank: int = 0, world: int = 1, status: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """llp_embedding on one shard: scale * weight[token_ids - offset] in weight's dtype (bf16 or
    fp32), rows of zeros for masked tokens and for those of other shards."""
    dev = _tensor(weight, "weight").device
    if weight.dtype not in _DTYPE:
        raise TypeError(f"weight must be a bf16 or fp32 tensor, got {weight.dtype}")
    _need(weight, "weight", weight.dtype, 2, dev)
    V, H = weight.shape
    _need(token_ids, "token_ids", _I64, 1, dev)
    T = token_ids.shape[0]
    r = _embedding_request(token_ids, token_mask, T, H, V, scale, offset, real_vocab, padded_vocab,
                           rank, world, status, dev)
    if out is not None:
        _need(out, "out", weight.dtype, 2, dev, (T, H))
    _ready(dev)
    if out is None:
        out = torch.empty((T, H), dtype=weight.dtype, device=dev)
    _call(dev, "llp_embedding", C.byref(r), _ptr(weight), _DTYPE[weight.dtype],
          _stride(weight, V, H), _ptr(out), _stride(out, T, H))
    return out


def embedding_backward(token_ids: torch.Tensor, dout: torch.Tensor, *,
                       dweight: Optional[torch.Tensor] = None, local_size: Optional[int] = None,
                       scale: float = 1.0, token_mask: Optional[torch.Tensor] = None,
                       offset: int = 0, real_vocab: Optional[int] = None,
                       padded_vocab: Optional[int] = None, rank: int = 0, world: int = 1,
                       overwrite: bool = False, status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """llp_embedding_backward on one shard: dweight (fp32 [local_size, H]) += the gradient of
    ``embedding_forward`` for the upstream dout (bf16 or fp32 [T, H]), the rows of each token
    summed in fp32. With a tied head this is ``backward``'s own dweight. overwrite=True writes
    every row instead (0 where no token is). A missing dweight is allocated (local_size rows)."""
    dev = _tensor(dout, "dout").device
    if dout.dtype not in _DTYPE:
        raise TypeError(f"dout must be a bf16 or fp32 tensor, got {dout.dtype}")
    _need(dout, "dout", dout.dtype, 2, dev)
    T, H = dout.shape
    _at(token_ids, "token_ids", _I64, T, dev)
    if dweight is not None:
        _need(dweight, "dweight", _F32, 2, dev, (local_size, H))
        local_size = dweight.shape[0]
    elif local_size is None:
        raise ValueError("local_size is needed where dweight is not given")
    elif int(local_size) < 0:
        raise ValueError(f"local_size {local_size} < 0")
    V = int(local_size)
    r = _embedding_request(token_ids, token_mask, T, H, V, scale, offset, real_vocab, padded_vocab,
                           rank, world, status, dev)
    r.flags = A.LLP_FLAG_OVERWRITE_GRADS if overwrite else 0
    _check_space(workspace, dev)
    _ready(dev)
    if dweight is None:
        dweight = (torch.empty if overwrite else torch.zeros)((V, H), dtype=_F32, device=dev)
    ws, size, _keep = _space("llp_embedding_workspace_bytes", r, dev, workspace)
    _call(dev, "llp_embedding_backward", C.byref(r), _ptr(dout), _DTYPE[dout.dtype],
          _stride(dout, T, H), _ptr(dweight), _stride(dweight, V, H), ws, size)
    return dweight


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, token_ids, weight, token_mask, scale, real_vocab, status):
        out = embedding_forward(token_ids, weight, scale=scale, token_mask=token_mask,
                                real_vocab=real_vocab, status=status)
        ctx.save_for_backward(token_ids, token_mask)
        ctx.cfg = (scale, real_vocab, weight.shape[0], weight.dtype)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        token_ids, token_mask = ctx.saved_tensors
        scale, real_vocab, V, dtype = ctx.cfg
        if not ctx.needs_input_grad[1]:
            return None, None, None, None, None, None
        # An expanded or transposed upstream gradient, or a view that starts between 16 bytes.
        if not dout.is_contiguous() or dout.data_ptr() % 16:
            dout = dout.clone(memory_format=torch.contiguous_format)
        g = embedding_backward(token_ids, dout, local_size=V, scale=scale, token_mask=token_mask,
                               real_vocab=real_vocab, overwrite=True)
        return None, g.to(dtype), None, None, None, None


def embedding(token_ids: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0,
              token_mask: Optional[torch.Tensor] = None, real_vocab: Optional[int] = None,
              status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * weight[token_ids] as an autograd node (one full-vocabulary shard): token_ids of
    any shape, the result has it with the hidden size behind. The weight gradient is summed in
    fp32 and handed to autograd in weight's dtype; where the weight is also the head's
    (``linear_logp``), autograd adds the two."""
    shape = _tensor(token_ids, "token_ids").shape
    mask = _mask_u8(token_mask)
    out = _Embedding.apply(token_ids.reshape(-1), weight,
                           None if mask is None else mask.reshape(-1), scale, real_vocab, status)
    return out.reshape(*shape, weight.shape[1])
