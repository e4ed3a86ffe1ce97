"""Measured calls of the operators that decode and train with a head in 8-bit floating point: the
quantisation in blocks of 128, the product of such operands with its gradients, and a beam search's
selection over beams and vocabulary with the reordering of the beams' states.

Each case is one call, or the run of calls that belongs together, as a serving or training program
makes it. With ``own`` false, ``run`` computes it in elementary torch operations; with ``own`` true
it calls the package. ``exact`` gives the same outputs from the operators' definitions in 64 bits.

Sizes are those of the repository's own workloads (hidden size 4096, vocabulary 151669 real /
151936 padded, shards of 37984, chunks of 4096 tokens), and ragged sizes between them.
"""
import math

import torch

own = False

H_FULL, V_REAL, V_PAD, V_SHARD = 4096, 151669, 151936, 37984
BLOCK, TOP = 128, 448.0        # values that share a scale along a row; the largest e4m3 value
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # The logits of the one token a rollout is about to sample: the weight's bytes, latency.
        dict(name="fp8 linear, 1 token", op="linear", T=1, K=H_FULL, V=V_PAD, bias="none", out="f32"),
        # A decode batch on one of four vocabulary shards.
        dict(name="fp8 linear, 37 tokens, shard", op="linear", T=37, K=H_FULL, V=V_SHARD, bias="f32",
             out="f32"),
        # A short prompt or a speculative batch: too many rows to stream, few to fill the chip.
        dict(name="fp8 linear, 300 tokens, shard", op="linear", T=300, K=H_FULL, V=V_SHARD,
             bias="none", out="bf16"),
        # A training chunk's logits over the whole head: the matrix product bounds it.
        dict(name="fp8 linear, 4096 tokens", op="linear", T=4096, K=H_FULL, V=V_PAD, bias="none",
             out="bf16"),
        # Forward and both gradients of one chunk on a shard, weight quantised anew as a step does.
        dict(name="fp8 linear step, shard", op="step", T=4096, K=H_FULL, V=V_SHARD, dtype="bf16"),
        # The head's own quantisation when a checkpoint is loaded: blocks of 128 x 128.
        dict(name="fp8 quantise, head shard", op="quant", R=V_SHARD, C=H_FULL, dtype="bf16", rows=128,
             transpose=False),
        # An activation quantised along its tokens for the weight gradient.
        dict(name="fp8 quantise, transposed", op="quant", R=4096, C=V_SHARD, dtype="bf16", rows=1,
             transpose=True),
        # One sequence's beams choose their next tokens: latency.
        dict(name="beam select, 4 beams", op="beam", B=1, beams=4, num=8, V=V_REAL, pad=V_PAD, shards=1,
             dtype="f32", tau=1.0, finished=False),
        # A batch on four vocabulary shards, logits in bf16, some beams already ended.
        dict(name="beam select, 16 x 5, shards", op="beam", B=16, beams=5, num=10, V=V_REAL, pad=V_PAD,
             shards=4, dtype="bf16", tau=0.7, finished=True),
        # A large decode batch: one pass over 311 MB of logits.
        dict(name="beam select, 64 x 8", op="beam", B=64, beams=8, num=16, V=V_REAL, pad=V_PAD, shards=1,
             dtype="f32", tau=1.0, finished=True),
        # One sequence's caches of a small model follow their beams, in place.
        dict(name="beam reorder, 4 beams", op="reorder", B=1, beams=4, tensors=8, heads=8, room=1024,
             length=513, dim=128),
        # A batch's caches with long prefixes.
        dict(name="beam reorder, 16 x 8", op="reorder", B=16, beams=8, tensors=8, heads=8, room=2048,
             length=1531, dim=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "step", "quant", "beam", "reorder"))
    K = rng.choice((256, 320, 1000, 1024, 2048, H_FULL))
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 4096), K=K, V=_log_int(rng, 200, V_PAD),
                    bias=rng.choice(("none", "bf16", "f32")), out=rng.choice(("bf16", "f32")))
    if op == "step":
        return dict(op=op, T=_log_int(rng, 1, 4096), K=K - K % 8, V=8 * _log_int(rng, 25, V_SHARD // 8),
                    dtype=rng.choice(("bf16", "f32")))
    if op == "quant":
        return dict(op=op, R=_log_int(rng, 1, V_SHARD), C=rng.choice((K, K - 8, K + 40, 1001)),
                    dtype=rng.choice(("bf16", "f32")), rows=rng.choice((1, BLOCK)),
                    transpose=rng.random() < 0.5)
    if op == "beam":
        beams = rng.choice((1, 2, 3, 4, 5, 8, 16))
        V = _log_int(rng, 300, V_REAL)
        return dict(op=op, B=_log_int(rng, 1, max(1, 512 // beams)), beams=beams,
                    num=beams * rng.choice((1, 2)), V=V, pad=V + rng.choice((0, 24, 267)),
                    shards=rng.choice((1, 1, 4)), dtype=rng.choice(("bf16", "f32")),
                    tau=rng.choice((0.7, 1.0, 1.3)), finished=rng.random() < 0.5)
    beams = rng.choice((2, 3, 4, 5, 8, 16))
    length = _log_int(rng, 1, 1531)
    return dict(op=op, B=_log_int(rng, 1, 128 // beams), beams=beams, tensors=2 * _log_int(rng, 1, 4),
                heads=rng.choice((1, 4, 8)), room=length + rng.choice((0, 1, 500)), length=length,
                dim=rng.choice((64, 80, 128)))


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pad(n):
    return n + -n % BLOCK


def _divided(x, s):
    """x / s (fp32), as e4m3."""
    return (x / s).clamp_(-TOP, TOP).to(FP8)


def _blocked(x, rows):
    """x [R, C] in e4m3 with a scale for each 1 or 128 rows by 128 columns: q [R, C padded to 128]
    (zeros behind C) and scale [groups of rows, C padded / 128]."""
    R, C = x.shape
    P = torch.nn.functional.pad(x.float(), (0, -C % BLOCK, 0, -R % rows))
    g = P.reshape(P.shape[0] // rows, rows, -1, BLOCK)
    s = g.abs().amax(dim=(1, 3)).clamp_min(1e-30) / TOP
    q = _divided(g, s[:, None, :, None]).reshape(P.shape)
    return q[:R], s


def _scaled(q, s, rows):
    """The values that q and its scales stand for, in fp32."""
    wide = s.repeat_interleave(BLOCK, dim=1).repeat_interleave(rows, dim=0)[:q.shape[0]]
    return q.float() * wide


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    c, s = case, dict(case=case)
    if c["op"] == "linear":
        # A hidden state's channels differ in size, and a few stand out.
        s["x"] = (normal(c["T"], c["K"]) * torch.exp(normal(c["K"], std=0.7))).to(torch.bfloat16)
        # What such a program keeps: the frozen weight as it was quantised when it was loaded.
        s["wq"], s["ws"] = _blocked(normal(c["V"], c["K"], std=0.02, dtype=torch.bfloat16), BLOCK)
        s["bias"] = None if c["bias"] == "none" else normal(c["V"], std=0.5, dtype=_dtype(c["bias"]))
    elif c["op"] == "step":
        d = _dtype(c["dtype"])
        s["x"] = (normal(c["T"], c["K"]) * torch.exp(normal(c["K"], std=0.7))).to(d)
        s["w"] = normal(c["V"], c["K"], std=0.02, dtype=d)
        # Gradients of a mean over tokens, of different sizes from token to token.
        s["dy"] = (normal(c["T"], c["V"]) * torch.exp(normal(c["T"], 1)) / c["T"]).to(d)
    elif c["op"] == "quant":
        s["x"] = normal(c["R"], c["C"], std=0.02, dtype=_dtype(c["dtype"]))
    elif c["op"] == "beam":
        B, k, V = c["B"], c["beams"], c["pad"]
        z = normal(B * k, V, std=2.0)
        # A few likely tokens in each row, as a model's logits have; padding holds anything.
        at = torch.randint(0, c["V"], (B * k, 12), generator=g, device="cuda")
        z.scatter_(1, at, 8.0 + 6.0 * torch.rand(B * k, 12, generator=g, device="cuda"))
        z = z.to(_dtype(c["dtype"]))
        n = c["shards"]
        width = -(-V // n)
        width += -width % 8
        # Each shard's rows are 16-byte aligned, as a head's product writes them.
        s["z"], s["at"] = [], []
        for r in range(n):
            part = z[:, r * width:(r + 1) * width]
            room = torch.zeros(B * k, part.shape[1] + -part.shape[1] % 8, dtype=z.dtype, device="cuda")
            s["z"].append(room[:, :part.shape[1]].copy_(part))
            s["at"].append(min(r * width, V))
        s["scores"] = -torch.rand(B, k, generator=g, device="cuda").mul_(6).sort(dim=1).values
        s["finished"] = None
        if c["finished"]:
            s["finished"] = (torch.rand(B, k, generator=g, device="cuda") < 0.15).to(torch.uint8)
        s["c"] = float(torch.tensor(1.0 / c["tau"], dtype=torch.float32))
    else:
        B, k = c["B"], c["beams"]
        s["room"] = [normal(B * k, c["heads"], c["room"], c["dim"], dtype=torch.bfloat16)
                     for _ in range(c["tensors"])]
        s["states"] = [t[:, :, :c["length"]] for t in s["room"]]
        s["parents"] = torch.randint(0, k, (B, k), generator=g, device="cuda").to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------
END = 2   # the token that an ended beam goes on with


def _own(s):
    import lm_head_linear_logp_amd as llp
    c = s["case"]
    if c["op"] == "linear":
        q, scale = llp.quantize_blocks(s["x"])
        y = llp.linear_fp8(q, scale, s["wq"], s["ws"], bias=s["bias"], out_dtype=_dtype(c["out"]))
        return dict(y=y, q=q, scale=scale)
    if c["op"] == "step":
        x, w = s["x"].detach().requires_grad_(), s["w"].detach().requires_grad_()
        y = llp.fp8_linear(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"])
        return dict(y=y, dx=dx, dw=dw)
    if c["op"] == "quant":
        return llp.quantize_blocks(s["x"], rows=c["rows"], transpose=c["transpose"])
    if c["op"] == "beam":
        parts = [llp.beam_candidates(z, c["num"], temperature=c["tau"], offset=at, real_vocab=c["V"],
                                     padded_vocab=c["pad"], rank=r, world=c["shards"])
                 for r, (z, at) in enumerate(zip(s["z"], s["at"]))]
        return llp.beam_select(parts, s["scores"], c["num"], temperature=c["tau"],
                               finished=s["finished"], end_id=END)
    llp.beam_reorder(s["states"], s["parents"])
    return s["states"]


def _plain_beam(s):
    c = s["case"]
    B, k = c["B"], c["beams"]
    z = torch.cat(s["z"], dim=1)[:, :c["V"]].double() * s["c"]
    logp = torch.log_softmax(z, dim=1).reshape(B, k, -1)
    total = s["scores"].double()[:, :, None] + logp
    if s["finished"] is not None:
        # An ended beam goes on with one token, at its own score.
        kept = torch.full_like(total, -math.inf)
        kept[:, :, END] = s["scores"].double()
        total = torch.where(s["finished"][:, :, None] != 0, kept, total)
    # Stable: among equals the lowest beam, then the lowest token, comes first.
    best, at = torch.sort(total.reshape(B, -1), dim=1, descending=True, stable=True)
    best, at = best[:, :c["num"]], at[:, :c["num"]]
    beam = torch.div(at, c["V"], rounding_mode="floor")
    return dict(token=at - beam * c["V"], parent=beam.to(torch.int32), score=best.float())


def _plain(s):
    c = s["case"]
    if c["op"] == "linear":
        q, scale = _blocked(s["x"], 1)
        y = _scaled(q, scale, 1) @ _scaled(s["wq"], s["ws"], BLOCK).T
        if s["bias"] is not None:
            y += s["bias"].float()
        return dict(y=y.to(_dtype(c["out"])), q=q, scale=scale)
    if c["op"] == "step":
        T, K, V = c["T"], c["K"], c["V"]
        x, w, dy = s["x"], s["w"], s["dy"]
        wd = _scaled(*_blocked(w, BLOCK), BLOCK)[:, :K]
        y = _scaled(*_blocked(x, 1), 1)[:, :K] @ wd.T
        dx = _scaled(*_blocked(dy, 1), 1)[:, :V] @ wd
        # Along the tokens: dy in blocks of 128 x 128, x in groups of 128.
        gt = _scaled(*_blocked(dy.T, BLOCK), BLOCK)[:, :T]
        xt = _scaled(*_blocked(x.T, 1), 1)[:, :T]
        return dict(y=y.to(x.dtype), dx=dx.to(x.dtype), dw=(gt @ xt.T).to(w.dtype))
    if c["op"] == "quant":
        return _blocked(s["x"].T if c["transpose"] else s["x"], c["rows"])
    if c["op"] == "beam":
        return _plain_beam(s)
    k = c["beams"]
    at = (s["parents"].long() + torch.arange(c["B"], device="cuda")[:, None] * k).reshape(-1)
    for t in s["states"]:
        t.copy_(t[at])
    return s["states"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "linear":
        T, K, V = c["T"], _pad(c["K"]), c["V"]
        out = 2 if c["out"] == "bf16" else 4
        return dict(bytes=V * K + T * (2 * c["K"] + K + K // 32) + T * V * out, flops=2 * T * c["K"] * V)
    if c["op"] == "step":
        T, K, V = c["T"], c["K"], c["V"]
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=size * 2 * (T * K + V * K + T * V), flops=6 * T * K * V)
    if c["op"] == "quant":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["R"] * c["C"] * (size + 1), flops=3 * c["R"] * c["C"])
    if c["op"] == "beam":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["B"] * (c["beams"] * (c["V"] * size + 5) + c["num"] * 16),
                    flops=4 * c["B"] * c["beams"] * c["V"])
    # A slot keeps its own rows, or reads another's: (k - 1) / k of them with parents drawn evenly.
    k = c["beams"]
    row = c["heads"] * c["length"] * c["dim"] * 2 * c["tensors"]
    return dict(bytes=c["B"] * ((k - 1) * row + k * (1 - (1 - 1 / k) ** k) * row), flops=0)


# ------------------------------------------------------------------------------------------
# The same outputs from the definitions, in 64 bits
# ------------------------------------------------------------------------------------------
def _tiles64(x, rows):
    """x's quantised values in 64 bits, block by block: whole e4m3 values that the fp32 quotient
    fixes, times top / 448 in 64 bits; and those scales."""
    R, C = x.shape
    x = torch.cat([x.float(), torch.zeros(-R % rows, C, device="cuda")], dim=0)
    x = torch.cat([x, torch.zeros(x.shape[0], -C % BLOCK, device="cuda")], dim=1)
    t = x.unfold(0, rows, rows).unfold(1, BLOCK, BLOCK)          # [row groups, groups, rows, 128]
    top = t.abs().flatten(2).max(dim=2).values
    top = torch.maximum(top, torch.tensor(1e-30, device="cuda"))
    code = (t / (top / 448.0)[:, :, None, None]).to(FP8).double()
    value = code * (top.double() / 448.0)[:, :, None, None]
    value = value.permute(0, 2, 1, 3).reshape(x.shape)
    return value[:R, :C], top.double() / 448.0


def _mm64(a, b):
    """a . b^T in 64 bits, in strips of b's rows."""
    strips = [torch.mm(a, b[v:v + 8192].t().contiguous()) for v in range(0, b.shape[0], 8192)]
    return torch.cat(strips, dim=1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        x, scale = _tiles64(s["x"], 1)
        strips = []
        for v in range(0, c["V"], 8192):
            e = min(c["V"], v + 8192)
            rows = torch.arange(v, e, device="cuda") // BLOCK
            w = s["wq"][v:e].double().reshape(e - v, -1, BLOCK) * s["ws"].double()[rows].unsqueeze(2)
            z = torch.mm(x, w.reshape(e - v, -1)[:, :c["K"]].t().contiguous())
            strips.append(z if s["bias"] is None else z + s["bias"][v:e].double().unsqueeze(0))
        return dict(y=torch.cat(strips, dim=1), q=None, scale=scale)
    if c["op"] == "step":
        x, w, dy = s["x"], s["w"], s["dy"]
        w64 = _tiles64(w, BLOCK)[0]
        y = _mm64(_tiles64(x, 1)[0], w64)
        dx = _mm64(_tiles64(dy, 1)[0], w64.t().contiguous())
        dw = _mm64(_tiles64(dy.t().contiguous(), BLOCK)[0], _tiles64(x.t().contiguous(), 1)[0])
        return dict(y=y, dx=dx, dw=dw)
    if c["op"] == "quant":
        x = s["x"].t().contiguous() if c["transpose"] else s["x"]
        return (None, _tiles64(x, c["rows"])[1])
    if c["op"] == "beam":
        B, k = c["B"], c["beams"]
        best = torch.empty(B, c["num"], dtype=torch.float64, device="cuda")
        z = torch.cat(s["z"], dim=1)[:, :c["V"]]
        for b in range(B):
            rows = z[b * k:(b + 1) * k].double() * s["c"]
            top = rows.max(dim=1, keepdim=True).values
            lp = rows - top - torch.log(torch.exp(rows - top).sum(dim=1, keepdim=True))
            lp = lp + s["scores"][b].double()[:, None]
            if s["finished"] is not None:
                over = s["finished"][b] != 0
                lp[over] = -math.inf
                lp[over, END] = s["scores"][b].double()[over]
            best[b] = torch.topk(lp.flatten(), c["num"]).values
        return dict(token=None, parent=None, score=best)
    return None
