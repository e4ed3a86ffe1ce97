"""Measured calls of the operators around the fused linear log-prob: 8-bit scoring with a frozen
head, the clipped policy loss, the paired preference loss, and the (tied) token embedding.

Each case is one call as a training or serving program makes it. With ``own`` false, ``run``
computes it in elementary torch operations; with ``own`` true it calls the package. ``exact``
gives the same outputs from the operators' definitions in 64 bits.

Sizes are those of the repository's own workloads (hidden size 4096, vocabulary 151669 real /
151936 padded, shards of 37984, 4096-token chunks, packs of 16 sequences of up to 7168 tokens,
and the small forward's 256 x 1024 head), and ragged sizes between them.
"""
import math
import random

import torch

own = False

H_FULL, V_REAL, V_PAD, V_SHARD = 4096, 151669, 151936, 37984
LOG_RATIO_MAX = 20.0


# ------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # A frozen head scores the one token a rollout just sampled: weight bandwidth and latency.
        dict(name="int8 score, 1 token", op="score", T=1, H=H_FULL, local=V_PAD, offset=0,
             real=V_REAL, padded=V_PAD, world=1, bias="none", mask=0.0, entropy=True, tau=1.0),
        # A decode batch on the last of four vocabulary shards, whose end is padding.
        dict(name="int8 score, 37 tokens, shard", op="score", T=37, H=H_FULL, local=V_SHARD,
             offset=3 * V_SHARD, real=V_REAL, padded=V_PAD, world=4, bias="f32", mask=0.0,
             entropy=True, tau=0.7),
        # A training chunk of reference log-probs: the matrix product bounds it.
        dict(name="int8 score, 4096 tokens", op="score", T=4096, H=H_FULL, local=V_PAD, offset=0,
             real=V_REAL, padded=V_PAD, world=1, bias="none", mask=0.1, entropy=True, tau=0.7),
        # The head's own quantisation when a reference model is frozen: one pass over the weight.
        dict(name="int8 quantise, head shard", op="quant", R=V_SHARD, H=H_FULL, dtype="bf16"),
        # One chunk's policy loss and the gradients that its backward takes: latency.
        dict(name="policy, 4096 tokens", op="policy", T=4096, seqs=4, reduction="token_mean",
             kl="k3", ref=True, entropy=True, dual=0.0, mask=0.3),
        # A whole global batch of packed responses, averaged by sequence.
        dict(name="policy, 1M tokens by sequence", op="policy", T=1048573, seqs=256,
             reduction="seq_mean", kl="k3", ref=True, entropy=True, dual=3.0, mask=0.3),
        # A small batch of chosen/rejected pairs, ragged.
        dict(name="preference, 8 pairs", op="pref", pairs=8, T=4607, kind="sigmoid",
             average=False, ref=True, smooth=0.0, mask=0.4),
        # A large one, with label smoothing, responses up to the longest of the workload.
        dict(name="preference, 512 pairs", op="pref", pairs=512, T=4128769, kind="sigmoid",
             average=False, ref=True, smooth=0.1, mask=0.3),
        # Embedding rows for one decode step of 64 sequences.
        dict(name="embedding, 64 tokens", op="embed", T=64, H=H_FULL, local=V_PAD, offset=0,
             real=V_REAL, padded=V_PAD, world=1, dtype="bf16", scale=64.0, skew=1.0),
        # Embedding rows of a whole pack, fp32 master weight's bf16 copy.
        dict(name="embedding, 56583 tokens", op="embed", T=56583, H=H_FULL, local=V_PAD, offset=0,
             real=V_REAL, padded=V_PAD, world=1, dtype="bf16", scale=64.0, skew=1.0),
        # The dense gradient of one shard's rows from one chunk.
        dict(name="embedding grad, 4096, shard", op="egrad", T=4096, H=H_FULL, local=V_SHARD,
             offset=0, real=V_REAL, padded=V_PAD, world=4, dtype="bf16", scale=1.0, skew=1.0),
        # The dense gradient of the whole table from a pack: a few ids hold most positions.
        dict(name="embedding grad, 56583 tokens", op="egrad", T=56583, H=H_FULL, local=V_PAD,
             offset=0, real=V_REAL, padded=V_PAD, world=1, dtype="bf16", scale=64.0, skew=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _shard(rng):
    """A vocabulary and one shard of it: the whole, one of four, or a small head."""
    k = rng.choice(("whole", "shard", "small"))
    if k == "whole":
        return dict(local=V_PAD, offset=0, real=V_REAL, padded=V_PAD, world=1)
    if k == "shard":
        return dict(local=V_SHARD, offset=V_SHARD * rng.randrange(4), real=V_REAL, padded=V_PAD,
                    world=4)
    real = _log_int(rng, 300, 30000)
    return dict(local=real + 24, offset=0, real=real, padded=real + 24, world=1)


def draw(rng):
    op = rng.choice(("score", "quant", "policy", "pref", "embed", "egrad"))
    H = rng.choice((256, 320, 1024, 2048, H_FULL))
    if op == "score":
        return dict(op=op, T=_log_int(rng, 1, 4096), H=H, bias=rng.choice(("none", "bf16", "f32")),
                    mask=rng.choice((0.0, 0.1, 0.5)), entropy=rng.random() < 0.7,
                    tau=rng.choice((0.7, 1.0, 1.3)), **_shard(rng))
    if op == "quant":
        return dict(op=op, R=_log_int(rng, 1, V_SHARD), H=rng.choice((H, H - 8, H + 40, 1000)),
                    dtype=rng.choice(("bf16", "f32")))
    if op == "policy":
        T = _log_int(rng, 64, 1 << 20)
        return dict(op=op, T=T, seqs=_log_int(rng, 1, max(2, T // 16)),
                    reduction=rng.choice(("token_mean", "seq_mean", "sum")),
                    kl=rng.choice(("k1", "k2", "k3")), ref=rng.random() < 0.8,
                    entropy=rng.random() < 0.6, dual=rng.choice((0.0, 3.0)),
                    mask=rng.choice((0.0, 0.3, 0.6)))
    if op == "pref":
        pairs = _log_int(rng, 1, 512)
        return dict(op=op, pairs=pairs, T=pairs * _log_int(rng, 32, 8063),
                    kind=rng.choice(("sigmoid", "hinge", "ipo")), average=rng.random() < 0.4,
                    ref=rng.random() < 0.7, smooth=rng.choice((0.0, 0.1)),
                    mask=rng.choice((0.0, 0.3)))
    return dict(op=op, T=_log_int(rng, 1, 56583), H=H, dtype=rng.choice(("bf16", "f32")),
                scale=rng.choice((1.0, 64.0)), skew=rng.choice((0.0, 1.0)), **_shard(rng))


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _quantised(w):
    """Rows of int8 and their fp32 scales (a frozen head's, made when it was loaded)."""
    pad = -w.shape[1] % 128
    amax = w.float().abs().amax(dim=1)
    scale = amax.clamp_min(1e-30) / 127.0
    q = torch.zeros((w.shape[0], w.shape[1] + pad), dtype=torch.int8, device=w.device)
    for r in range(0, w.shape[0], 16384):
        q[r:r + 16384, :w.shape[1]] = torch.round(w[r:r + 16384].float() / scale[r:r + 16384, None])
    return q, scale


def _skewed_ids(g, T, real, skew):
    """Token ids: uniform, or with the heavy head of text (a few ids in most positions)."""
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    if not skew:
        return (u * real).long().clamp_(0, real - 1)
    # log-uniform rank, then a fixed scatter of ranks over the table
    rank = torch.exp(u * math.log(real)).long() - 1
    return (rank.clamp_(0, real - 1) * 40503 + 7) % real


def _cuts(seed, T, seqs):
    """Boundaries of `seqs` packed sequences of ragged lengths over T tokens (some may be empty)."""
    r = random.Random(seed)
    inner = sorted(r.randint(0, T) for _ in range(seqs - 1))
    return [0] + inner + [T]


def _ragged(seed, T, seqs):
    """Boundaries of `seqs` packed responses over T tokens, none empty, the longest about eight
    times the shortest."""
    r = random.Random(seed)
    share = [r.uniform(1, 8) for _ in range(seqs)]
    cuts, at, whole = [0], 0.0, sum(share)
    for k, x in enumerate(share):
        at += x
        cuts.append(max(cuts[-1] + 1, min(int(T * at / whole), T - (seqs - 1 - k))))
    cuts[-1] = T
    return cuts


def _prompt_mask(cuts, share, g):
    """1 = scored: the first part of each sequence (its prompt) is not."""
    T = cuts[-1]
    cu = torch.tensor(cuts, device="cuda", dtype=torch.int64)
    lens = cu[1:] - cu[:-1]
    f = torch.rand(lens.shape[0], generator=g, device="cuda", dtype=torch.float64) * 2 * share
    first = torch.repeat_interleave(cu[:-1] + (f.clamp_max(1.0) * lens).long(), lens)
    return (torch.arange(T, device="cuda") >= first).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    c, s = case, dict(case=case)
    if c["op"] == "score":
        T, H = c["T"], c["H"]
        s["h"] = normal(T, H, dtype=torch.bfloat16)
        s["wq"], s["ws"] = _quantised(normal(c["local"], H, std=0.02, dtype=torch.bfloat16))
        s["bias"] = None if c["bias"] == "none" else normal(c["local"], std=0.5,
                                                            dtype=_dtype(c["bias"]))
        s["targets"] = torch.randint(0, c["real"], (T,), generator=g, device="cuda")
        s["mask"] = None if not c["mask"] else (
            torch.rand(T, generator=g, device="cuda") >= c["mask"]).to(torch.uint8)
    elif c["op"] == "quant":
        s["x"] = normal(c["R"], c["H"], std=0.02, dtype=_dtype(c["dtype"]))
    elif c["op"] == "policy":
        T = c["T"]
        cuts = _cuts(seed, T, c["seqs"])
        s["cu"] = torch.tensor(cuts, device="cuda", dtype=torch.int32)
        s["mask"] = _prompt_mask(cuts, c["mask"], g) if c["mask"] else None
        s["logp"] = -torch.rand(T, generator=g, device="cuda").exp() * 2 + 2
        s["old"] = s["logp"] + normal(T, std=0.15)
        s["ref"] = s["logp"] + normal(T, std=0.1) if c["ref"] else None
        s["adv"] = torch.repeat_interleave(normal(c["seqs"]), (s["cu"][1:] - s["cu"][:-1]).long())
        s["entropy"] = torch.rand(T, generator=g, device="cuda") * 3 if c["entropy"] else None
    elif c["op"] == "pref":
        T = c["T"]
        cuts = _ragged(seed, T, 2 * c["pairs"])
        s["cu"] = torch.tensor(cuts, device="cuda", dtype=torch.int32)
        s["mask"] = _prompt_mask(cuts, c["mask"], g) if c["mask"] else None
        s["logp"] = -torch.rand(T, generator=g, device="cuda").exp() * 2 + 2
        s["ref"] = s["logp"] + normal(T, std=0.1) if c["ref"] else None
        s["beta"] = 0.1 if c["ref"] or c["average"] else 0.01
    else:
        ids = _skewed_ids(g, c["T"], c["real"], c["skew"])
        s["ids"] = ids
        if c["op"] == "embed":
            s["weight"] = normal(c["local"], c["H"], std=0.02, dtype=_dtype(c["dtype"]))
        else:
            s["dout"] = normal(c["T"], c["H"], dtype=_dtype(c["dtype"]))
    return s


# ------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------
CLIP_LOW, CLIP_HIGH, KL_COEF, ENT_COEF = 0.2, 0.28, 0.05, 0.01


def _part(c):
    return dict(offset=c["offset"], real_vocab=c["real"], padded_vocab=c["padded"],
                rank=c["offset"] // c["local"] if c["world"] > 1 else 0, world=c["world"])


def _own(s):
    import lm_head_linear_logp_amd as llp
    c = s["case"]
    if c["op"] == "score":
        q, scale = llp.quantize_rows(s["h"])
        o = llp.forward_int8(q, scale, s["wq"], s["ws"], s["targets"], temperature=c["tau"],
                             bias=s["bias"], loss_mask=s["mask"], want_entropy=c["entropy"],
                             **_part(c))
        return dict(o, q=q, scale=scale)
    if c["op"] == "quant":
        return llp.quantize_rows(s["x"])
    if c["op"] == "policy":
        return llp.policy_grads(s["logp"], s["old"], s["adv"], ref_logp=s["ref"],
                                entropy=s["entropy"], loss_mask=s["mask"], cu_seqlens=s["cu"],
                                clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual"],
                                kl=c["kl"], kl_coef=KL_COEF if c["ref"] else 0.0,
                                entropy_coef=ENT_COEF if c["entropy"] else 0.0,
                                reduction=c["reduction"])
    if c["op"] == "pref":
        return llp.preference_grads(s["logp"], s["cu"], ref_logp=s["ref"], loss_mask=s["mask"],
                                    beta=s["beta"], kind=c["kind"], average=c["average"],
                                    label_smoothing=c["smooth"] if c["kind"] == "sigmoid" else 0.0)
    if c["op"] == "embed":
        return llp.embedding_forward(s["ids"], s["weight"], scale=c["scale"], **_part(c))
    return llp.embedding_backward(s["ids"], s["dout"], local_size=c["local"], scale=c["scale"],
                                  overwrite=True, **_part(c))


def _plain_quant(x):
    amax = x.float().abs().amax(dim=1)
    scale = amax.clamp_min(1e-30) / 127.0
    q = torch.round(x.float() / scale[:, None]).to(torch.int8)
    pad = -x.shape[1] % 128
    return (torch.nn.functional.pad(q, (0, pad)) if pad else q), scale


def _plain_score(s):
    c = s["case"]
    q, scale = _plain_quant(s["h"])
    n = max(0, min(c["real"] - c["offset"], c["local"]))
    z = (q.float() @ s["wq"][:n].float().T) * scale[:, None] * s["ws"][:n]
    if s["bias"] is not None:
        z += s["bias"][:n].float()
    z *= 1.0 / c["tau"]
    lse = torch.logsumexp(z, dim=1)
    at = s["targets"] - c["offset"]
    hit = (at >= 0) & (at < n)
    tz = z.gather(1, at.clamp(0, n - 1)[:, None])[:, 0]
    tz = torch.where(hit, tz, torch.zeros_like(tz))
    logp = torch.where(hit, tz - lse, torch.full_like(tz, -math.inf))
    ent = None
    if c["entropy"]:
        z -= lse[:, None]
        ent = -(torch.exp(z) * z).sum(dim=1)
    in_range = hit.to(torch.uint8)
    if s["mask"] is not None:
        off = s["mask"] == 0
        tz, lse, logp = (x.masked_fill(off, 0.0) for x in (tz, lse, logp))
        ent = None if ent is None else ent.masked_fill(off, 0.0)
        in_range = in_range.masked_fill(off, 0)
    return dict(target_logit=tz, in_range=in_range, lse=lse, entropy=ent, logp=logp, q=q,
                scale=scale)


def _policy(s, dt):
    """Policy term, KL term and their gradients by logp for every token, in type `dt`; the clip's
    borders are compared in 64 bits."""
    c = s["case"]
    m = torch.ones_like(s["logp"], dtype=torch.bool) if s["mask"] is None else s["mask"] != 0
    d64 = s["logp"].double() - s["old"].double()
    a = s["adv"].to(dt)
    up = d64 > math.log1p(CLIP_HIGH)
    dn = d64 < math.log1p(-CLIP_LOW)
    inside = d64.abs() <= LOG_RATIO_MAX
    ratio = torch.exp(d64.clamp(-LOG_RATIO_MAX, LOG_RATIO_MAX).to(dt))
    pos = a > 0
    clipped = torch.where(pos, up, dn) & (a != 0)
    used = torch.where(clipped, torch.where(pos, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW).to(dt), ratio)
    if c["dual"]:
        far = (a < 0) & (d64 > math.log(c["dual"]))
        clipped = clipped | far
        used = torch.where(far, torch.full_like(used, c["dual"]), used)
    pg = -a * used
    dpg = torch.where(clipped | ~inside, torch.zeros_like(a), -a * ratio)
    kl = dkl = torch.zeros_like(a)
    if s["ref"] is not None:
        x = s["ref"].double() - s["logp"].double()
        if c["kl"] == "k1":
            kl, dkl = -x, torch.ones_like(x)
        elif c["kl"] == "k2":
            kl, dkl = 0.5 * x * x, -x
        else:
            y = x.clamp(-LOG_RATIO_MAX, LOG_RATIO_MAX)
            kl = torch.expm1(y) - y
            dkl = torch.where(x.abs() <= LOG_RATIO_MAX, -torch.expm1(y), torch.zeros_like(y))
        kl, dkl = kl.to(dt), dkl.to(dt)
    return m, pg, dpg, kl, dkl, clipped, ratio, d64


def _policy_out(s, dt):
    c = s["case"]
    m, pg, dpg, kl, dkl, clipped, ratio, d64 = _policy(s, dt)
    if c["reduction"] == "sum":
        w = m.double()
    elif c["reduction"] == "token_mean":
        w = m.double() / m.sum().clamp_min(1)
    else:
        lens = (s["cu"][1:] - s["cu"][:-1]).long()
        seq = torch.repeat_interleave(torch.arange(c["seqs"], device="cuda"), lens,
                                      output_size=c["T"])
        n = torch.zeros(c["seqs"], dtype=torch.float64, device="cuda").index_add_(0, seq, m.double())
        w = m.double() / (n.clamp_min(1)[seq] * (n > 0).sum().clamp_min(1))
    kc = KL_COEF if s["ref"] is not None else 0.0
    ec = ENT_COEF if s["entropy"] is not None else 0.0
    ent = s["entropy"].double() if s["entropy"] is not None else torch.zeros_like(w)

    def mean(x):
        return torch.where(m, w * x.double(), torch.zeros_like(w)).sum()

    terms = [mean(pg), mean(kl), mean(ent)]
    loss = terms[0] + kc * terms[1] - ec * terms[2]
    stats = torch.stack([loss] + terms + [mean(clipped), mean(ratio), mean(-d64),
                                          m.sum().double()])
    dlogp = torch.where(m, w * (dpg + kc * dkl).double(), torch.zeros_like(w))
    dent = torch.where(m, -ec * w, torch.zeros_like(w)) if s["entropy"] is not None else None
    out = dt if dt == torch.float64 else torch.float32
    return dict(loss=loss.to(out).reshape(1), stats=stats.to(out), dlogp=dlogp.to(out),
                dentropy=None if dent is None else dent.to(out))


def _pref_out(s, out):
    c = s["case"]
    P, beta = c["pairs"], s["beta"]
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    T = s["logp"].shape[0]
    seq = torch.repeat_interleave(torch.arange(2 * P, device="cuda"), lens, output_size=T)
    m = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    x = s["logp"].double()
    if s["ref"] is not None:
        x = x - s["ref"].double()
    zero = torch.zeros(2 * P, dtype=torch.float64, device="cuda")
    tot = zero.clone().index_add_(0, seq, torch.where(m, x, torch.zeros_like(x)))
    n = zero.clone().index_add_(0, seq, m.double()).clamp_min(1)
    per = 1.0 / n if c["average"] else torch.ones_like(n)
    r = (tot * per).reshape(P, 2)
    h = r[:, 0] - r[:, 1]
    if c["kind"] == "sigmoid":
        eps = c["smooth"]
        d = beta * h
        loss = (1 - eps) * torch.logaddexp(-d, torch.zeros_like(d)) + eps * torch.logaddexp(
            d, torch.zeros_like(d))
        dh = beta * (-(1 - eps) * torch.sigmoid(-d) + eps * torch.sigmoid(d))
    elif c["kind"] == "hinge":
        loss = (1 - beta * h).clamp_min(0)
        dh = torch.where(beta * h < 1, -beta * torch.ones_like(h), torch.zeros_like(h))
    else:
        loss = (h - 0.5 / beta) ** 2
        dh = 2 * (h - 0.5 / beta)
    coef = (torch.stack([dh, -dh], dim=1).reshape(-1) * per) / P
    return dict(loss=loss.mean().to(out).reshape(1), pair_loss=loss.to(out),
                chosen=(beta * r[:, 0]).to(out), rejected=(beta * r[:, 1]).to(out),
                dlogp=torch.where(m, coef[seq], torch.zeros_like(x)).to(out))


def _rows_of(s):
    """Local rows of the ids and whether each lies among the shard's real ones."""
    c = s["case"]
    n = max(0, min(c["real"] - c["offset"], c["local"]))
    at = s["ids"] - c["offset"]
    return at, (at >= 0) & (at < n)


def _plain(s):
    c = s["case"]
    if c["op"] == "score":
        return _plain_score(s)
    if c["op"] == "quant":
        return _plain_quant(s["x"])
    if c["op"] == "policy":
        return _policy_out(s, torch.float32)
    if c["op"] == "pref":
        return _pref_out(s, torch.float32)
    at, hit = _rows_of(s)
    if c["op"] == "embed":
        rows = s["weight"][at.clamp(0, c["local"] - 1)].float() * c["scale"]
        return torch.where(hit[:, None], rows, torch.zeros_like(rows)).to(s["weight"].dtype)
    grad = torch.zeros((c["local"], c["H"]), dtype=torch.float32, device="cuda")
    rows = s["dout"].float() * c["scale"]
    if c["world"] > 1:
        rows = torch.where(hit[:, None], rows, torch.zeros_like(rows))
        at = at.clamp(0, c["local"] - 1)
    return grad.index_add_(0, at, rows)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "score":
        T, H = c["T"], c["H"] + -c["H"] % 128
        n = max(0, min(c["real"] - c["offset"], c["local"]))
        scored = T * (1 - c["mask"])
        return dict(bytes=n * (H + 4) + T * (2 * c["H"] + H + 4) + T * (8 + 17),
                    flops=2 * scored * n * c["H"])
    if c["op"] == "quant":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["R"] * (c["H"] * size + c["H"] + -c["H"] % 128 + 4),
                    flops=3 * c["R"] * c["H"])
    if c["op"] == "policy":
        per = 4 * (3 + c["ref"] + c["entropy"]) + (c["mask"] > 0) + 4 * (1 + c["entropy"])
        return dict(bytes=c["T"] * per, flops=40 * c["T"])
    if c["op"] == "pref":
        T = c["T"]
        return dict(bytes=T * (4 * (1 + c["ref"]) + (c["mask"] > 0) + 4), flops=4 * T)
    size = 2 if c["dtype"] == "bf16" else 4
    share = c["local"] / c["padded"]
    if c["op"] == "embed":
        return dict(bytes=c["T"] * (8 + c["H"] * size * (1 + share)), flops=c["T"] * c["H"] * share)
    return dict(bytes=c["T"] * (8 + c["H"] * size * share) + c["local"] * c["H"] * 4,
                flops=c["T"] * c["H"] * share)


# ------------------------------------------------------------------------------------------
# The same outputs from the definitions, in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_score(c, s):
    # Quantised values are whole numbers fixed by the fp32 division; everything after is in 64.
    x = s["h"].float()
    scale32 = torch.maximum(x.abs().max(dim=1).values, torch.tensor(1e-30, device="cuda")) / 127.0
    q = torch.round(x / scale32.unsqueeze(1)).double()
    scale = torch.maximum(s["h"].double().abs().max(dim=1).values,
                          torch.tensor(1e-30, device="cuda", dtype=torch.float64)) / 127.0
    n = max(0, min(c["real"] - c["offset"], c["local"]))
    T, width = c["T"], c["H"]
    at = s["targets"] - c["offset"]
    hit = (at >= 0) & (at < n)
    tz = torch.zeros(T, dtype=torch.float64, device="cuda")
    m = torch.full((T,), -math.inf, dtype=torch.float64, device="cuda")
    total, first = torch.zeros_like(m), torch.zeros_like(m)
    for v in range(0, n, 8192):
        e = min(n, v + 8192)
        z = torch.mm(q, s["wq"][v:e, :width].double().t().contiguous())
        z = z * scale32.double().unsqueeze(1) * s["ws"][v:e].double().unsqueeze(0)
        if s["bias"] is not None:
            z = z + s["bias"][v:e].double().unsqueeze(0)
        z = z / c["tau"]
        here = hit & (at >= v) & (at < e)
        tz = torch.where(here, z[torch.arange(T, device="cuda"), (at - v).clamp(0, e - v - 1)], tz)
        new = torch.maximum(m, z.max(dim=1).values)
        keep = torch.exp(m - new)
        p = torch.exp(z - new.unsqueeze(1))
        total = total * keep + p.sum(dim=1)
        first = first * keep + (p * z).sum(dim=1)
        m = new
    lse = m + torch.log(total)
    on = torch.ones(T, dtype=torch.float64, device="cuda")
    if s["mask"] is not None:
        on = (s["mask"] > 0).double()
    logp = torch.where(hit, tz - lse, torch.full_like(tz, -math.inf))
    logp = torch.where(on > 0, logp, torch.zeros_like(logp))
    return dict(target_logit=tz * on, in_range=None, lse=lse * on,
                entropy=(lse - first / total) * on if c["entropy"] else None, logp=logp, q=None,
                scale=scale)


def _exact_policy(c, s):
    import numpy as np

    def f64(x):
        return None if x is None else x.double().cpu().numpy()

    logp, old, adv, ref, ent = (f64(s[k]) for k in ("logp", "old", "adv", "ref", "entropy"))
    on = np.ones(c["T"]) if s["mask"] is None else (s["mask"].cpu().numpy() != 0).astype(np.float64)
    cu = s["cu"].cpu().numpy().astype(np.int64)
    if c["reduction"] == "sum":
        w = on
    elif c["reduction"] == "token_mean":
        w = on / max(on.sum(), 1.0)
    else:
        upto = np.concatenate([[0.0], np.cumsum(on)])
        n = upto[cu[1:]] - upto[cu[:-1]]
        per = np.where(n > 0, 1.0 / np.maximum(n, 1.0), 0.0) / max((n > 0).sum(), 1)
        w = on * np.repeat(per, np.diff(cu))
    kc = KL_COEF if ref is not None else 0.0
    ec = ENT_COEF if ent is not None else 0.0
    d = logp - old
    ratio = np.exp(np.clip(d, -LOG_RATIO_MAX, LOG_RATIO_MAX))
    lo, hi = 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH
    # -min(A r, A clip(r)), then for A < 0 at most -c A
    first = adv * ratio
    second = adv * np.clip(ratio, lo, hi)
    bound = (second < first)
    pg = -np.minimum(first, second)
    if c["dual"]:
        worst = -c["dual"] * adv
        bound = bound | ((adv < 0) & (pg > worst))
        pg = np.where(adv < 0, np.minimum(pg, worst), pg)
    dpg = np.where(bound | (np.abs(d) > LOG_RATIO_MAX), 0.0, -first)
    kl = dkl = np.zeros_like(d)
    if ref is not None:
        x = ref - logp
        if c["kl"] == "k1":
            kl, dkl = -x, np.ones_like(x)
        elif c["kl"] == "k2":
            kl, dkl = x * x / 2, -x
        else:
            y = np.clip(x, -LOG_RATIO_MAX, LOG_RATIO_MAX)
            kl, dkl = np.expm1(y) - y, np.where(y == x, -np.expm1(y), 0.0)
    e = np.zeros_like(d) if ent is None else ent
    terms = [np.sum(w * pg), np.sum(w * kl), np.sum(w * e)]
    loss = terms[0] + kc * terms[1] - ec * terms[2]
    stats = [loss] + terms + [np.sum(w * bound), np.sum(w * ratio), np.sum(-w * d), on.sum()]
    return dict(loss=np.array([loss]), stats=np.array(stats), dlogp=w * (dpg + kc * dkl),
                dentropy=None if ent is None else -ec * w)


def _exact_pref(c, s):
    import numpy as np
    x = s["logp"].double().cpu().numpy()
    if s["ref"] is not None:
        x = x - s["ref"].double().cpu().numpy()
    on = np.ones(x.shape[0]) if s["mask"] is None else (s["mask"].cpu().numpy() != 0).astype(np.float64)
    cu = s["cu"].cpu().numpy().astype(np.int64)
    x = x * on
    tot = np.add.reduceat(x, cu[:-1])
    n = np.maximum(np.add.reduceat(on, cu[:-1]), 1.0)
    if c["average"]:
        tot = tot / n
    beta, h = s["beta"], tot[0::2] - tot[1::2]
    d = beta * h
    if c["kind"] == "sigmoid":
        e = c["smooth"]
        loss = (1 - e) * np.logaddexp(0, -d) + e * np.logaddexp(0, d)
        dh = beta * (e - 1 / (1 + np.exp(d)))
    elif c["kind"] == "hinge":
        loss, dh = np.maximum(0, 1 - d), np.where(d < 1, -beta, 0.0)
    else:
        loss, dh = (h - 1 / (2 * beta)) ** 2, 2 * h - 1 / beta
    coef = np.repeat(dh / c["pairs"], 2) * np.tile([1.0, -1.0], c["pairs"])
    if c["average"]:
        coef = coef / n
    return dict(loss=np.array([loss.sum() / c["pairs"]]), pair_loss=loss, chosen=beta * tot[0::2],
                rejected=beta * tot[1::2], dlogp=np.repeat(coef, np.diff(cu)) * on)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "score":
        return _exact_score(c, s)
    if c["op"] == "quant":
        top = s["x"].double().abs().max(dim=1).values
        return (None, torch.maximum(top, torch.full_like(top, 1e-30)) / 127.0)
    if c["op"] == "policy":
        return _exact_policy(c, s)
    if c["op"] == "pref":
        return _exact_pref(c, s)
    n = max(0, min(c["real"] - c["offset"], c["local"]))
    at = s["ids"] - c["offset"]
    mine = torch.nonzero((at >= 0) & (at < n)).flatten()
    if c["op"] == "embed":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        out[mine] = s["weight"][at[mine]].double() * c["scale"]
        return out
    out = torch.zeros((c["local"], c["H"]), dtype=torch.float64, device="cuda")
    out.index_add_(0, at[mine], s["dout"][mine].double() * c["scale"])
    return out
