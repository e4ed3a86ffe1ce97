"""fp64 CPU oracle of the operators around the linear log-prob: 8-bit scoring, the policy and
preference losses, the token embedding (plain NumPy, from the formulas in include/llp.h)."""
from __future__ import annotations

import numpy as np

LOG_RATIO_MAX = 20.0


def quantize(x):
    """int8 rows (columns padded to a multiple of 128) and fp32 scales of fp32 rows `x`. The
    definition fixes an fp32 product and an fp32 division, so these are carried out in fp32."""
    x = np.asarray(x, dtype=np.float32)
    R, K = x.shape
    q = np.zeros((R, -(-K // 128) * 128), dtype=np.int8)
    scale = np.empty(R, dtype=np.float32)
    for r in range(R):
        if not np.isfinite(x[r]).all():
            scale[r] = np.nan
            continue
        scale[r] = np.maximum(np.abs(x[r]).max(), np.float32(1e-30)) * (np.float32(1) / np.float32(127))
        q[r, :K] = np.rint(x[r] / scale[r]).astype(np.int8)
    return q, scale


def int8_logits(hq, hs, wq, ws, bias, temperature, real):
    """z [T, real] in fp64."""
    z = hq.astype(np.float64) @ wq[:real].astype(np.float64).T
    z *= hs.astype(np.float64)[:, None] * ws[:real].astype(np.float64)
    if bias is not None:
        z += np.asarray(bias, dtype=np.float64)[:real]
    return z * np.float64(np.float32(1.0 / temperature))


def score(z, targets, mask, offset=0):
    """Partials of one shard's logits z [T, n_real] (targets are global ids)."""
    T, n = z.shape
    out = dict(target_logit=np.zeros(T), in_range=np.zeros(T, np.uint8), lse=np.zeros(T),
               entropy=np.zeros(T), logp=np.zeros(T))
    for t in range(T):
        if mask is not None and mask[t] == 0:
            continue
        loc = targets[t] - offset
        hit = 0 <= loc < n
        if n == 0:
            out["lse"][t], out["logp"][t] = -np.inf, -np.inf
            continue
        m = z[t].max()
        p = np.exp(z[t] - m)
        lse = m + np.log(p.sum())
        out["lse"][t] = lse
        out["entropy"][t] = lse - (p * z[t]).sum() / p.sum()
        out["in_range"][t] = hit
        out["target_logit"][t] = z[t, loc] if hit else 0.0
        out["logp"][t] = z[t, loc] - lse if hit else -np.inf
    return out


def policy(logp, old, adv, ref=None, entropy=None, mask=None, cu=None, clip_low=0.2,
           clip_high=0.2, dual_clip=0.0, kl="k3", kl_coef=0.0, entropy_coef=0.0,
           reduction="token_mean", denominator=None, dloss=1.0):
    """loss, stats[8], dlogp, dentropy, and `size`: per row, what its rounding is measured by
    (|A| r (1 + |d|) + |kl_coef| (|g| + |kl|) (1 + |x|), times its weight), `mags`: the sums of the
    statistics' magnitudes (the ratio's times 1 + |d|)."""
    T = len(logp)
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    w = np.zeros(T)
    if reduction == "sum":
        w[on] = 1.0
    elif reduction == "token_mean":
        n = on.sum() if denominator is None else denominator
        w[on] = 1.0 / n if n > 0 else 0.0
    else:
        counts = [int(on[cu[s]:cu[s + 1]].sum()) for s in range(len(cu) - 1)]
        n = sum(c > 0 for c in counts) if denominator is None else denominator
        for s, c in enumerate(counts):
            rows = np.arange(cu[s], cu[s + 1])
            if c and n > 0:
                w[rows[on[rows]]] = 1.0 / (c * n)
    dlogp, dent, size = np.zeros(T), np.zeros(T), np.zeros(T)
    sums, mags = np.zeros(6), np.zeros(6)
    for t in np.nonzero(on)[0]:
        vals = [logp[t], old[t], adv[t]] + ([ref[t]] if ref is not None else []) + (
            [entropy[t]] if entropy is not None else [])
        if not np.isfinite(vals).all():
            continue
        lp, d, a = float(logp[t]), float(logp[t]) - float(old[t]), float(adv[t])
        r = np.exp(np.clip(d, -LOG_RATIO_MAX, LOG_RATIO_MAX))
        # one-sided forms of -min(A r, A clip(r)): each border as the definition states it
        hold, used = False, r
        if a > 0 and d > np.log1p(clip_high):
            hold, used = True, 1.0 + clip_high
        elif a < 0 and d < np.log1p(-clip_low) if clip_low < 1 else False:
            hold, used = True, 1.0 - clip_low
        elif a < 0 and dual_clip > 0 and d > np.log(dual_clip):
            hold, used = True, dual_clip
        pg = -a * used
        g = 0.0 if hold or abs(d) > LOG_RATIO_MAX else -a * r
        size[t] = abs(a) * max(r, abs(used)) * (1 + abs(d))
        k = 0.0
        if ref is not None:
            x = float(ref[t]) - lp
            y = np.clip(x, -LOG_RATIO_MAX, LOG_RATIO_MAX)
            k, gk = {"k1": (-x, 1.0), "k2": (0.5 * x * x, -x),
                     "k3": (np.expm1(y) - y, -np.expm1(y) if x == y else 0.0)}[kl]
            g += kl_coef * gk
            size[t] += abs(kl_coef) * (abs(gk) + abs(k)) * (1 + abs(x))
        e = float(entropy[t]) if entropy is not None else 0.0
        terms = np.array([pg, k, e, float(hold), r, -d])
        sums += w[t] * terms
        mags += w[t] * np.abs(terms) * np.array([1, 1, 1, 1, 1 + abs(d), 1])
        dlogp[t] = dloss * w[t] * g
        dent[t] = -dloss * w[t] * entropy_coef
        size[t] = size[t] * w[t] + w[t] * abs(entropy_coef * e)
    loss = sums[0] + kl_coef * sums[1] - entropy_coef * sums[2]
    return dict(loss=loss, stats=np.concatenate([[loss], sums, [float(on.sum())]]), dlogp=dlogp,
                dentropy=dent, size=size, mags=mags)


def preference(logp, cu, ref=None, mask=None, pair_weight=None, beta=0.1, kind="sigmoid",
               label_smoothing=0.0, gamma=0.0, average=False, reduction="mean", dloss=1.0):
    """loss, pair_loss, chosen, rejected, dlogp."""
    T, P = len(logp), (len(cu) - 1) // 2
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    x = np.zeros(T)
    x[on] = np.asarray(logp, np.float64)[on]
    if ref is not None:
        x[on] -= np.asarray(ref, np.float64)[on]
    out = dict(pair_loss=np.zeros(P), chosen=np.zeros(P), rejected=np.zeros(P), dlogp=np.zeros(T))
    total = 0.0
    per_pair = 1.0 / P if reduction == "mean" and P else 1.0
    for i in range(P):
        wt = 1.0 if pair_weight is None else float(pair_weight[i])
        R, rows, per = [], [], []
        for s in (2 * i, 2 * i + 1):
            k = np.arange(cu[s], cu[s + 1])
            k = k[on[k]]
            f = (1.0 / len(k) if len(k) else 0.0) if average else 1.0
            rows.append(k)
            per.append(f)
            R.append(x[k].sum() * f)
        if not np.isfinite(wt) or not np.isfinite(x[np.concatenate(rows)]).all():
            continue
        h = R[0] - R[1]
        m = beta * h - gamma
        if kind == "sigmoid":
            e = label_smoothing
            l = (1 - e) * np.logaddexp(0, -m) + e * np.logaddexp(0, m)
            g = beta * (e - np.exp(-np.logaddexp(0, m)))
        elif kind == "hinge":
            l, g = max(0.0, 1 - m), (-beta if m < 1 else 0.0)
        else:
            l, g = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
        out["pair_loss"][i], out["chosen"][i], out["rejected"][i] = l, beta * R[0], beta * R[1]
        total += wt * l
        out["dlogp"][rows[0]] = dloss * per_pair * wt * g * per[0]
        out["dlogp"][rows[1]] = -dloss * per_pair * wt * g * per[1]
    out["loss"] = total * per_pair
    return out


def embedding_grad(ids, dout, scale, n_real, local_size, offset=0, mask=None):
    """dweight [local_size, H], and per row the number of its tokens and the sum of |scale dout|."""
    dout = np.asarray(dout, np.float64)
    g = np.zeros((local_size, dout.shape[1]))
    n, size = np.zeros(local_size, np.int64), np.zeros_like(g)
    for t, i in enumerate(ids):
        loc = i - offset
        if (mask is not None and mask[t] == 0) or not 0 <= loc < n_real:
            continue
        g[loc] += scale * dout[t]
        size[loc] += abs(scale) * np.abs(dout[t])
        n[loc] += 1
    return g, n, size
