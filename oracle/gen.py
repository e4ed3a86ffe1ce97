"""fp64 CPU oracle of the operators that decode and train with a head in 8-bit floating point: plain
definitions, no code shared with the HIP path."""
import math

import numpy as np

BLOCK = 128


def e4m3_values():
    """The finite values of e4m3 that are not negative, by code 0 .. 126 (code 127 is NaN)."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    return np.array(out)


VALUES = e4m3_values()


def to_e4m3(x):
    """Codes of the nearest e4m3 values, ties to the even code; |x| up to 464 goes to 448."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(VALUES, a), 1, len(VALUES) - 1)
    mid = (VALUES[hi - 1] + VALUES[hi]) / 2
    code = np.where(a > mid, hi, np.where(a < mid, hi - 1, hi - 1 + (hi - 1) % 2))
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def from_e4m3(code):
    code = np.asarray(code)
    low = code & 0x7F
    v = np.where(low == 127, np.nan, VALUES[np.minimum(low, 126)])
    return np.where(code & 0x80, -v, v)


def quantize_blocks(x, rows=1, transpose=False):
    """x: fp32 values. Returns (codes [M, K padded], fp32 scales [row groups, groups])."""
    x = np.asarray(x, np.float32)
    x = x.T if transpose else x
    M, K = x.shape
    pad = np.zeros((M + -M % rows, K + -K % BLOCK), np.float32)
    pad[:M, :K] = x
    q = np.zeros(pad.shape, np.uint8)
    s = np.zeros((pad.shape[0] // rows, pad.shape[1] // BLOCK), np.float32)
    for i in range(s.shape[0]):
        for g in range(s.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(g * BLOCK, (g + 1) * BLOCK))
            b = pad[at]
            if not np.isfinite(b).all():
                s[i, g] = np.nan
                continue
            s[i, g] = np.float32(max(np.abs(b).max(), np.float32(1e-30))) * (np.float32(1) / np.float32(448))
            q[at] = to_e4m3((b / s[i, g]).astype(np.float32))
    return q[:M], s


def values(q, s, rows):
    """What codes and their scales stand for, in 64 bits."""
    wide = np.repeat(np.repeat(s.astype(np.float64), BLOCK, axis=1), rows, axis=0)[:q.shape[0]]
    return from_e4m3(q) * wide


def linear(x, w, bias=None):
    """x . w^T (+ bias) of values in 64 bits, and the sum of the products' sizes."""
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    return (y, size) if bias is None else (y + bias, size + np.abs(bias))


def beam_candidates(logits, num, c, offset=0, n_real=None):
    """value, token, max, sum of each row; c = fl32(1 / temperature)."""
    R, V = logits.shape
    n = V if n_real is None else n_real
    value = np.full((R, num), -np.inf)
    token = np.full((R, num), -1, np.int64)
    top, total = np.full(R, -np.inf), np.zeros(R)
    for r in range(R):
        x = logits[r, :n].astype(np.float64)
        if np.isnan(x).any() or np.isposinf(x).any():
            total[r] = -1
            continue
        order = sorted((v for v in range(n) if x[v] > -np.inf), key=lambda v: (-x[v], v))[:num]
        value[r, :len(order)] = x[order]
        token[r, :len(order)] = np.array(order, np.int64) + offset
        if order:
            top[r] = x[order[0]]
            total[r] = math.fsum(np.exp((x[x > -np.inf] - top[r]) * c))
    return value, token, top, total


def beam_select(logits, scores, num, c, finished=None, end_id=-1):
    """One step over the whole vocabulary: logits [B, K, V] (real columns), scores [B, K]."""
    B, K, V = logits.shape
    token = np.full((B, num), -1, np.int64)
    parent = np.full((B, num), -1, np.int64)
    score = np.full((B, num), -np.inf)
    for b in range(B):
        every = []
        for k in range(K):
            s = float(scores[b, k])
            if not s < np.inf or s == -np.inf:
                continue
            if finished is not None and finished[b, k]:
                every.append((-s, k, -1, end_id))
                continue
            x = logits[b, k].astype(np.float64)
            if np.isnan(x).any() or np.isposinf(x).any() or not (x > -np.inf).any():
                continue
            top = x.max()
            norm = math.log(math.fsum(np.exp((x[x > -np.inf] - top) * c)))
            every += [(-(s + ((x[v] - top) * c - norm)), k, v, v) for v in range(V) if x[v] > -np.inf]
        every = sorted(e for e in every if e[0] < np.inf)[:num]
        for i, (t, k, _, v) in enumerate(every):
            token[b, i], parent[b, i], score[b, i] = v, k, -t
    return token, parent, score


def beam_reorder(state, parents, out=None):
    """state [B * K, ...], parents [B, N]; what out (or the state) holds after."""
    B, N = parents.shape
    K = state.shape[0] // B
    out = state.copy() if out is None else out.copy()
    for b in range(B):
        for j in range(N):
            if 0 <= parents[b, j] < K:
                out[b * N + j] = state[b * K + parents[b, j]]
    return out
