"""The normalisers of a beam search's rows where few tokens hold the mass, against sums in 64 bits, and choices
between beams whose totals lie close together."""
import math

import numpy as np
import pytest
import torch

from tests._gpu import dev, host, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def sums(x, c):
    """Of each row: the sum, and how far it may be off. A term e = 2^t, t = (x - m) c log2 e with m the largest of
    its block, no further off than the row's largest: the exponential is off by an ulp, 2^-23 e at most; t by two
    roundings to fp32, 2^-24 |t| each, which move e by ln 2 |t| 2^-23 e = (m - x) c 2^-23 e; below 2^-126 it may be 0.
    A block's largest is 1 exactly. All else is in 64 bits: 2^-53 for each of the fewer than 128 additions that a term
    goes through, and as little again for the blocks' factors."""
    x = x.astype(np.float64)
    top = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = np.where(x > -np.inf, (x - top) * c, -np.inf)
        e = np.exp(d)
        off = np.where((d < 0) & (e > 0), e * (1 - d), 0.0)
    total = np.array([math.fsum(r) for r in e])
    return total, 2.0 ** -23 * off.sum(1) + 2.0 ** -126 * x.shape[1] + 2.0 ** -45 * total


def rows(kind, g, R, V):
    x = (g.standard_normal((R, V)) * 2).astype(np.float32)
    at = g.integers(0, V, R)
    if kind == "one token":
        x[np.arange(R), at] = 25 + g.random(R)
    elif kind == "one token and a mask":
        x[:] = -np.inf
        x[:, ::3] = -18
        x[np.arange(R), at] = 1
    elif kind == "a few tokens":
        for _ in range(4):
            x[np.arange(R), g.integers(0, V, R)] = 22 + 3 * g.random(R)
    elif kind == "far below one":
        x = (-17.0 - 0.01 * g.random((R, V))).astype(np.float32)
        x[np.arange(R), at] = 0
    elif kind == "equal":
        x[:] = -3
        x[np.arange(R), at] = 6
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["one token", "one token and a mask", "a few tokens", "far below one", "equal", "flat"])
@pytest.mark.parametrize("V", [9, 2048, 5001, 151669])
def test_sums_of_rows_that_few_tokens_dominate(llp, V, kind, dtype):
    say(f"beam sums V={V} {kind} {dtype}")
    R = 16 if V > 100000 else 64
    x = rows(kind, np.random.default_rng(V), R, V)
    z = torch.zeros((R, V + -V % 8), dtype=dtype, device="cuda")[:, :V]
    z.copy_(torch.from_numpy(x))
    for tau in (1.0, 0.5):
        got = llp.beam_candidates(z, 4, temperature=tau)
        total, off = sums(host(z.float()), 1.0 / tau)
        err = np.abs(host(got["sum"]) - total)
        assert (err <= off).all(), f"{float((err / off).max()):.3g} of the bound, {float((err / total).max()):.2g} off"


def test_choices_between_beams_close_together(llp):
    # Two beams, each of one token and little beside it, 1e-8 apart in their totals (and 3e-8, 1e-7, 3e-7): what
    # is beside the token, under a thousandth of the mass, moves a total by less than 1e-3 * 2^-23 (1 + 18).
    g = np.random.default_rng(9)
    B, V = 400, 6007
    x = (g.standard_normal((2 * B, V))).astype(np.float32)
    top = (18 + 2 * g.random(2 * B)).astype(np.float32)
    x[np.arange(2 * B), g.integers(0, V, 2 * B)] = top
    total, _ = sums(x, 1.0)
    assert (total - 1 < 1e-3).all()
    norm = np.log(total).reshape(B, 2)
    gap = np.array([1e-8, -1e-8, 3e-8, -3e-8, 1e-7, -1e-7, 3e-7, -3e-7])[np.arange(B) % 8]
    scores = np.stack([(norm[:, 0] - norm[:, 1] + gap), np.zeros(B)], axis=1).astype(np.float32)
    t = scores.astype(np.float64) - norm
    diff = t[:, 0] - t[:, 1]
    assert (np.abs(diff) > 5e-9).all()
    z = torch.zeros((2 * B, V + -V % 8), device="cuda")[:, :V]
    z.copy_(torch.from_numpy(x))
    got = llp.beam_select([llp.beam_candidates(z, 2)], dev(scores), 2)
    assert np.array_equal(host(got["parent"])[:, 0], (diff < 0).astype(np.int32))
