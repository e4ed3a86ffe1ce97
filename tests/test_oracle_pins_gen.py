"""Pins of the oracle of the fp8 and beam-search operators (oracle/gen.py): torch's own conversions, softmax and
sorts in fp64, closed forms and invariants. Runs on the CPU."""
import math

import numpy as np
import pytest
import torch

from oracle import gen as O

G = np.random.default_rng(11)


def test_e4m3_against_torch():
    assert len(O.VALUES) == 127 and O.VALUES[-1] == 448 and O.VALUES[1] == 2.0 ** -9 and O.VALUES[8] == 2.0 ** -6
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.from_e4m3(codes), want.astype(np.float64), equal_nan=True)
    mids = (O.VALUES[1:] + O.VALUES[:-1]) / 2
    x = np.concatenate([G.standard_normal(4000) * 10.0 ** G.uniform(-5, 2.2, 4000), mids, -mids, O.VALUES, [0.0, -0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    assert np.array_equal(O.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("rows,transpose", [(1, False), (1, True), (128, False), (128, True)])
def test_quantise_holds_every_value_within_half_a_step(rows, transpose):
    x = (G.standard_normal((140, 300)) * 10.0 ** G.uniform(-4, 4, (140, 1))).astype(np.float32)
    q, s = O.quantize_blocks(x, rows, transpose)
    y = x.T if transpose else x
    M, K = y.shape
    assert q.shape == (M, K + -K % 128) and s.shape == (-(-M // rows), q.shape[1] // 128)
    assert not q[:, K:].any()
    v = O.values(q, s, rows)[:, :K]
    wide = np.repeat(np.repeat(s, 128, axis=1), rows, axis=0)[:M, :K]
    # e4m3: 2^-4 of the value, or half of 2^-9 below the normal numbers, and the quotient's rounding
    assert (np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 1e-6)).all()
    tops = [np.abs(y[:, g:g + 128]).max(axis=1) for g in range(0, K, 128)]
    if rows == 1:
        assert np.allclose(s, np.stack(tops, axis=1) / 448.0, rtol=2e-7, atol=0)
    # The largest of a block is held at the largest code.
    assert (np.abs(O.from_e4m3(q)).max(axis=1) <= 448).all() and (np.abs(O.from_e4m3(q)) == 448).any()
    t, ts = O.quantize_blocks(np.ascontiguousarray(y), rows)
    assert np.array_equal(t, q) and np.array_equal(ts, s)


def test_quantise_of_blocks_that_are_not_finite_or_zero():
    x = np.ones((130, 260), np.float32)
    x[0, 5], x[129, 259] = np.nan, np.inf
    x[1] = 0
    q, s = O.quantize_blocks(x)
    assert np.isnan(s[0, 0]) and np.isnan(s[129, 2]) and np.isnan(s).sum() == 2 and not q[0, :128].any()
    assert not q[1].any() and (s[1] == np.float32(1e-30) * (np.float32(1) / np.float32(448))).all()
    q, s = O.quantize_blocks(x, 128)
    assert np.isnan(s[0, 0]) and np.isnan(s[1, 2]) and np.isnan(s).sum() == 2
    assert (O.values(q, s, 128)[3, 128:260] == 448.0 * float(s[0, 1])).all()


def test_linear_against_torch_and_its_transposes():
    x = (G.standard_normal((9, 200))).astype(np.float32)
    w = (G.standard_normal((140, 200))).astype(np.float32)
    xv, wv = O.values(*O.quantize_blocks(x), 1), O.values(*O.quantize_blocks(w, 128), 128)
    y, size = O.linear(xv, wv, np.arange(140.0))
    want = torch.nn.functional.linear(torch.from_numpy(xv), torch.from_numpy(wv), torch.arange(140.0, dtype=torch.float64))
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-12) and (size >= np.abs(y) - 1e-9).all()
    # A weight's blocks are its transpose's: the input gradient reads the same values.
    wt = O.values(*O.quantize_blocks(w, 128, True), 128)
    assert np.array_equal(wt[:200, :140], wv[:140, :200].T)


@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_candidates_against_torch(tau):
    c = float(np.float32(1 / np.float32(tau).astype(np.float64)))
    x = (G.standard_normal((5, 333)) * 3).astype(np.float32)
    value, token, top, total = O.beam_candidates(x, 7, c, offset=100, n_real=300)
    t = torch.from_numpy(x[:, :300]).double()
    v, i = torch.topk(t, 7)
    assert np.array_equal(value, v.numpy()) and np.array_equal(token, i.numpy() + 100)
    lse = torch.logsumexp(t * c, dim=1).numpy()
    assert np.allclose(top * c + np.log(total), lse, rtol=1e-13, atol=0)


def test_candidates_of_masked_broken_and_equal_rows():
    x = np.full((4, 6), -np.inf, np.float32)
    x[1, [2, 5]] = 3.0
    x[2] = [1, np.nan, 2, 3, 4, 5]
    x[3] = [1, 1, 0, 1, -np.inf, 1]
    value, token, top, total = O.beam_candidates(x, 3, 1.0)
    assert token.tolist() == [[-1, -1, -1], [2, 5, -1], [-1, -1, -1], [0, 1, 3]]
    assert total[0] == 0 and total[1] == 2 and total[2] == -1 and top[0] == -np.inf


def test_select_against_torch_and_rules():
    B, K, V, c = 2, 3, 50, 1.0
    x = (G.standard_normal((B, K, V)) * 2).astype(np.float32)
    scores = -G.uniform(0, 3, (B, K)).astype(np.float32)
    token, parent, score = O.beam_select(x, scores, 6, c)
    t = torch.from_numpy(scores).double()[:, :, None] + torch.log_softmax(torch.from_numpy(x).double(), dim=2)
    v, i = torch.sort(t.reshape(B, -1), dim=1, descending=True, stable=True)
    assert np.allclose(score, v[:, :6].numpy(), rtol=1e-13, atol=1e-13)
    assert np.array_equal(parent * V + token, i[:, :6].numpy())
    # All of a softmax: the scores' exponentials sum to the beams' own.
    token, parent, score = O.beam_select(x, scores, K * V, c)
    assert np.allclose(np.exp(score).sum(axis=1), np.exp(scores.astype(np.float64)).sum(axis=1), rtol=1e-12)
    # A finished beam offers one candidate at its own score; the others go on as they did.
    done = np.zeros((B, K), np.uint8)
    done[0, 1] = 1
    token, parent, score = O.beam_select(x, scores, 2 * V + 2, c, done, 7)
    at = np.nonzero(parent[0] == 1)[0]
    assert len(at) == 1 and token[0, at[0]] == 7 and score[0, at[0]] == scores[0, 1]
    assert token[0, -1] == -1 and score[0, -1] == -np.inf and parent[0, -1] == -1
    # Equal beams: the lowest comes first.
    token, parent, score = O.beam_select(np.stack([x[:, 0]] * 3, axis=1), np.zeros((B, 3)), 6, c)
    assert (parent[:, :3] == [0, 1, 2]).all() and (parent[:, 3:] == [0, 1, 2]).all()
    scores[0, 0], scores[0, 1] = np.nan, np.inf
    assert (O.beam_select(x, scores, 4, c)[1][0] == 2).all()


def test_reorder_against_indexing():
    s = G.standard_normal((6, 2, 5))
    p = np.array([[2, 0, 0], [-1, 1, 5]])
    assert np.array_equal(O.beam_reorder(s, p), s[[2, 0, 0, 3, 4, 5]])
    out = np.full((4, 2, 5), 9.0)
    got = O.beam_reorder(s, np.array([[1, -1], [2, 2]]), out)
    assert np.array_equal(got[0], s[1]) and (got[1] == 9).all() and np.array_equal(got[2:], s[[5, 5]])


@pytest.mark.parametrize("mistake", ["scale of the row", "ties away", "normaliser left out", "tie to the higher token",
                                     "finished beam spreads"])
def test_planted_mistakes_fail_a_pin(mistake, monkeypatch):
    if mistake == "scale of the row":
        real = O.quantize_blocks
        monkeypatch.setattr(O, "quantize_blocks", lambda x, rows=1, transpose=False: (
            real(x, rows, transpose)[0], np.roll(real(x, rows, transpose)[1], 1, axis=0)))
        with pytest.raises(AssertionError):
            test_quantise_holds_every_value_within_half_a_step(1, False)
    elif mistake == "ties away":
        monkeypatch.setattr(O, "to_e4m3", lambda x: (np.searchsorted(
            (O.VALUES[1:] + O.VALUES[:-1]) / 2, np.abs(x), side="right") | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8))
        with pytest.raises(AssertionError):
            test_e4m3_against_torch()
    else:
        real = O.beam_select
        if mistake == "normaliser left out":
            def wrong(logits, scores, num, c, finished=None, end_id=-1):
                return real(logits - 1.0, scores + 1.0, num, c, finished, end_id)
        elif mistake == "tie to the higher token":
            def wrong(logits, scores, num, c, finished=None, end_id=-1):
                t, p, s = real(logits[:, ::-1], scores[:, ::-1], num, c, finished, end_id)
                return t, logits.shape[1] - 1 - p, s
        else:
            def wrong(logits, scores, num, c, finished=None, end_id=-1):
                return real(logits, scores, num, c)
        monkeypatch.setattr(O, "beam_select", wrong)
        with pytest.raises(AssertionError):
            test_select_against_torch_and_rules()
