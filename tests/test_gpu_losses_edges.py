"""Losses where a value, a weight or a layout is at its edge: pairs of weight 0, terms past
fp32's range, layouts that name the same rows for every sequence."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def _pairs(P, T, seed):
    g = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.sort(g.integers(0, T + 1, 2 * P - 1)), [T]]).astype(np.int32)
    lp = -g.exponential(2.0, T)
    return g, cu, dict(logp=lp.astype(np.float32), ref=(lp + 0.3 * g.standard_normal(T)).astype(np.float32),
                       mask=(g.random(T) < 0.7).astype(np.uint8))


# One workgroup; few pairs in two launches; many in three.
@pytest.mark.parametrize("P,T", [(3, 500), (20, 9000), (200, 9000)])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
def test_pairs_of_weight_zero_keep_their_own_outputs(llp, P, T, kind):
    say(f"pair weights P={P} T={T} {kind}")
    g, cu, x = _pairs(P, T, P)
    w = np.where(np.arange(P) % 3 == 1, 0, 1 + np.arange(P) % 4).astype(np.float32)
    kw = dict(ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]), beta=0.2, kind=kind)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = llp.preference_grads(dev(x["logp"]), dev(cu), pair_weight=dev(w), status=st, **kw)
    same = llp.preference_grads(dev(x["logp"]), dev(cu), **kw)
    ref = O.preference(x["logp"], cu, ref=x["ref"], mask=x["mask"], pair_weight=w, beta=0.2, kind=kind)
    assert int(st) == 0
    for k in ("pair_loss", "chosen", "rejected"):
        assert bytes_equal(out[k], same[k]), k          # their own: whatever the weights
        # fp64 sums and pair terms (1e-13 of the magnitudes), rounded once; twice the value for ipo
        lim = 2 * EPS * np.abs(ref[k]) + 1e-13 * (1 + np.abs(x["logp"]).sum()) * (1 + 2 * np.sqrt(np.abs(ref[k])))
        assert np.all(np.abs(host(out[k]) - ref[k]) <= lim), k
    own = host(out["pair_loss"]).astype(np.float64)     # half a step of each, and of the loss
    assert abs(float(out["loss"]) - (w * own).sum() / P) <= 2 * EPS * (w * np.abs(own)).sum() / P
    for i in np.nonzero(w == 0)[0]:
        assert not host(out["dlogp"])[cu[2 * i]:cu[2 * i + 2]].any()
        assert host(out["chosen"])[i] != 0 or cu[2 * i] == cu[2 * i + 1] or not x["mask"][cu[2 * i]:cu[2 * i + 1]].any()


# One workgroup, and several.
@pytest.mark.parametrize("T", [8, 5000])
@pytest.mark.parametrize("case", ["k2 of coefficient 0", "large advantages", "no denominator", "far reference"])
def test_policy_terms_past_fp32_of_finite_rows(llp, T, case):
    # Finite inputs whose term passes 3.4e38 before its weight: 0 of it is 0, a mean of it is finite.
    say(f"policy {case} T={T}")
    g = np.random.default_rng(T)
    low = np.finfo(np.float32).min
    lp = (-g.exponential(2.0, T)).astype(np.float32)
    x = dict(logp=lp, old=(lp - np.float32(0.125)).astype(np.float32), adv=g.standard_normal(T).astype(np.float32))
    ref = (lp + np.float32(0.25)).astype(np.float32)
    kw = dict(kl="k2", kl_coef=0.0)
    if case == "k2 of coefficient 0":
        x["logp"][3] = x["old"][3] = low
    elif case == "far reference":
        kw = dict(kl="k1", kl_coef=1e-3)
        x["logp"][3] = x["old"][3] = np.float32(-3e38)
        ref[3] = np.float32(3e38)
    else:
        x["adv"][3] = np.float32(3.3e38)     # times r = e^0.125 = 1.133, inside the clip
    den = {}
    if case == "no denominator":
        den = dict(denominator=torch.zeros(1, device="cuda"))
    out = llp.policy_grads(dev(x["logp"]), dev(x["old"]), dev(x["adv"]), ref_logp=dev(ref), **kw, **den)
    for k in ("loss", "dlogp"):
        assert np.isfinite(host(out[k])).all(), (k, case)
    if den:
        assert not any(host(out[k])[:7].any() for k in ("loss", "stats", "dlogp"))
        return
    r = O.policy(x["logp"], x["old"], x["adv"], ref=ref, **kw)
    # the exponential 2 steps, its argument |d| half steps, the products 4, the last rounding
    lim = 16 * EPS * np.maximum(np.abs(r["dlogp"]), 1e-30)
    assert np.all(np.abs(host(out["dlogp"]) - r["dlogp"]) <= lim)
    size = np.abs(x["adv"].astype(np.float64)).sum() * 1.2 / T + abs(r["loss"])
    assert abs(float(out["loss"]) - r["loss"]) <= 16 * EPS * size
    with np.errstate(over="ignore"):
        want = r["stats"][2].astype(np.float32)
    assert float(out["stats"][2]) == want or abs(float(out["stats"][2]) - r["stats"][2]) <= 16 * EPS * abs(want)


def test_layouts_that_name_all_rows_for_every_sequence_cost_no_more(llp):
    # 2^19 sequences of 2^22 rows each: read as they stand, 2e12 mask bytes and 2e13 of log-probs.
    S, T = 1 << 20, 1 << 22
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    lp = torch.randn(T, device="cuda")
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = (lambda: llp.policy_grads(lp, lp, lp, cu_seqlens=cu, loss_mask=mask, reduction="seq_mean", status=st),
             lambda: llp.preference_grads(lp, cu, loss_mask=mask, status=st))
    for name, call in zip(("policy", "preference"), calls):
        say(f"layout of {S} x {T} rows: {name}")
        st.zero_()
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ends[0].record()
        out = call()
        ends[1].record()
        torch.cuda.synchronize()
        for k in out:
            assert out[k] is None or not host(out[k]).any(), k
        assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]
        ms = ends[0].elapsed_time(ends[1])
        say(f"{name}: {ms:.2f} ms")
        assert ms < 200     # 2e12 bytes take longer than this at twice the memory's rate


def test_losses_of_well_formed_layouts_looked_over_first(llp):
    # 2^20 sequences, most of them empty, of 2^18 rows: the layout is looked over before it is used.
    S, T = 1 << 20, 1 << 18
    g = np.random.default_rng(2)
    cu = np.concatenate([[0], np.sort(g.integers(0, T + 1, S - 1)), [T]]).astype(np.int32)
    lp, adv = -g.exponential(1.0, T).astype(np.float32), g.standard_normal(T).astype(np.float32)
    mask = (g.random(T) < 0.7).astype(np.uint8)
    on = mask != 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("policy and preference of 2^20 sequences")
    out = llp.policy_grads(dev(lp), dev(lp), dev(adv), cu_seqlens=dev(cu), loss_mask=dev(mask),
                           reduction="seq_mean", status=st)
    seq = np.searchsorted(cu, np.arange(T), side="right") - 1
    n = np.bincount(seq[on], minlength=S)
    w = np.where(on, 1.0 / (np.maximum(n, 1)[seq] * (n > 0).sum()), 0.0)
    # ratios are 1: each term is its advantage, exact; fp64 sums, rounded once
    assert np.all(np.abs(host(out["dlogp"]) + w * adv) <= 2 * EPS * w * np.abs(adv))
    assert abs(float(out["loss"]) + (w * adv).sum()) <= 2 * EPS * (w * np.abs(adv)).sum()
    assert float(out["stats"][7]) == on.sum() and int(st) == 0
    p = llp.preference_grads(dev(lp), dev(cu), loss_mask=dev(mask), beta=0.5, status=st)
    R = np.bincount(seq[on], weights=lp[on].astype(np.float64), minlength=S)
    h = R[0::2] - R[1::2]
    lim = 2 * EPS * np.abs(R) + 1e-12
    assert np.all(np.abs(host(p["chosen"]) - 0.5 * R[0::2]) <= lim[0::2])
    assert np.all(np.abs(host(p["rejected"]) - 0.5 * R[1::2]) <= lim[1::2])
    per = np.logaddexp(0, -0.5 * h)
    assert abs(float(p["loss"]) - per.mean()) <= 2 * EPS * per.mean() + 1e-12 and int(st) == 0
    gr = -0.5 / (1 + np.exp(0.5 * h)) / (S // 2)
    want = np.where(on, np.where(seq % 2 == 0, 1, -1) * gr[seq // 2], 0.0)
    assert np.all(np.abs(host(p["dlogp"]) - want) <= 2 * EPS * np.abs(want) + 1e-18)
