"""Losses where a value, a weight or a layout is at its edge: pairs of weight 0, terms past
fp32's range."""
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
