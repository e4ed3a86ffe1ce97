"""The policy and preference losses against the fp64 oracle and against differences, their
refusal to read masked rows, malformed layouts, odd alignments, and the autograd nodes."""
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


def _cuts(g, T, S):
    return np.concatenate([[0], np.sort(g.integers(0, T + 1, S - 1)), [T]]).astype(np.int32)


def _rows(T, seed, spread=0.3):
    g = np.random.default_rng(seed)
    lp = -g.exponential(2.0, T)
    return dict(logp=lp.astype(np.float32), old=(lp + g.standard_normal(T) * spread).astype(np.float32),
                adv=g.standard_normal(T).astype(np.float32),
                ref=(lp + g.standard_normal(T) * spread).astype(np.float32),
                ent=g.exponential(1.0, T).astype(np.float32),
                mask=(g.random(T) < 0.7).astype(np.uint8), g=g)


def _run_policy(llp, x, use=("ref", "ent", "mask"), cu=None, **kw):
    def t(k):
        return dev(x[k]) if k in use else None
    out = llp.policy_grads(dev(x["logp"]), dev(x["old"]), dev(x["adv"]), ref_logp=t("ref"),
                           entropy=t("ent"), loss_mask=t("mask"),
                           cu_seqlens=None if cu is None else dev(cu), **kw)
    ref = O.policy(x["logp"], x["old"], x["adv"], ref=x["ref"] if "ref" in use else None,
                   entropy=x["ent"] if "ent" in use else None,
                   mask=x["mask"] if "mask" in use else None, cu=cu,
                   **{k: v for k, v in kw.items() if k not in ("status", "denominator", "dloss")},
                   **({"denominator": float(kw["denominator"])} if "denominator" in kw else {}),
                   **({"dloss": float(kw["dloss"])} if "dloss" in kw else {}))
    return out, ref


def _close_policy(out, ref, dloss=1.0):
    """A row's terms: the exponential 2 steps, its argument's rounding |d| or |x| half steps
    (counted in `size`), the products 4: at most 16 half steps of `size`. Sums are fp64, rounded
    once."""
    lim = 16 * EPS * ref["size"] * abs(dloss)
    err = np.abs(host(out["dlogp"]) - ref["dlogp"])
    assert np.all(err <= lim + 2 * EPS * np.abs(ref["dlogp"])), (err - lim).max()
    if out["dentropy"] is not None:
        assert np.all(np.abs(host(out["dentropy"]) - ref["dentropy"]) <= 2 * EPS * np.abs(ref["dentropy"]))
    total = 16 * EPS * ref["size"].sum() + 2 * EPS * abs(ref["loss"])
    assert abs(float(out["loss"]) - ref["loss"]) <= total
    s = host(out["stats"]).astype(np.float64)
    assert s[0] == float(out["loss"]) and s[7] == ref["stats"][7]
    assert abs(s[1] - ref["stats"][1]) <= total + 2 * EPS * abs(ref["stats"][1])
    # entropy, clipped, -d: exact per row; kl and r: 16 half steps of their magnitudes
    for k, n in ((2, 16), (3, 2), (4, 2), (5, 16), (6, 2)):
        assert abs(s[k] - ref["stats"][k]) <= n * EPS * max(ref["mags"][k - 1], 1e-30), k


@pytest.mark.parametrize("T", [0, 1, 2, 63, 1024, 1025, 4097, 40001])
@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean", "sum"])
def test_policy_sizes(llp, T, reduction):
    say(f"policy T={T} {reduction}")
    x = _rows(T, T + 1)
    cu = _cuts(x["g"], T, max(1, min(9, T)))
    out, ref = _run_policy(llp, x, cu=cu, reduction=reduction, kl_coef=0.1, entropy_coef=0.02,
                           dual_clip=3.0)
    _close_policy(out, ref)


@pytest.mark.parametrize("use", [(), ("ref",), ("ent",), ("mask",), ("ref", "ent", "mask")])
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
def test_policy_terms(llp, use, kl):
    x = _rows(700, 17)
    out, ref = _run_policy(llp, x, use=use, kl=kl, kl_coef=0.3 if "ref" in use else 0.0,
                           entropy_coef=0.05 if "ent" in use else 0.0, clip_high=0.28)
    _close_policy(out, ref)
    assert (out["dentropy"] is None) == ("ent" not in use)


def test_policy_ranges_borders_and_far_ratios(llp):
    # d from -60 to 60, zeros and both signs of the advantage, clip_low = 1 and 0 width.
    x = _rows(4000, 23)
    x["old"] = (x["logp"] + np.linspace(-60, 60, 4000)).astype(np.float32)
    x["ref"] = (x["logp"] + np.linspace(60, -60, 4000)).astype(np.float32)
    x["adv"][::7] = 0
    for kw in (dict(clip_low=1.0, clip_high=0.2), dict(clip_low=0.0, clip_high=0.0),
               dict(dual_clip=2.0), dict(dual_clip=1.0001)):
        out, ref = _run_policy(llp, x, kl_coef=0.1, **kw)
        _close_policy(out, ref)
        assert np.isfinite(host(out["dlogp"])).all()
    # d on the borders themselves: not clipped there, clipped one step outside
    lo, hi = np.float32(np.log1p(-0.2)), np.float32(np.log1p(0.2))
    steps = np.array([lo, np.nextafter(lo, np.float32(-9)), np.nextafter(lo, np.float32(9)), hi,
                      np.nextafter(hi, np.float32(9)), np.nextafter(hi, np.float32(-9))], np.float32)
    y = dict(logp=np.tile(steps, 2), old=np.zeros(12, np.float32),
             adv=np.repeat(np.float32([1, -1]), 6))
    out, ref = _run_policy(llp, y, use=())
    _close_policy(out, ref)
    assert np.array_equal(host(out["dlogp"]) == 0, ref["dlogp"] == 0)


def test_policy_k3_keeps_small_differences(llp):
    # exp(x) - x - 1 at |x| from 1e-6 to 1: its own size, not that of 1, measures the error.
    T = 300
    x = _rows(T, 3)
    x["logp"] = np.zeros(T, np.float32)
    x["ref"] = (np.logspace(-6, 0, T) * np.where(np.arange(T) % 2, 1, -1)).astype(np.float32)
    for t in (0, 150, 299):
        m = np.zeros(T, np.uint8)
        m[t] = 1
        out, ref = _run_policy(llp, dict(x, mask=m), kl_coef=1.0)
        assert abs(float(out["stats"][2]) - ref["stats"][2]) <= 16 * EPS * ref["stats"][2]


def test_policy_masked_rows_may_hold_anything(llp):
    x = _rows(3000, 5)
    cu = _cuts(x["g"], 3000, 12)
    clean, _ = _run_policy(llp, x, cu=cu, reduction="seq_mean", kl_coef=0.1, entropy_coef=0.1)
    off = np.nonzero(x["mask"] == 0)[0]
    for k, v in (("logp", np.nan), ("old", -np.inf), ("adv", np.inf), ("ref", np.finfo(np.float32).min),
                 ("ent", np.nan)):
        x[k][off] = v
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = _run_policy(llp, x, cu=cu, reduction="seq_mean", kl_coef=0.1, entropy_coef=0.1, status=st)
    for k in out:
        assert bytes_equal(out[k], clean[k]), k
    assert int(st) == 0 and not host(out["dlogp"])[off].any()


def test_policy_not_finite_rows_add_nothing(llp):
    x = _rows(500, 6)
    x["mask"][:] = 1
    for i, (k, v) in enumerate((("logp", -np.inf), ("old", np.nan), ("adv", np.inf), ("ref", np.nan),
                                ("ent", -np.inf))):
        x[k][10 * i + 3] = v
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ref = _run_policy(llp, x, kl_coef=0.1, entropy_coef=0.1, status=st)
    _close_policy(out, ref)
    assert int(st) == llp.STATUS_BITS["VALUE_NOT_FINITE"]
    assert not host(out["dlogp"])[3:50:10].any() and float(out["stats"][7]) == 500


def test_policy_nothing_scored_and_empty_sequences(llp):
    x = _rows(200, 8)
    x["mask"][:] = 0
    cu = np.array([0, 0, 50, 50, 200, 200], np.int32)
    for red in ("token_mean", "seq_mean", "sum"):
        out, _ = _run_policy(llp, x, cu=cu, reduction=red, kl_coef=0.1, entropy_coef=0.1)
        for k in out:
            assert not host(out[k]).any(), (red, k)
    x["mask"][60:70] = 1    # one of five sequences has rows
    out, ref = _run_policy(llp, x, cu=cu, reduction="seq_mean", kl_coef=0.1)
    _close_policy(out, ref)


def test_policy_denominator_and_upstream(llp):
    x = _rows(900, 9)
    cu = _cuts(x["g"], 900, 7)
    d = torch.tensor([123.0], device="cuda")
    up = torch.tensor([-2.5], device="cuda")
    for red in ("token_mean", "seq_mean"):
        out, ref = _run_policy(llp, x, cu=cu, reduction=red, kl_coef=0.1, denominator=d, dloss=up)
        _close_policy(out, ref, dloss=-2.5)
    for v in (0.0, -1.0, float("nan"), float("inf")):
        out, _ = _run_policy(llp, x, kl_coef=0.1, denominator=torch.tensor([v], device="cuda"))
        assert float(out["loss"]) == 0 and not host(out["dlogp"]).any()


@pytest.mark.parametrize("cu", [[0, 10, 5, 90], [1, 90], [0, 89], [0, 91], [0, -5, 90],
                                [0, 2000000000, 90], [-7, 40, 90]])
def test_losses_malformed_layouts(llp, cu):
    T = 90
    x = _rows(T, 10)
    cu = np.array(cu, np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = llp.policy_grads(dev(x["logp"]), dev(x["old"]), dev(x["adv"]), cu_seqlens=dev(cu),
                           reduction="seq_mean", status=st)
    for k in ("loss", "dlogp"):
        assert not host(out[k]).any()
    assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]
    st.zero_()
    mean, ref = _run_policy(llp, x, status=st, kl_coef=0.1)     # no layout: nothing to report
    _close_policy(mean, ref)
    assert int(st) == 0
    got = llp.policy_grads(dev(x["logp"]), dev(x["old"]), dev(x["adv"]), cu_seqlens=dev(cu), status=st)
    assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]
    assert bytes_equal(got["dlogp"], llp.policy_grads(dev(x["logp"]), dev(x["old"]), dev(x["adv"]))["dlogp"])
    if len(cu) % 2 == 1:
        st.zero_()
        p = llp.preference_grads(dev(x["logp"]), dev(cu), status=st)
        for k in p:
            assert not host(p[k]).any(), k
        assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]


@pytest.mark.parametrize("S", [4, 40, 600, 5000])
@pytest.mark.parametrize("kind", ["end", "start", "falls", "past", "below"])
def test_losses_malformed_layouts_of_many_rows(llp, S, kind):
    # The forms of several launches: no row is read or written past the ends, everything is 0.
    T = 9001
    say(f"malformed layout {kind} S={S}")
    x = _rows(T, S)
    cu = _cuts(x["g"], T, S)
    k = S // 2
    if kind == "end":
        cu[S] = T - 1
    elif kind == "start":
        cu[0] = 1
    elif kind == "falls":
        cu[k] = cu[k + 1] + 1
    elif kind == "past":
        cu[k] = 2 ** 31 - 1
    else:
        cu[k] = -2 ** 31
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = [dev(x[n]) for n in ("logp", "old", "adv")]
    out = llp.policy_grads(*a, cu_seqlens=dev(cu), reduction="seq_mean", loss_mask=dev(x["mask"]), status=st)
    for n in ("loss", "dlogp"):
        assert not host(out[n]).any(), n
    assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]
    st.zero_()
    got = llp.policy_grads(*a, cu_seqlens=dev(cu), loss_mask=dev(x["mask"]), status=st)
    assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]
    assert bytes_equal(got["dlogp"], llp.policy_grads(*a, loss_mask=dev(x["mask"]))["dlogp"])
    st.zero_()
    p = llp.preference_grads(a[0], dev(cu), loss_mask=dev(x["mask"]), status=st)
    for n in p:
        assert not host(p[n]).any(), n
    assert int(st) == llp.STATUS_BITS["LAYOUT_INVALID"]


@pytest.mark.parametrize("T", [700, 4096, 20001])
@pytest.mark.parametrize("S", [1024, 1025, 2048, 2049, 5000])
def test_policy_many_sequences(llp, T, S):
    say(f"policy T={T} S={S}")
    x = _rows(T, T + S)
    cu = _cuts(x["g"], T, S)
    kw = dict(reduction="seq_mean", kl_coef=0.1, entropy_coef=0.01)
    out, ref = _run_policy(llp, x, cu=cu, **kw)
    _close_policy(out, ref)
    again, _ = _run_policy(llp, x, cu=cu, **kw)
    assert all(bytes_equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("P,T", [(1, 8192), (8, 8192), (9, 8192), (8, 8193), (8, 16), (128, 5000), (129, 5000)])
def test_preference_where_the_launches_change(llp, P, T):
    say(f"preference P={P} T={T}")
    x = _rows(T, P + T)
    cu = _cuts(x["g"], T, 2 * P)
    out = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]), beta=0.2)
    ref = O.preference(x["logp"], cu, ref=x["ref"], mask=x["mask"], beta=0.2)
    _close_pref(out, ref, x)
    x["logp"][x["mask"] == 0] = np.nan             # rows that are not scored are not looked at
    same = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]), beta=0.2)
    assert all(bytes_equal(out[k], same[k]) for k in out)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_losses_on_unaligned_views_match_aligned(llp, shift):
    T = 2051
    x = _rows(T, 12)
    cu = dev(_cuts(x["g"], T, 8))

    def view(a):
        buf = torch.zeros(T + 8, dtype=torch.from_numpy(a).dtype, device="cuda")
        buf[shift:shift + T] = dev(a)
        return buf[shift:shift + T]
    kw = dict(cu_seqlens=cu, reduction="seq_mean", kl_coef=0.1, entropy_coef=0.1)
    a = llp.policy_grads(*(dev(x[k]) for k in ("logp", "old", "adv")), ref_logp=dev(x["ref"]),
                         entropy=dev(x["ent"]), loss_mask=dev(x["mask"]), **kw)
    b = llp.policy_grads(*(view(x[k]) for k in ("logp", "old", "adv")), ref_logp=view(x["ref"]),
                         entropy=view(x["ent"]), loss_mask=view(x["mask"]), **kw)
    for k in a:
        assert bytes_equal(a[k], b[k]), k
    out = dict(loss=torch.empty(1, device="cuda"), pair_loss=torch.empty(4, device="cuda"),
               chosen=torch.empty(4, device="cuda"), rejected=torch.empty(4, device="cuda"),
               dlogp=torch.empty(T + 8, device="cuda")[shift:shift + T])
    c = llp.preference_grads(dev(x["logp"]), cu, ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]))
    d = llp.preference_grads(view(x["logp"]), cu, ref_logp=view(x["ref"]), loss_mask=view(x["mask"]),
                             out=out)
    for k in c:
        assert bytes_equal(c[k], d[k]), k


def test_policy_gradient_against_differences(llp):
    # Central differences in fp64 of the oracle at rows away from the clip's borders.
    x = _rows(40, 14, spread=0.1)
    kw = dict(kl_coef=0.2, dual_clip=3.0)
    out, ref = _run_policy(llp, x, use=("ref", "mask"), **kw)
    h = 1e-6
    for t in range(40):
        d = float(x["logp"][t]) - float(x["old"][t])
        if min(abs(d - np.log1p(0.2)), abs(d - np.log1p(-0.2))) < 1e-3:
            continue
        v = []
        for s in (h, -h):
            lp = x["logp"].astype(np.float64)
            lp[t] += s
            v.append(O.policy(lp, x["old"], x["adv"], ref=x["ref"], mask=x["mask"], **kw)["loss"])
        # the loss's fp64 rounding over h, and the third derivative's h^2, stay below 1e-9
        lim = 16 * EPS * ref["size"][t] + 1e-9
        assert abs(float(out["dlogp"][t]) - (v[0] - v[1]) / (2 * h)) <= lim


PREF = [("sigmoid", dict()), ("sigmoid", dict(label_smoothing=0.2, gamma=0.5)), ("hinge", dict(gamma=-0.3)),
        ("ipo", dict())]


def _close_pref(out, ref, x):
    """Sums and pair terms are fp64: one final rounding, and 1e-13 of the summed magnitudes."""
    small = 1e-13 * (1 + np.abs(x["logp"][np.isfinite(x["logp"])]).sum())
    for k in ("loss", "pair_loss", "chosen", "rejected", "dlogp"):
        a, r = host(out[k]).astype(np.float64).reshape(-1), np.asarray(ref[k]).reshape(-1)
        # ipo squares the sum: its error grows by twice the value
        lim = 2 * EPS * np.abs(r) + small * (1 + 2 * np.sqrt(np.abs(r)))
        assert np.all(np.abs(a - r) <= lim), (k, np.abs(a - r).max())


@pytest.mark.parametrize("kind,kw", PREF)
@pytest.mark.parametrize("P,T", [(1, 2), (1, 1), (2, 63), (7, 3000), (33, 40000), (2, 70001), (1100, 9000)])
def test_preference(llp, kind, kw, P, T):
    say(f"preference {kind} P={P} T={T}")
    x = _rows(T, P * 31 + T)
    cu = _cuts(x["g"], T, 2 * P)
    for average, use_ref, use_mask, red in ((False, True, True, "mean"), (True, True, False, "sum"),
                                            (True, False, True, "mean")):
        out = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]) if use_ref else None,
                                   loss_mask=dev(x["mask"]) if use_mask else None, beta=0.2, kind=kind,
                                   average=average, reduction=red, **kw)
        ref = O.preference(x["logp"], cu, ref=x["ref"] if use_ref else None,
                           mask=x["mask"] if use_mask else None, beta=0.2, kind=kind, average=average,
                           reduction=red, **kw)
        _close_pref(out, ref, x)


def test_preference_weights_masks_and_not_finite(llp):
    P, T = 6, 600
    x = _rows(T, 77)
    cu = np.arange(0, T + 1, 50).astype(np.int32)
    x["mask"][100:200] = 0                       # pair 1 has no scored row
    x["logp"][130] = np.nan                      # masked: never read
    w = np.array([1, 2, 0, 0.5, 1, np.inf], np.float32)
    x["logp"][230] = np.nan                      # pair 2 has weight 0
    x["mask"][230] = 1
    x["logp"][330], x["mask"][330] = -np.inf, 1  # pair 3 is dropped and reported
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    up = torch.tensor([3.0], device="cuda")
    out = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]),
                               pair_weight=dev(w), status=st, dloss=up)
    ref = O.preference(x["logp"], cu, ref=x["ref"], mask=x["mask"], pair_weight=w, dloss=3.0)
    _close_pref(out, ref, x)
    assert int(st) == llp.STATUS_BITS["VALUE_NOT_FINITE"]
    assert np.isfinite(host(out["dlogp"])).all() and not host(out["dlogp"])[200:400].any()
    st.zero_()
    w[3], w[5] = 0, 1
    llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]),
                         pair_weight=dev(w), status=st)
    assert int(st) == 0


def test_preference_extreme_margins_and_no_pairs(llp):
    T = 400
    x = _rows(T, 80)
    x["logp"] = (x["logp"] * 50).astype(np.float32)
    cu = np.array([0, 100, 200, 390, 400], np.int32)
    for kind, kw in PREF:
        out = llp.preference_grads(dev(x["logp"]), dev(cu), beta=5.0, kind=kind, **kw)
        _close_pref(out, O.preference(x["logp"], cu, beta=5.0, kind=kind, **kw), x)
    none = llp.preference_grads(torch.empty(0, device="cuda"), dev(np.zeros(1, np.int32)))
    assert float(none["loss"]) == 0 and none["pair_loss"].shape == (0,)


def test_preference_sum_does_not_depend_on_the_packing_bitwise(llp):
    # A pair's rewards are those of its own rows, wherever they lie in the batch.
    x = _rows(30000, 81)
    cu = np.array([0, 12000, 17001, 17002, 30000], np.int32)
    whole = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]))
    sl = slice(17001, 30000)
    part = llp.preference_grads(dev(x["logp"][sl]), dev(cu[2:] - 17001), ref_logp=dev(x["ref"][sl]),
                                loss_mask=dev(x["mask"][sl]))
    for k in ("chosen", "rejected", "pair_loss"):
        assert bytes_equal(part[k], whole[k][1:]), k


def test_autograd_nodes(llp):
    T = 500
    x = _rows(T, 90)
    cu = _cuts(x["g"], T, 4)
    lp, ent = dev(x["logp"]).requires_grad_(True), dev(x["ent"]).requires_grad_(True)
    kw = dict(ref_logp=dev(x["ref"]), cu_seqlens=dev(cu), reduction="seq_mean", kl_coef=0.1,
              entropy_coef=0.05)
    loss, stats = llp.policy_loss(lp, dev(x["old"]), dev(x["adv"]), entropy=ent,
                                  loss_mask=dev(x["mask"]).bool(), **kw)
    assert loss.shape == () and not stats.requires_grad
    (loss * 3 + 1).backward()
    with torch.no_grad():
        g = llp.policy_grads(lp.detach(), dev(x["old"]), dev(x["adv"]), entropy=ent.detach(),
                             loss_mask=dev(x["mask"]), dloss=torch.tensor([3.0], device="cuda"), **kw)
    assert bytes_equal(lp.grad, g["dlogp"]) and bytes_equal(ent.grad, g["dentropy"])
    assert float(loss.detach()) == float(g["loss"])
    lp2 = dev(x["logp"]).requires_grad_(True)
    loss, chosen, rejected = llp.preference_loss(lp2, dev(cu), ref_logp=dev(x["ref"]),
                                                 loss_mask=dev(x["mask"]).bool())
    assert not chosen.requires_grad and not rejected.requires_grad
    loss.backward()
    g = llp.preference_grads(dev(x["logp"]), dev(cu), ref_logp=dev(x["ref"]), loss_mask=dev(x["mask"]))
    assert bytes_equal(lp2.grad, g["dlogp"])
