"""The operators together, as a training step uses them: a tied head embedded, scored, held against
a frozen 8-bit copy of itself, its policy or preference loss formed and everything differentiated
into one fp32 gradient; the same calls captured into a HIP graph and replayed, and run on several
streams at once."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
T, H, VR, VP, TAU, SCALE = 300, 256, 1900, 2048, 0.8, 16.0


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def _inputs(seed, n=T):
    g = np.random.default_rng(seed)
    w = torch.from_numpy((g.standard_normal((VP, H)) * 0.05).astype(np.float32)).to(torch.bfloat16).cuda()
    ids = g.integers(0, VR, n)
    ids[::5] = 7
    mask = (g.random(n) < 0.7).astype(np.uint8)
    cuts = np.concatenate([[0], np.sort(g.integers(0, n + 1, 7)), [n]]).astype(np.int32)
    return dict(w=w, ids=dev(ids), tg=dev(g.integers(0, VR, n)), mask=dev(mask), cu=dev(cuts),
                adv=dev(g.standard_normal(n).astype(np.float32)))


def _vocab():
    return dict(real_vocab=VR, padded_vocab=VP)


def test_policy_step_of_a_tied_head(llp):
    x = _inputs(1)
    kw = dict(kl_coef=0.1, entropy_coef=0.01, reduction="seq_mean", cu_seqlens=x["cu"])
    hidden = llp.embedding_forward(x["ids"], x["w"], scale=SCALE, real_vocab=VR)
    # the frozen reference: the same head in 8-bit integers
    hq, hs = llp.quantize_rows(hidden)
    wq, ws = llp.quantize_rows(x["w"])
    ref = llp.forward_int8(hq, hs, wq, ws, x["tg"], temperature=TAU, loss_mask=x["mask"], **_vocab())
    out = llp.forward(hidden, x["w"], x["tg"], temperature=TAU, loss_mask=x["mask"], **_vocab())
    old = out["logp"] + 0.1 * torch.randn(T, device="cuda")
    pg = llp.policy_grads(out["logp"], old, x["adv"], ref_logp=ref["logp"], entropy=out["entropy"],
                          loss_mask=x["mask"], **kw)
    want = O.policy(host(out["logp"]), host(old), host(x["adv"]), ref=host(ref["logp"]),
                    entropy=host(out["entropy"]), mask=host(x["mask"]), cu=host(x["cu"]), kl_coef=0.1,
                    entropy_coef=0.01, reduction="seq_mean")
    assert abs(float(pg["loss"]) - want["loss"]) <= 16 * EPS * want["size"].sum() + 2 * EPS * abs(want["loss"])
    bw = llp.backward(hidden, x["w"], x["tg"], out["lse"], pg["dlogp"], temperature=TAU, loss_mask=x["mask"],
                      dentropy=pg["dentropy"], entropy=out["entropy"], overwrite=True, **_vocab())
    head = bw["dweight"].clone()
    # the input side adds into the head's own gradient
    total = llp.embedding_backward(x["ids"], bw["dhidden"], dweight=bw["dweight"], scale=SCALE, real_vocab=VR)
    side, n, size = O.embedding_grad(host(x["ids"]), bw["dhidden"].float().cpu().numpy(), SCALE, VR, VP)
    err = np.abs(host(total).astype(np.float64) - (host(head) + side))
    assert np.all(err <= EPS * (n + 3)[:, None] * (size + np.abs(host(head))))
    # the autograd nodes give the same, each gradient in the parameter's type
    w = x["w"].clone().requires_grad_(True)
    h = llp.embedding(x["ids"], w, scale=SCALE, real_vocab=VR)
    logp, ent, _ = llp.linear_logp(h, w, x["tg"], temperature=TAU, loss_mask=x["mask"], **_vocab())
    loss, _ = llp.policy_loss(logp, old, x["adv"], ref_logp=ref["logp"], entropy=ent, loss_mask=x["mask"], **kw)
    loss.backward()
    assert bytes_equal(loss.detach().reshape(1), pg["loss"])
    alone = llp.embedding_backward(x["ids"], bw["dhidden"], local_size=VP, scale=SCALE, real_vocab=VR,
                                   overwrite=True)
    assert bytes_equal(w.grad, head.to(torch.bfloat16) + alone.to(torch.bfloat16))


def test_preference_step(llp):
    x = _inputs(2)
    w = x["w"].clone().requires_grad_(True)
    h = llp.embedding(x["ids"], w, scale=SCALE, real_vocab=VR)
    logp, _, _ = llp.linear_logp(h, w, x["tg"], temperature=TAU, loss_mask=x["mask"], want_entropy=False, **_vocab())
    hq, hs = llp.quantize_rows(h.detach())
    wq, ws = llp.quantize_rows(x["w"])
    ref = llp.forward_int8(hq, hs, wq, ws, x["tg"], temperature=TAU, loss_mask=x["mask"], want_entropy=False, **_vocab())
    loss, chosen, rejected = llp.preference_loss(logp, x["cu"], ref_logp=ref["logp"], loss_mask=x["mask"])
    loss.backward()
    want = O.preference(host(logp.detach()), host(x["cu"]), ref=host(ref["logp"]), mask=host(x["mask"]))
    assert abs(float(loss.detach()) - want["loss"]) <= 2 * EPS * abs(want["loss"]) + 1e-10
    bw = llp.backward(h.detach(), x["w"], x["tg"], llp.forward(
        h.detach(), x["w"], x["tg"], temperature=TAU, loss_mask=x["mask"], want_entropy=False, **_vocab())["lse"],
        dev(want["dlogp"].astype(np.float32)), temperature=TAU, loss_mask=x["mask"], overwrite=True, **_vocab())
    side = llp.embedding_backward(x["ids"], bw["dhidden"], local_size=VP, scale=SCALE, real_vocab=VR, overwrite=True)
    assert bytes_equal(w.grad, bw["dweight"].to(torch.bfloat16) + side.to(torch.bfloat16))


def _calls(llp, x, many):
    """Every new execution call, in its forms for few and for many rows."""
    emb = llp.embedding_forward(x["ids"], x["w"], scale=SCALE, real_vocab=VR)
    hq, hs = llp.quantize_rows(emb)
    wq, ws = llp.quantize_rows(x["w"])
    o = {"q": hq, "scale": hs, "emb": emb}
    for n in (40, emb.shape[0]):
        p = llp.forward_int8(hq[:n], hs[:n], wq, ws, x["tg"][:n], temperature=TAU, loss_mask=x["mask"][:n], **_vocab())
        o.update({f"int8.{n}.{k}": v for k, v in p.items()})
    lp, ent = o[f"int8.{emb.shape[0]}.logp"], o[f"int8.{emb.shape[0]}.entropy"]
    for red in ("token_mean", "seq_mean", "sum"):
        p = llp.policy_grads(lp, x["adv"] - 8, x["adv"], ref_logp=lp, entropy=ent, loss_mask=x["mask"],
                             cu_seqlens=x["cu"], reduction=red, kl_coef=0.1, entropy_coef=0.1)
        o.update({f"policy.{red}.{k}": v for k, v in p.items()})
    p = llp.preference_grads(lp, x["cu"], loss_mask=x["mask"])
    o.update({f"pref.{k}": v for k, v in p.items()})
    p = llp.preference_grads(lp, many, loss_mask=x["mask"])
    o.update({f"prefs.{k}": v for k, v in p.items()})
    o["dw"] = llp.embedding_backward(x["ids"], emb, local_size=VP, scale=SCALE, real_vocab=VR, overwrite=True)
    return o


def _many(n):
    return dev(np.linspace(0, n, 2 * 150 + 1).astype(np.int32))


def _fill(t):
    t.fill_(7) if t.dtype in (torch.uint8, torch.int8) else t.fill_(float("nan"))


@pytest.mark.parametrize("n", [300, 9000])
def test_graph_replays_match_eager(llp, n):
    # 300 rows: one workgroup for the policy loss, ids sorted without a pass; 9000: the other forms.
    x, other, many = _inputs(3, n), _inputs(4, n), _many(n)
    say(f"graph: eager calls, {n} rows")
    ref = {k: v.clone() for k, v in _calls(llp, x, many).items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _calls(llp, x, many)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    say("graph: capture")
    with torch.cuda.graph(g):
        outs = _calls(llp, x, many)
    torch.cuda.synchronize()
    for rep in range(4):
        say(f"graph: replay {rep}")
        _calls(llp, other, many)
        for v in outs.values():
            _fill(v)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in ref.items():
            assert bytes_equal(outs[k], v), (rep, k)


def test_two_graphs_and_two_streams_at_once(llp):
    a, b, many = _inputs(5, 2000), _inputs(6, 2000), _many(2000)
    ra = {k: v.clone() for k, v in _calls(llp, a, many).items()}
    rb = {k: v.clone() for k, v in _calls(llp, b, many).items()}
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            oa = _calls(llp, a, many)
        with torch.cuda.stream(s2):
            ob = _calls(llp, b, many)
        torch.cuda.synchronize()
        for k in ra:
            assert bytes_equal(oa[k], ra[k]) and bytes_equal(ob[k], rb[k]), k
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        oa = _calls(llp, a, many)
    with torch.cuda.graph(gb):
        ob = _calls(llp, b, many)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        torch.cuda.synchronize()
        for k in ra:
            assert bytes_equal(oa[k], ra[k]) and bytes_equal(ob[k], rb[k]), k


def test_losses_through_captured_autograd(llp):
    # Forward and backward of the nodes in one graph, upstream gradient included.
    x = _inputs(7)
    lp0 = llp.forward(llp.embedding_forward(x["ids"], x["w"]), x["w"], x["tg"], temperature=TAU, **_vocab())["logp"]
    lp = lp0.clone().requires_grad_(True)
    old = lp0 + 0.1

    def step():
        loss, _ = llp.policy_loss(lp, old, x["adv"], loss_mask=x["mask"])
        pref, _, _ = llp.preference_loss(lp, x["cu"], loss_mask=x["mask"])
        (gr,) = torch.autograd.grad(2 * loss + pref, lp)
        return gr

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = step().clone()
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        _fill(got)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert bytes_equal(got, want)
