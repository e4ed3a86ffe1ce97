"""Scoring with a head in 8-bit integers against the fp64 oracle: quantised rows exactly, the
partials within what their roundings allow, and the forward's guarantees (shards, masks, batch
invariance bitwise, empty shards, status bits)."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24   # half a step of fp32


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


@pytest.mark.parametrize("R,K,dtype,ld", [
    (1, 1, "f32", 1), (3, 7, "bf16", 7), (5, 128, "bf16", 136), (9, 130, "f32", 131),
    (257, 320, "bf16", 320), (33, 4096, "bf16", 4096), (17, 4104, "f32", 4104),
    (4, 8192 + 24, "bf16", 8224), (2, 5001, "f32", 5003), (66, 1000, "bf16", 1001)])
def test_quantize_rows_exactly(llp, R, K, dtype, ld):
    say(f"quantize R={R} K={K} {dtype} ld={ld}")
    g = np.random.default_rng(R * 10007 + K)
    x = torch.from_numpy((g.standard_normal((R, ld)) * 10.0 ** g.uniform(-6, 6, (R, 1))).astype(np.float32))
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    x[0, 0] = 0
    if R > 2:
        x[1] = 0                                   # a row of zeros
        # halves of a step: with the row's top at 127 the scale is 1 and ties go to even
        x[2, :K] = torch.arange(K).remainder(253).sub(126).to(x.dtype) / 2
        x[2, 0] = 127
    xd = x.cuda()[:, :K]
    q, s = llp.quantize_rows(xd)
    torch.cuda.synchronize()
    rq, rs = O.quantize(x[:, :K].float().numpy())
    assert q.shape == rq.shape and np.array_equal(host(s), rs)
    assert np.array_equal(host(q), rq)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [511, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193])
def test_quantize_rows_where_the_team_of_lanes_changes(llp, K, dtype):
    say(f"quantize K={K} {dtype}")
    g = np.random.default_rng(K)
    x = torch.from_numpy((g.standard_normal((11, K)) * 10.0 ** g.uniform(-6, 6, (11, 1))).astype(np.float32))
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    x[3, K - 1] = 9e8                              # the row's top in its last column
    x[4, K // 2] = float("inf")
    q, s = llp.quantize_rows(x.cuda())
    rq, rs = O.quantize(x.float().numpy())
    fine = np.arange(11) != 4
    assert np.array_equal(host(s)[fine], rs[fine]) and np.array_equal(host(q)[fine], rq[fine])
    assert np.isnan(host(s)[4]) and not host(q)[4].any()


def test_quantize_rows_near_ties_and_odd_values(llp):
    # Every bf16 value of two binades against scales that put quotients next to the halves.
    bits = np.arange(0x3F80, 0x4080, dtype=np.uint16)
    vals = (bits.astype(np.uint32) << 16).view(np.float32)
    rows = np.stack([np.concatenate([vals, [np.float32(m)]]) for m in
                     np.linspace(4.0, 9.0, 301, dtype=np.float32)])
    q, s = llp.quantize_rows(torch.from_numpy(rows).cuda())
    rq, rs = O.quantize(rows)
    assert np.array_equal(host(s), rs) and np.array_equal(host(q), rq)
    bad = np.ones((5, 200), np.float32)
    bad[0, 3], bad[1, 199], bad[2, 0] = np.nan, np.inf, -np.inf
    bad[3] = 1e-38
    bad[4] = 3e38
    q, s = llp.quantize_rows(torch.from_numpy(bad).cuda())
    rq, rs = O.quantize(bad)
    assert np.array_equal(host(s), rs, equal_nan=True) and np.array_equal(host(q), rq)
    empty = llp.quantize_rows(torch.empty((0, 64), device="cuda"))
    assert empty[0].shape == (0, 128) and empty[1].shape == (0,)


def _case(T, H, real, pad, seed, bias=None, mask_frac=0.0, spread=0.05):
    g = np.random.default_rng(seed)
    h = g.standard_normal((T, H)).astype(np.float32)
    w = (g.standard_normal((pad, H)) * spread).astype(np.float32)
    hq, hs = O.quantize(h)
    wq, ws = O.quantize(w)
    b = None
    if bias:
        b = torch.from_numpy(g.standard_normal(pad).astype(np.float32))
        b = b.to(torch.bfloat16) if bias == "bf16" else b
    mask = None if not mask_frac else (g.random(T) >= mask_frac).astype(np.uint8)
    return dict(hq=hq, hs=hs, wq=wq, ws=ws, b=b, mask=mask, tg=g.integers(0, real, T))


def _dev(c):
    return dict(hq=dev(c["hq"]), hs=dev(c["hs"]), wq=dev(c["wq"]), ws=dev(c["ws"]),
                tg=dev(c["tg"]), b=None if c["b"] is None else c["b"].cuda(),
                mask=None if c["mask"] is None else dev(c["mask"]))


def _close(out, ref, z, entropy=True):
    """z carries 4 roundings (scales, bias, 1/tau) and d2 = z log2 e two more, each relative to
    z; the sums of exponentials 160 (64 in a lane, the pair, the halves, 16 chains, the fold;
    the exponential's own 2); the rest is final. Entropy weighs the sums by its size."""
    top = np.abs(z).max() if z.size else 0.0
    tol = EPS * (16 * top + 160)
    for k in ("target_logit", "lse", "logp") + (("entropy",) if entropy else ()):
        x, r = host(out[k]).astype(np.float64), ref[k]
        assert np.array_equal(np.isneginf(x), np.isneginf(r)), k
        fin = np.isfinite(r)
        lim = tol * (2 + np.abs(r[fin])) if k == "entropy" else tol
        assert np.all(np.abs(x[fin] - r[fin]) <= lim), (k, np.abs(x[fin] - r[fin]).max(), tol)
    assert np.array_equal(host(out["in_range"]), ref["in_range"])


@pytest.mark.parametrize("T,H,real,pad,bias,mask,tau", [
    (1, 128, 5, 5, None, 0.0, 1.0), (1, 256, 1000, 1024, None, 0.0, 0.7),
    (2, 384, 257, 300, "f32", 0.0, 1.0), (33, 128, 256, 256, "bf16", 0.3, 0.7),
    (64, 256, 1000, 1024, None, 0.0, 1.0), (65, 512, 2003, 2048, "f32", 0.2, 1.3),
    (256, 320, 511, 512, "bf16", 0.0, 0.7), (257, 640, 700, 704, None, 0.5, 0.7),
    (300, 1024, 1900, 2000, "bf16", 0.25, 0.8), (7, 4096, 3001, 3008, None, 0.0, 1.0),
    (17, 1000, 901, 910, "f32", 0.1, 0.7), (130, 256, 20000, 20001, None, 0.1, 0.7)])
def test_forward_int8_parity(llp, T, H, real, pad, bias, mask, tau):
    say(f"int8 forward T={T} H={H} V={real}/{pad} bias={bias} mask={mask} tau={tau}")
    c = _case(T, H, real, pad, seed=T * 7 + H, bias=bias, mask_frac=mask)
    d = _dev(c)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], temperature=tau,
                           bias=d["b"], loss_mask=d["mask"], real_vocab=real, padded_vocab=pad,
                           status=st)
    torch.cuda.synchronize()
    b = None if c["b"] is None else c["b"].float().numpy()
    z = O.int8_logits(c["hq"], c["hs"], c["wq"], c["ws"], b, tau, real)
    _close(out, O.score(z, c["tg"], c["mask"]), z)
    assert int(st) == 0
    again = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], temperature=tau,
                             bias=d["b"], loss_mask=d["mask"], real_vocab=real, padded_vocab=pad)
    for k in out:
        assert bytes_equal(out[k], again[k]), k
    if mask:
        off = c["mask"] == 0
        for k in out:
            assert not host(out[k])[off].any(), k


@pytest.mark.parametrize("T", [3, 16, 17, 30, 32, 33, 48, 49, 64, 70])
def test_forward_int8_many_tiles_and_few_rows(llp, T):
    # 2344 vocabulary tiles: more than a few-row combine holds in LDS; masked rows among them.
    H, real, pad = 128, 600000, 600064
    g = np.random.default_rng(T)
    h = g.standard_normal((T, H)).astype(np.float32)
    hq, hs = O.quantize(h)
    wq = torch.randint(-127, 128, (pad, H), dtype=torch.int8, device="cuda",
                       generator=torch.Generator(device="cuda").manual_seed(T))
    ws = torch.rand(pad, device="cuda") * 1e-3
    mask = (np.arange(T) % 7 != 2).astype(np.uint8)
    tg = g.integers(0, real, T)
    out = llp.forward_int8(dev(hq), dev(hs), wq, ws, dev(tg), temperature=0.9, real_vocab=real,
                           padded_vocab=pad, loss_mask=dev(mask))
    z = O.int8_logits(hq, hs, host(wq), host(ws), None, 0.9, real)
    _close(out, O.score(z, tg, mask), z)


def test_forward_int8_extreme_values(llp):
    # Every product at its largest: sums of +-127 * 127 * 4096 (past 2^24) and -128 as stored.
    T, K, V = 5, 4096, 300
    hq = np.full((T, K), 127, np.int8)
    wq = np.full((V, K), 127, np.int8)
    wq[1::3] = -127
    wq[2::3] = -128
    hq[3] = -128
    hs, ws = np.full(T, 1e-3, np.float32), np.full(V, 5e-4, np.float32)
    tg = np.arange(T)
    out = llp.forward_int8(dev(hq), dev(hs), dev(wq), dev(ws), dev(tg), temperature=1.0)
    z = O.int8_logits(hq, hs, wq, ws, None, 1.0, V)
    _close(out, O.score(z, tg, None), z)


def test_forward_int8_shards_merge_and_empty_shard(llp):
    T, H, real, pad, tau = 70, 256, 1500, 2048, 0.7
    c = _case(T, H, real, pad, seed=5, bias="f32", mask_frac=0.2)
    d = _dev(c)
    z = O.int8_logits(c["hq"], c["hs"], c["wq"], c["ws"], c["b"].numpy(), tau, real)
    ref = O.score(z, c["tg"], c["mask"])
    parts, n = [], pad // 4
    for r in range(4):
        lo = r * n
        parts.append(llp.forward_int8(
            d["hq"], d["hs"], d["wq"][lo:lo + n], d["ws"][lo:lo + n], d["tg"], temperature=tau,
            bias=d["b"][lo:lo + n], loss_mask=d["mask"], offset=lo, real_vocab=real,
            padded_vocab=pad, rank=r, world=4))
        zs = z[:, lo:min(real, lo + n)] if lo < real else z[:, :0]
        _close(parts[-1], O.score(zs, c["tg"], c["mask"], offset=lo), z)
    mg = llp.merge(parts, loss_mask=d["mask"])
    tol = EPS * (16 * np.abs(z).max() + 200)
    for k in ("logp", "lse"):
        assert np.abs(host(mg[k]) - ref[k]).max() <= 2 * tol
    assert np.all(np.abs(host(mg["entropy"]) - ref["entropy"]) <= 2 * tol * (2 + ref["entropy"]))


def test_forward_int8_rows_do_not_depend_on_the_batch_bitwise(llp):
    T, H, real, pad = 600, 512, 3000, 3011
    c = _case(T, H, real, pad, seed=11, bias="bf16")
    d = _dev(c)
    kw = dict(temperature=0.7, bias=d["b"], real_vocab=real, padded_vocab=pad)
    whole = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], **kw)
    for rows in ([0], [599], list(range(5, 38)), list(range(100, 165)), list(range(200, 330)),
                 list(range(599, 0, -2))):
        i = torch.tensor(rows, device="cuda")
        part = llp.forward_int8(d["hq"][i], d["hs"][i], d["wq"], d["ws"], d["tg"][i], **kw)
        for k in part:
            assert bytes_equal(part[k], whole[k][i]), (k, len(rows))
    # the same rows as the scored ones of a masked batch
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[::29] = 1
    part = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], loss_mask=mask, **kw)
    for k in part:
        assert bytes_equal(part[k][::29], whole[k][::29]), k


def test_forward_int8_strides_status_and_no_rows(llp):
    T, H, real, pad = 40, 256, 600, 640
    c = _case(T, H, real, pad, seed=3)
    d = _dev(c)
    kw = dict(temperature=1.0, real_vocab=real, padded_vocab=pad)
    ref = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], **kw)
    wide_h = torch.full((T, H + 48), 99, dtype=torch.int8, device="cuda")
    wide_w = torch.full((pad, H + 16), -99, dtype=torch.int8, device="cuda")
    wide_h[:, :H], wide_w[:, :H] = d["hq"], d["wq"]
    got = llp.forward_int8(wide_h[:, :H], d["hs"], wide_w[:, :H], d["ws"], d["tg"], **kw)
    for k in ref:
        assert bytes_equal(ref[k], got[k]), k
    # padded columns are never read into a result
    ws = d["ws"].clone()
    ws[real:] = float("nan")
    wide_w[real:] = 127
    got = llp.forward_int8(wide_h[:, :H], d["hs"], wide_w[:, :H], ws, d["tg"], **kw)
    for k in ref:
        assert bytes_equal(ref[k], got[k]), k
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg = d["tg"].clone()
    tg[3], tg[5] = real, -1
    cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    bad = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], tg, status=st, cu_seqlens=cu, **kw)
    B = llp.STATUS_BITS
    assert int(st) == B["TARGET_OUT_OF_RANGE"] | B["TARGET_NOT_FOUND"] | B["LAYOUT_INVALID"]
    lp = host(bad["logp"])
    assert np.isneginf(lp[[3, 5]]).all() and np.isfinite(np.delete(lp, [3, 5])).all()
    none = llp.forward_int8(d["hq"][:0], d["hs"][:0], d["wq"], d["ws"], d["tg"][:0], **kw)
    assert none["logp"].shape == (0,)
    off = torch.zeros(T, dtype=torch.uint8, device="cuda")
    for k, v in llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], loss_mask=off, **kw).items():
        assert not host(v).any(), k


def test_int8_logp_stays_near_the_bf16_forward(llp):
    # Not a bound on quantisation in general: the same operands through both paths. Each product
    # is off by at most half a step of either operand, |dz| <= sum_k (|h| ws + |w| hs) / 2 + hs ws / 4.
    T, H, V = 64, 512, 4000
    g = np.random.default_rng(9)
    h = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((g.standard_normal((V, H)) * 0.02).astype(np.float32)).to(torch.bfloat16).cuda()
    tg = torch.from_numpy(g.integers(0, V, T)).cuda()
    hq, hs = llp.quantize_rows(h)
    wq, ws = llp.quantize_rows(w)
    a = llp.forward(h, w, tg, temperature=1.0)
    b = llp.forward_int8(hq, hs, wq, ws, tg, temperature=1.0)
    hd, wd, hsd, wsd = h.double().abs(), w.double().abs(), hs.double(), ws.double()
    lim = (hd.sum(1)[:, None] * wsd + wd.sum(1) * hsd[:, None]) / 2 + H * hsd[:, None] * wsd / 4
    err = (a["logp"].double() - b["logp"].double()).abs()
    assert bool((err <= 2 * lim.amax(1) + 1e-4).all())
