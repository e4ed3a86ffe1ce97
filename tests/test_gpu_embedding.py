"""Token embedding and its gradient: the lookup bitwise, the gradient within the rounding of its
fp32 sums, for every way ids can repeat; shards, masks, bad ids, accumulation, strides; the sum's
order fixed (bitwise repeats); the autograd node and the head's own dweight."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def _matrix(g, rows, H, dtype, ld=None):
    t = torch.from_numpy(g.standard_normal((rows, ld or H)).astype(np.float32)).to(DT[dtype])
    return t.cuda()[:, :H]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,H,ld", [(0, 5, 8, 8), (1, 1, 8, 8), (1, 900, 4096, 4096), (3, 50, 24, 32),
                                      (65, 300, 520, 528), (777, 1000, 256, 256), (2500, 40, 8200, 8200)])
def test_lookup_bitwise(llp, dtype, T, V, H, ld):
    say(f"embedding T={T} V={V} H={H} {dtype}")
    g = np.random.default_rng(T + H)
    w = _matrix(g, V, H, dtype, ld)
    ids = dev(g.integers(0, V, T))
    for scale in (1.0, 64.0, -0.3):
        out = llp.embedding_forward(ids, w, scale=scale)
        ref = (w.float().cpu()[ids.cpu()] * scale).to(DT[dtype])
        assert bytes_equal(out.cpu(), ref)


def test_lookup_shards_masks_and_bad_ids(llp):
    g = np.random.default_rng(4)
    T, H, real, pad = 300, 64, 150, 160
    w = _matrix(g, pad, H, "bf16")
    w[real:] = float("nan")                          # padding is never read
    ids = g.integers(0, real, T)
    mask = (g.random(T) < 0.8).astype(np.uint8)
    whole = llp.embedding_forward(dev(ids), w, token_mask=dev(mask), real_vocab=real)
    total = torch.zeros_like(whole)
    for r in range(4):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        total += llp.embedding_forward(dev(ids), w[40 * r:40 * r + 40], token_mask=dev(mask), offset=40 * r,
                                       real_vocab=real, padded_vocab=pad, rank=r, world=4, status=st)
        assert int(st) == 0
    assert torch.equal(total, whole) and not whole[dev(mask) == 0].any()
    bad = ids.copy()
    bad[[0, 7, 9, 11]] = [real, -1, 2 ** 40, -2 ** 62]
    mask[[0, 7, 9, 11]] = 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = llp.embedding_forward(dev(bad), w, token_mask=dev(mask), real_vocab=real, status=st)
    assert int(st) == llp.STATUS_BITS["TOKEN_OUT_OF_RANGE"]
    assert not out[[0, 7, 9, 11]].any()
    mask[[0, 7, 9, 11]] = 0
    st.zero_()
    llp.embedding_forward(dev(bad), w, token_mask=dev(mask), real_vocab=real, status=st)
    assert int(st) == 0
    # rows behind a strided output's width stay as they were
    buf = torch.full((T, H + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    llp.embedding_forward(dev(ids), w, real_vocab=real, out=buf[:, :H])
    assert bool((buf[:, H:] == 7).all())


def _check_grad(got, ids, dout, scale, n_real, V, offset=0, mask=None, old=None):
    """n terms summed in fp32 in any grouping, the scale and the addition to what was there:
    (n + 3) half steps of the magnitudes added up."""
    ref, n, size = O.embedding_grad(ids, dout.float().cpu().numpy(), scale, n_real, V, offset, mask)
    if old is not None:
        ref, size = ref + old, size + np.abs(old)
    err = np.abs(host(got).astype(np.float64) - ref)
    lim = EPS * (n + 3)[:, None] * size
    assert np.all(err <= lim), (err - lim).max()
    return n


IDS = {
    "distinct": lambda g, T, V: g.permutation(max(T, V))[:T] % V,
    "uniform": lambda g, T, V: g.integers(0, V, T),
    "skewed": lambda g, T, V: (np.exp(g.random(T) * np.log(V)).astype(np.int64) - 1),
    "one": lambda g, T, V: np.full(T, V - 1),
    "two": lambda g, T, V: np.where(np.arange(T) % 2, 0, V - 1),
    "runs": lambda g, T, V: (np.arange(T) // 37) % V,
}


@pytest.mark.parametrize("kind", sorted(IDS))
@pytest.mark.parametrize("T,V,H,dtype", [(1, 3, 8, "f32"), (31, 40, 64, "bf16"), (32, 7, 72, "bf16"),
                                         (33, 1000, 256, "bf16"), (65, 1, 16, "f32"),
                                         (1500, 300, 136, "f32"), (4099, 2500, 64, "bf16")])
def test_gradient(llp, kind, T, V, H, dtype):
    say(f"embedding grad {kind} T={T} V={V} H={H} {dtype}")
    g = np.random.default_rng(T * 3 + V)
    ids = IDS[kind](g, T, V).astype(np.int64)
    dout = _matrix(g, T, H, dtype)
    got = llp.embedding_backward(dev(ids), dout, local_size=V, scale=0.5, overwrite=True)
    n = _check_grad(got, ids, dout, 0.5, V, V)
    assert not host(got)[n == 0].any()
    again = llp.embedding_backward(dev(ids), dout, local_size=V, scale=0.5, overwrite=True)
    assert bytes_equal(got, again)
    # accumulated: rows without a token keep their bits
    old = torch.from_numpy(g.standard_normal((V, H)).astype(np.float32)).cuda()
    acc = llp.embedding_backward(dev(ids), dout, dweight=old.clone(), scale=0.5)
    _check_grad(acc, ids, dout, 0.5, V, V, old=old.double().cpu().numpy())
    keep = torch.from_numpy(n == 0).cuda()
    assert bytes_equal(acc[keep], old[keep])


@pytest.mark.parametrize("T,H,dtype,kind", [(9001, 64, "f32", "skewed"), (12500, 4104, "bf16", "uniform"),
                                            (33000, 4104, "bf16", "two"), (33000, 4104, "bf16", "skewed"),
                                            (17000, 1544, "f32", "one"), (8193, 8, "bf16", "runs")])
def test_gradient_of_large_batches(llp, T, H, dtype, kind):
    # Ids in a pass of their own, zeros in a launch of their own, rows read past the caches; a shard
    # in the middle of the table and rows of NaN where the mask is 0.
    say(f"embedding grad, large, {kind} T={T} H={H} {dtype}")
    g = np.random.default_rng(T + H)
    V, lo, nl = 5000, 1200, 2600
    ids = IDS[kind](g, T, V).astype(np.int64)
    if kind in ("one", "two"):
        ids = np.where(ids == V - 1, lo + nl - 1, lo)
    mask = (g.random(T) < 0.9).astype(np.uint8)
    dout = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).to(DT[dtype])
    dout[torch.from_numpy(mask == 0).cuda()] = float("nan")
    buf = torch.full((nl, H + 8), 5.0, device="cuda")
    kw = dict(token_mask=dev(mask), offset=lo, real_vocab=V, padded_vocab=V, rank=1, world=2, scale=0.7)
    got = llp.embedding_backward(dev(ids), dout, dweight=buf[:, :H], overwrite=True, **kw)
    for c in (slice(0, 8), slice(H // 2, H // 2 + 4), slice(H - 8, H)):
        part = torch.where(dev(mask)[:, None] != 0, dout[:, c].float(), 0.0)
        n = _check_grad(got[:, c], ids, part, 0.7, nl, nl, offset=lo, mask=mask)
    assert not got[torch.from_numpy(n == 0).cuda()].any() and bool((buf[:, H:] == 5).all())
    again = llp.embedding_backward(dev(ids), dout, local_size=nl, overwrite=True, **kw)
    assert bytes_equal(got.contiguous(), again)


def test_gradient_of_many_groups_and_rows_behind(llp):
    # More local rows than one sort group per compute unit holds, wide rows, strides.
    g = np.random.default_rng(8)
    T, V, H = 3000, 600000, 24
    ids = g.integers(0, V - 100, T)
    ids[::50] = V - 101
    dout = _matrix(g, T, H, "f32", H + 8)
    buf = torch.full((V + 1, H + 16), 3.0, device="cuda")
    got = llp.embedding_backward(dev(ids), dout, dweight=buf[:V, :H], real_vocab=V - 100, overwrite=True)
    u, inv = np.unique(ids, return_inverse=True)
    ref, n, size = O.embedding_grad(inv, dout.cpu().numpy(), 1.0, len(u), len(u))
    err = np.abs(host(got[torch.from_numpy(u).cuda()]) - ref)
    assert np.all(err <= EPS * (n + 3)[:, None] * size)
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(u).cuda()] = False
    assert not got[rest].any()
    assert bool((buf[:, H:] == 3).all()) and bool((buf[V] == 3).all())


def test_gradient_shards_masks_bad_ids_and_nothing(llp):
    g = np.random.default_rng(9)
    T, H, real, pad = 700, 40, 190, 200
    ids = g.integers(0, real, T)
    mask = (g.random(T) < 0.5).astype(np.uint8)
    dout = _matrix(g, T, H, "bf16")
    dout[torch.from_numpy(mask == 0).cuda()] = float("nan")        # masked rows are never read
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for r in range(4):
        lo = 50 * r
        got = llp.embedding_backward(dev(ids), dout, local_size=50, token_mask=dev(mask), offset=lo,
                                     real_vocab=real, padded_vocab=pad, rank=r, world=4, overwrite=True,
                                     status=st)
        clean = torch.where(dev(mask)[:, None] != 0, dout, torch.zeros_like(dout))
        _check_grad(got, ids, clean, 1.0, min(50, real - lo), 50, offset=lo, mask=mask)
    assert int(st) == 0
    bad = ids.copy()
    bad[mask == 1] = -5
    got = llp.embedding_backward(dev(bad), dout, local_size=pad, token_mask=dev(mask), real_vocab=real,
                                 overwrite=True, status=st)
    assert int(st) == llp.STATUS_BITS["TOKEN_OUT_OF_RANGE"] and not got.any()
    old = torch.randn(pad, H, device="cuda")
    got = llp.embedding_backward(dev(bad[:0]), dout[:0], dweight=old.clone())
    assert bytes_equal(got, old)
    got = llp.embedding_backward(dev(bad[:0]), dout[:0], dweight=old.clone(), overwrite=True)
    assert not got.any()
    # a shard of padding only still reports bad ids and writes its zeros
    st.zero_()
    got = llp.embedding_backward(dev(bad), dout, dweight=torch.ones(10, H, device="cuda"), token_mask=dev(mask),
                                 offset=190, real_vocab=real, padded_vocab=pad, rank=1, world=2,
                                 overwrite=True, status=st)
    assert int(st) == llp.STATUS_BITS["TOKEN_OUT_OF_RANGE"] and not got.any()


def test_autograd_node(llp):
    g = np.random.default_rng(10)
    V, H = 90, 64
    w = _matrix(g, V, H, "bf16").clone().requires_grad_(True)
    ids = dev(g.integers(0, V, (6, 7)))
    mask = torch.rand(6, 7, device="cuda") < 0.7
    out = llp.embedding(ids, w, scale=8.0, token_mask=mask)
    assert out.shape == (6, 7, H)
    up = torch.randn(6, 7, H, device="cuda", dtype=torch.bfloat16)
    (out * up).sum().backward()
    ref = llp.embedding_backward(ids.reshape(-1), up.reshape(-1, H), local_size=V, scale=8.0,
                                 token_mask=mask.reshape(-1).to(torch.uint8), overwrite=True)
    assert bytes_equal(w.grad, ref.to(torch.bfloat16))
    w.grad = None
    llp.embedding(ids, w).sum().backward()          # an expanded upstream gradient
    count = torch.bincount(ids.reshape(-1), minlength=V).float()
    assert torch.equal(w.grad.float(), count[:, None].expand(V, H).to(torch.bfloat16).float())
    w.grad = None
    x = llp.embedding(ids.reshape(-1)[:40], w)       # a transposed one
    (x.t() @ torch.ones(40, 3, device="cuda", dtype=torch.bfloat16)).sum().backward()
    assert bool((w.grad.float() == 3 * torch.bincount(ids.reshape(-1)[:40], minlength=V)[:, None].float()).all())
