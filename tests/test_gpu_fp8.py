"""Operands in 8-bit floating point against the fp64 oracle: quantised blocks exactly, products within
what their fp32 sums allow, an element's bits the same whatever the batch, gradients of the
autograd node against the formula."""
import numpy as np
import pytest
import torch

from oracle import gen as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24   # half a step of fp32


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def codes(q):
    return host(q.view(torch.uint8))


def same_scale(got, want):
    assert np.array_equal(host(got), want, equal_nan=True)


def wild(g, R, C):
    """Rows and columns of very different sizes."""
    return (g.standard_normal((R, C)) * 10.0 ** g.uniform(-5, 5, (R, 1)) * 10.0 ** g.uniform(-2, 2, (1, C))).astype(np.float32)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,C,dtype,ld", [
    (1, 1, "f32", 1), (3, 7, "bf16", 7), (5, 128, "bf16", 136), (129, 130, "f32", 131),
    (257, 320, "bf16", 320), (130, 1001, "bf16", 1003), (33, 264, "f32", 268), (128, 256, "bf16", 256)])
def test_quantize_blocks_exactly(llp, R, C, dtype, ld, transpose, rows):
    say(f"quantize_blocks R={R} C={C} {dtype} ld={ld} transpose={transpose} rows={rows}")
    g = np.random.default_rng(R * 10007 + C)
    x = torch.from_numpy(wild(g, R, ld))
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    if R > 2:
        x[1] = 0
    q, s = llp.quantize_blocks(x.cuda()[:, :C], rows=rows, transpose=transpose)
    rq, rs = O.quantize_blocks(x[:, :C].float().numpy(), rows, transpose)
    assert q.shape == rq.shape and s.shape == rs.shape and q.dtype == torch.float8_e4m3fn
    same_scale(s, rs)
    assert np.array_equal(codes(q), rq)


@pytest.mark.parametrize("R,C,dtype,ld", [
    (1, 1, "f32", 1), (3, 7, "bf16", 7), (129, 130, "f32", 131), (257, 320, "bf16", 320), (130, 1001, "bf16", 1003),
    (33, 264, "f32", 268), (300, 384, "bf16", 384), (0, 5, "f32", 5), (5, 0, "bf16", 0)])
def test_quantize_both_is_the_two_quantisations(llp, R, C, dtype, ld):
    say(f"quantize_both R={R} C={C} {dtype} ld={ld}")
    g = np.random.default_rng(R * 10007 + C)
    x = torch.from_numpy(wild(g, R, ld))
    x = (x.to(torch.bfloat16) if dtype == "bf16" else x).cuda()[:, :C]
    if R > 200:
        x[150, 140], x[3, 5], x[200] = float("nan"), float("inf"), 0
    q, s, qt, st = llp.quantize_both(x)
    want = (*llp.quantize_blocks(x), *llp.quantize_blocks(x, rows=128, transpose=True))
    for a, b in zip((q, s, qt, st), want):
        assert a.shape == b.shape and a.dtype == b.dtype
        assert a.numel() == 0 or np.array_equal(host(a.contiguous().view(torch.uint8)) if a.dtype == torch.float8_e4m3fn else host(a),
                                                host(b.contiguous().view(torch.uint8)) if a.dtype == torch.float8_e4m3fn else host(b),
                                                equal_nan=a.dtype == torch.float32)


def test_quantize_blocks_ties_and_odd_values(llp):
    # With 448 in a block its scale is fl(448 fl(1/448)) = 1: every midpoint of two e4m3 values, and its neighbours.
    mids = ((O.VALUES[1:] + O.VALUES[:-1]) / 2).astype(np.float32)
    x = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(500)),
                        O.VALUES.astype(np.float32), -mids, np.float32([0.0, -0.0])])
    blocks = [np.concatenate([x[i:i + 127], np.zeros(max(0, 127 - len(x[i:i + 127])), np.float32), [np.float32(448)]])
              for i in range(0, len(x), 127)]
    x = np.stack(blocks).astype(np.float32)
    q, s = llp.quantize_blocks(dev(x))
    rq, rs = O.quantize_blocks(x)
    assert (rs == 1).all()
    same_scale(s, rs)
    assert np.array_equal(codes(q), rq)
    assert np.array_equal(codes(q), host(dev(x).to(torch.float8_e4m3fn).view(torch.uint8)))
    # Quotients next to ties: every bf16 value of two binades over many scales.
    bits = np.arange(0x3F80, 0x4080, dtype=np.uint16)
    vals = (bits.astype(np.uint32) << 16).view(np.float32)
    rows = np.stack([np.concatenate([vals[:127], [m], vals[127:254], [m]]) for m in
                     np.linspace(4.0, 900.0, 301, dtype=np.float32)]).astype(np.float32)
    q, s = llp.quantize_blocks(dev(rows))
    rq, rs = O.quantize_blocks(rows)
    same_scale(s, rs)
    assert np.array_equal(codes(q), rq)
    bad = np.ones((130, 300), np.float32)
    bad[0, 3], bad[1, 299], bad[129, 0] = np.nan, np.inf, -np.inf
    bad[3], bad[4] = 1e-38, 3e38
    for rows in (1, 128):
        for tr in (False, True):
            q, s = llp.quantize_blocks(dev(bad), rows=rows, transpose=tr)
            rq, rs = O.quantize_blocks(bad, rows, tr)
            same_scale(s, rs)
            assert np.array_equal(codes(q), rq)


@pytest.mark.parametrize("R,C", [(0, 64), (7, 0), (0, 0)])
def test_quantize_blocks_of_nothing(llp, R, C):
    for rows in (1, 128):
        for tr in (False, True):
            q, s = llp.quantize_blocks(torch.empty((R, C), device="cuda"), rows=rows, transpose=tr)
            M, K = (C, R) if tr else (R, C)
            G = -(-K // 128)
            assert q.shape == (M, G * 128) and s.shape == (-(-M // rows), G)


def operands(llp, T, V, K, seed):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((T, K)) * np.exp(g.standard_normal((1, K)))).astype(np.float32)
    w = (g.standard_normal((V, K)) * 0.02).astype(np.float32)
    xq, xs = llp.quantize_blocks(dev(x))
    wq, ws = llp.quantize_blocks(dev(w), rows=128)
    xv = O.values(*O.quantize_blocks(x), 1)
    wv = O.values(*O.quantize_blocks(w, 128), 128)
    return xq, xs, wq, ws, xv, wv


def within(y, ref, size, K, step=EPS):
    """Into fp32 a group's 128 products are summed with at most one rounding each (2^-23, in case the
    matrix cores truncate), then scaled and added: 2 more of 2^-24 a group and the scales' product.
    `step` is half a step of the output's type; into bf16 the 8-bit matrix instructions sum instead,
    which cut each of 8 products towards zero at 2^-13 of the largest one's power of two (exponents of
    its factors): 7 such cuts, beside the largest itself, of at most the sum of 8 products' sizes."""
    G = -(-K // 128)
    slack = size * EPS * (2 * 128 + 2 * G + 4)
    if y.dtype == torch.bfloat16:
        slack += size * 7 * 2.0 ** -13
    bound = slack + (np.abs(ref) + slack) * step
    err = np.abs(host(y.float()).astype(np.float64) - ref)
    assert err.shape == bound.shape
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    assert (err <= bound).all(), f"{worst:.3g} of the bound"
    # The cuts are far apart in sign and place: over many elements they stay below 2^-13 of the norm.
    if y.dtype == torch.bfloat16 and err.size >= 1000:
        assert np.linalg.norm(err) <= (2.0 ** -8 + 2.0 ** -13) * np.linalg.norm(ref)


@pytest.mark.parametrize("T,V,K", [
    (1, 1, 1), (1, 1000, 640), (2, 129, 100), (31, 257, 130), (32, 128, 128), (33, 127, 4096),
    (64, 300, 1000), (65, 513, 256), (128, 260, 384), (129, 128, 512), (300, 600, 320),
    (513, 700, 640), (600, 257, 8320), (777, 1030, 128)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_fp8(llp, T, V, K, out):
    say(f"linear_fp8 T={T} V={V} K={K} {out}")
    xq, xs, wq, ws, xv, wv = operands(llp, T, V, K, T * 31 + V)
    g = np.random.default_rng(V)
    for bias in (None, "f32", "bf16"):
        b = bd = None
        if bias:
            bd = torch.from_numpy(g.standard_normal(V).astype(np.float32)).cuda()
            bd = bd.to(torch.bfloat16) if bias == "bf16" else bd
            b = host(bd.float()).astype(np.float64)
        y = llp.linear_fp8(xq, xs, wq, ws, bias=bd, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
        assert y.shape == (T, V)
        ref, size = O.linear(xv, wv, b)
        within(y, ref, size, K, EPS if out == "f32" else 2.0 ** -8)


def test_linear_fp8_rows_have_the_same_bits_in_any_batch(llp):
    # The tile changes with the number of rows (1 .. 32, .. 64, .. 512, beyond): the bits do not.
    T, V, K = 700, 517, 640
    xq, xs, wq, ws, _, _ = operands(llp, T, V, K, 5)
    for d in (torch.float32, torch.bfloat16):
        whole = llp.linear_fp8(xq, xs, wq, ws, out_dtype=d)
        for n in (1, 31, 32, 33, 64, 65, 128, 300, 512, 513):
            for at in (0, 37, T - n):
                part = llp.linear_fp8(xq[at:at + n], xs[at:at + n], wq, ws, out_dtype=d)
                assert bytes_equal(part, whole[at:at + n]), (n, at)
        again = llp.linear_fp8(xq, xs, wq, ws, out_dtype=d)
        assert bytes_equal(whole, again)


def test_linear_fp8_strides_and_rows_around_the_output(llp):
    T, V, K = 70, 201, 256
    xq, xs, wq, ws, _, _ = operands(llp, T, V, K, 6)
    wants = {d: llp.linear_fp8(xq, xs, wq, ws, out_dtype=d) for d in (torch.float32, torch.bfloat16)}
    want = wants[torch.float32]
    wide = torch.zeros((T, 2 * K), dtype=torch.uint8, device="cuda").fill_(0x7F).view(torch.float8_e4m3fn)
    wide[:, K:] = xq
    tall = torch.zeros((V, K + 48), dtype=torch.uint8, device="cuda").fill_(0x7F).view(torch.float8_e4m3fn)
    tall[:, 16:16 + K] = wq
    scales = torch.full((2, T + 5), float("nan"), device="cuda")
    scales[:, 3:3 + T] = xs.t()
    wscales = torch.full((2, 9), float("nan"), device="cuda")
    wscales[:, :2] = ws
    for dt, pad in ((torch.float32, 0), (torch.float32, 3), (torch.bfloat16, 1), (torch.bfloat16, 8)):
        room = torch.full((T + 2, V + pad), 7.0, dtype=dt, device="cuda")
        y = llp.linear_fp8(wide[:, K:], scales[:, 3:3 + T].t(), tall[:, 16:16 + K], wscales[:, :2],
                           out=room[1:T + 1, :V])
        assert torch.equal(y, wants[dt])
        assert (room[0] == 7).all() and (room[T + 1] == 7).all() and (room[:, V:] == 7).all()
    # Values that are not finite stay in their row (x) and in their block of 128 columns (weight).
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[3, 1] = float("nan")
    ws2[1, 0] = float("nan")
    y = llp.linear_fp8(xq, xs2.t().contiguous().t(), wq, ws2, out_dtype=torch.float32)
    bad = torch.zeros((T, V), dtype=torch.bool, device="cuda")
    bad[3] = True
    bad[:, 128:] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("V,H,T", [(1, 1, 1), (129, 257, 100), (300, 64, 130), (256, 256, 128), (517, 700, 1000),
                                   (128, 128, 0)])
def test_dweight_fp8(llp, V, H, T):
    say(f"dweight_fp8 V={V} H={H} T={T}")
    g = np.random.default_rng(V + T)
    dy = (g.standard_normal((T, V)) * np.exp(g.standard_normal((T, 1)))).astype(np.float32)
    x = g.standard_normal((T, H)).astype(np.float32)
    a = (*llp.quantize_blocks(dev(dy), rows=128, transpose=True), *llp.quantize_blocks(dev(x), transpose=True))
    gv = O.values(*O.quantize_blocks(dy, 128, True), 128)
    xv = O.values(*O.quantize_blocks(x, 1, True), 1)
    ref, size = O.linear(gv, xv)
    within(llp.dweight_fp8(*a), ref, size, max(T, 1))
    within(llp.dweight_fp8(*a, out_dtype=torch.bfloat16), ref, size, max(T, 1), 2.0 ** -8)
    start = g.standard_normal((V, H)).astype(np.float32)
    room = torch.full((V + 2, H + 3), 7.0, device="cuda")
    room[1:V + 1, :H] = dev(start)
    got = llp.dweight_fp8(*a, dweight=room[1:V + 1, :H])
    within(got, ref + start, size + np.abs(start), max(T, 1), EPS)
    assert (room[0] == 7).all() and (room[V + 1] == 7).all() and (room[:, H:] == 7).all()
    full = llp.dweight_fp8(*a)
    over = llp.dweight_fp8(*a, dweight=room[1:V + 1, :H], overwrite=True)
    assert torch.equal(over, full)
    room = torch.full((V + 2, H + 1), 7.0, device="cuda", dtype=torch.bfloat16)
    over = llp.dweight_fp8(*a, dweight=room[1:V + 1, :H], overwrite=True)
    assert torch.equal(over, llp.dweight_fp8(*a, out_dtype=torch.bfloat16))
    assert (room[0] == 7).all() and (room[V + 1] == 7).all() and (room[:, H:] == 7).all()


def test_products_without_rows_or_depth(llp):
    xq, xs, wq, ws, _, _ = operands(llp, 5, 7, 128, 1)
    e = torch.empty
    f8 = torch.float8_e4m3fn
    b = torch.arange(7, device="cuda", dtype=torch.float32)
    none = llp.linear_fp8(xq[:0], xs[:0], wq, ws)
    assert none.shape == (0, 7)
    assert llp.linear_fp8(xq, xs, wq[:0], ws[:0]).shape == (5, 0)
    y = llp.linear_fp8(e((5, 0), dtype=f8, device="cuda"), e((5, 0), device="cuda"), e((7, 0), dtype=f8, device="cuda"),
                       e((1, 0), device="cuda"), bias=b, out_dtype=torch.float32)
    assert torch.equal(y, b.expand(5, 7))


@pytest.mark.parametrize("T,K,V,dtype", [(1, 64, 40, "bf16"), (70, 200, 333, "f32"), (140, 256, 512, "bf16")])
def test_fp8_linear_gradients(llp, T, K, V, dtype):
    g = np.random.default_rng(T)
    d = torch.bfloat16 if dtype == "bf16" else torch.float32
    step = 2.0 ** -8 if dtype == "bf16" else EPS
    x = torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)).to(d)
    w = torch.from_numpy((g.standard_normal((V, K)) * 0.1).astype(np.float32)).to(d)
    dy = torch.from_numpy(g.standard_normal((T, V)).astype(np.float32)).to(d)
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = llp.fp8_linear(xd, wd)
    assert y.dtype == d and y.shape == (T, V)
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.cuda())
    xn, wn, gn = x.float().numpy(), w.float().numpy(), dy.float().numpy()
    qx, qw = O.values(*O.quantize_blocks(xn), 1)[:, :K], O.values(*O.quantize_blocks(wn, 128), 128)[:, :K]
    ref, size = O.linear(qx, qw)
    within(y.detach(), ref, size, K, step)
    qg = O.values(*O.quantize_blocks(gn), 1)[:, :V]
    ref, size = O.linear(qg, qw.T)
    within(dx, ref, size, V, step)
    gt = O.values(*O.quantize_blocks(gn, 128, True), 128)[:, :T]
    xt = O.values(*O.quantize_blocks(xn, 1, True), 1)[:, :T]
    ref, size = O.linear(gt, xt)
    within(dw, ref, size, T, step)
    assert dx.dtype == d and dw.dtype == d and dx.shape == x.shape and dw.shape == w.shape
    # Leading dims, an expanded upstream gradient, one input that needs none.
    y3 = llp.fp8_linear(xd.reshape(1, T, K), wd)
    assert torch.equal(y3[0], y)
    s, = torch.autograd.grad(y3.sum(), (wd,))
    ones = np.ones((T, V), np.float32)
    ref, size = O.linear(O.values(*O.quantize_blocks(ones, 128, True), 128)[:, :T], xt)
    within(s, ref, size, T, step)
    yt = llp.fp8_linear(x.cuda(), wd)
    assert torch.equal(yt, y)
    yt.backward(dy.cuda())
    assert torch.equal(wd.grad, dw)


def test_fp8_linear_gradient_against_differences(llp):
    # Where every operand is an e4m3 value times its block's scale already (whole numbers up to 15 with
    # one of 448 / 2^5 = 14 in the block's place to fix the scale at 2^-5), the products are those of
    # the operands themselves, and a loss's differences are its gradient.
    g = np.random.default_rng(3)
    T, K, V = 128, 128, 128
    x, w, c = (g.integers(-7, 8, s).astype(np.float32) * 2 for s in ((T, K), (V, K), (T, V)))
    for m in (x, w, c):
        m[:, 0] = 14
        m[0, :] = 14
    xd, wd = dev(x).requires_grad_(), dev(w).requires_grad_()
    dx, dw = torch.autograd.grad(llp.fp8_linear(xd, wd), (xd, wd), dev(c))
    f = lambda a, b: float((c.astype(np.float64) * (a.astype(np.float64) @ b.astype(np.float64).T)).sum())  # noqa: E731
    for i, j in ((1, 1), (5, 99), (127, 64)):
        for m, grad in ((x, dx), (w, dw)):
            lo, hi = m.copy(), m.copy()
            lo[i, j] -= 1
            hi[i, j] += 1
            diff = (f(hi, w) - f(lo, w)) / 2 if m is x else (f(x, hi) - f(x, lo)) / 2
            assert float(grad[i, j]) == diff   # whole numbers below 2^24


def quantised(llp, R, K, rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, K, generator=g, device="cuda") * torch.exp(torch.randn(R, 1, generator=g, device="cuda"))
    return llp.quantize_blocks(x, rows=rows)


# Each reaches another shape of workgroup; columns past several turns of the groups' order, ragged ends.
@pytest.mark.parametrize("T,V", [(65, 203), (130, 16389), (644, 10802), (258, 21804), (65, 32830), (130, 32900), (193, 33012),
                                 (259, 32795), (196, 20535), (386, 16432), (387, 21949), (130, 20681), (321, 21856), (65, 16411),
                                 (1, 70003), (33, 66001)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_products_have_the_same_bits_in_every_form(llp, T, V, out):
    K = 384
    say(f"forms T={T} V={V} K={K} {out}")
    x, w = quantised(llp, T, K, 1, T), quantised(llp, V, K, 128, V)
    d = torch.bfloat16 if out == "bf16" else torch.float32
    y = llp.linear_fp8(*x, *w, out_dtype=d)
    # Few rows, few columns: the groups' order repeats after 1280 * 3 columns.
    for v in range(0, V, 3840 * 4):
        part = w[0][v:v + 15360], w[1][v // 128:(min(v + 15360, V) + 127) // 128]
        few = torch.cat([llp.linear_fp8(x[0][t:t + 32], x[1][t:t + 32], *part, out_dtype=d) for t in range(0, T, 32)])
        assert bytes_equal(y[:, v:v + 15360].contiguous(), few.contiguous())
    dw = llp.dweight_fp8(*w, *x, out_dtype=d)
    assert torch.equal(dw, y.t())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_blocks_of_many_groups(llp, dtype):
    # From 2^19 groups on four rows go together: the same bytes as a few rows at a time.
    R, C = 131075, 500
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(R, C, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    q, s = llp.quantize_blocks(x)
    for r in (0, 65530, R - 1001):
        rq, rs = llp.quantize_blocks(x[r:r + 1001])
        assert bytes_equal(q[r:r + 1001].view(torch.uint8), rq.view(torch.uint8))
        assert bytes_equal(s[r:r + 1001].contiguous(), rs.contiguous())
