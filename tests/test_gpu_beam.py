"""A beam search's step against the fp64 oracle: candidates and selections exactly, normalisers and scores
within their roundings, masked and broken rows, shards, ties, and the reordering of states."""
import math

import numpy as np
import pytest
import torch

from oracle import gen as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def rows16(x, dtype):
    """A device copy whose rows are 16-byte aligned, NaN behind them."""
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    room = torch.full((x.shape[0], x.shape[1] + -x.shape[1] % 8 + 8), math.nan, dtype=dtype)
    room[:, :x.shape[1]] = t
    return room.cuda()[:, :x.shape[1]]


def check_candidates(got, x, num, tau, offset=0, n_real=None):
    """x: the logits' own values. A term of the sum: the exponential's rounding (about 2^-23), the
    rounding of x - max (2^-24 of up to ~30 log 2 where a term still counts) made up for to first order
    in t alone: 2^-24 |x - max| c, and fp32 sums of 32 values and of 64 lanes (38 roundings)."""
    c = float(np.float32(1.0 / np.float32(tau).astype(np.float64)))
    value, token, top, total = O.beam_candidates(x, num, c, offset, n_real)
    assert np.array_equal(host(got["token"]), token)
    assert np.array_equal(host(got["value"]).astype(np.float64), value)
    assert np.array_equal(host(got["max"]).astype(np.float64), top)
    s = host(got["sum"])
    assert (np.abs(s - total) <= np.maximum(total, 0) * 2.0 ** -24 * (2 + 40 + 38)).all()
    assert np.array_equal(s < 0, total < 0)
    return c


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,num", [(1, 1, 1), (1, 3, 8), (2, 63, 64), (3, 2047, 5), (4, 2048, 64), (2, 2049, 16),
                                     (7, 5000, 1), (5, 9001, 33), (300, 4100, 8), (4200, 300, 4), (1, 60000, 64)])
def test_beam_candidates(llp, R, V, num, dtype):
    say(f"beam_candidates R={R} V={V} num={num} {dtype}")
    g = np.random.default_rng(R * 31 + V)
    x = g.standard_normal((min(R, 300), V)) * 3
    x = np.concatenate([x] * (-(-R // len(x))))[:R]
    z = rows16(x, dtype)
    for tau in (1.0, 0.7):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = llp.beam_candidates(z, num, temperature=tau, status=st)
        if R <= 300:
            check_candidates(got, host(z.float()), num, tau)
        else:
            check_candidates({k: v[:300] for k, v in got.items()}, host(z[:300].float()), num, tau)
            for k, v in got.items():   # equal rows have equal bits
                assert bytes_equal(v[:300], v[300:600]) and bytes_equal(v[:300], v[3900:4200]), k
        assert int(st) == 0


def test_beam_candidates_bits_do_not_depend_on_the_batch(llp):
    g = np.random.default_rng(2)
    z = rows16(g.standard_normal((600, 21000)) * 4, torch.float32)
    whole = llp.beam_candidates(z, 16)
    for a, b in ((0, 1), (5, 9), (100, 300), (599, 600)):
        part = llp.beam_candidates(z[a:b], 16)
        for k in part:
            assert bytes_equal(part[k], whole[k][a:b]), k


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "lane by lane", "huge", "zeros of both signs"])
def test_beam_candidates_where_the_bar_is_hard_to_find(llp, kind):
    V, num = 6500, 64
    n = np.arange(V)
    x = dict(equal=np.full(V, -3.5), rising=n * 0.01, falling=-n * 0.01)
    x["two values"] = (n * 7919 % 13 == 0) * 1.0
    x["lane by lane"] = (n // 4 % 64 < 8) * 10.0 + n % 4
    x["huge"] = np.where(n % 5 == 0, np.finfo(np.float32).max, np.finfo(np.float32).min)
    x["zeros of both signs"] = np.where(n % 3 == 0, 0.0, -0.0)
    z = rows16(np.stack([x[kind], x[kind][::-1]]), torch.float32)
    check_candidates(llp.beam_candidates(z, num), host(z), num, 1.0)


def test_beam_candidates_of_masked_and_broken_rows(llp):
    g = np.random.default_rng(4)
    x = g.standard_normal((9, 4500)).astype(np.float32)
    lowest = np.finfo(np.float32).min
    x[0] = -np.inf                                   # a mask that leaves nothing
    x[1] = -np.inf
    x[1, [7, 4444]] = 1.0, 1.0                       # and two
    x[2] = lowest                                    # masked by the type's lowest value: even
    x[3, ::2] = lowest
    x[4, 4499] = np.nan
    x[5, 0] = np.inf
    x[6, 100] = -np.inf
    x[7, 2048:] = -np.inf                            # whole blocks
    z = rows16(x, torch.float32)
    for tau in (1.0, 0.5):                           # 0.5: the lowest value overflows fp32
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        check_candidates(llp.beam_candidates(z, 10, temperature=tau, status=st), x, 10, tau)
        assert int(st) == llp.STATUS_BITS["VALUE_NOT_FINITE"]
    # Padding may hold anything, and a shard may be padding only, or empty.
    x[:, 4000:] = np.nan
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = rows16(x, torch.float32)
    got = llp.beam_candidates(z[6:8], 10, real_vocab=4000, status=st)
    check_candidates(got, x[6:8], 10, 1.0, n_real=4000)
    got = llp.beam_candidates(z[6:8, 4000:], 10, offset=4000, real_vocab=4000, padded_vocab=4500, world=2, rank=1, status=st)
    assert int(st) == 0
    for k, v in dict(token=-1, value=-math.inf, max=-math.inf, sum=0).items():
        assert (got[k] == v).all(), k
    got = llp.beam_candidates(z[:, :0], 3, offset=0, real_vocab=4000, padded_vocab=4500, world=2, status=st)
    assert (got["token"] == -1).all() and (got["sum"] == 0).all()
    assert llp.beam_candidates(z[:0], 3, real_vocab=4000)["token"].shape == (0, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_candidates_find_what_is_not_finite_anywhere(llp, dtype):
    # 2 whole blocks of 2048 and 13 columns, of which the last few are no whole 16 bytes.
    V = 4109
    g = np.random.default_rng(11)
    good = g.standard_normal((1, V)).astype(np.float32)
    bad = []
    for at, what in ((0, np.nan), (2047, np.nan), (2048, np.inf), (4095, np.nan), (4096, np.nan), (4103, np.inf), (V - 1, np.nan),
                     (V - 1, np.inf), (slice(0, 2048), np.nan), (slice(2048, 4096), np.inf), (slice(4096, V), np.nan),
                     (slice(0, V), np.nan), (slice(0, V), np.inf)):
        x = good.copy()
        x[0, at] = what
        bad.append(x)
        y = np.full((1, V), -np.inf, np.float32)   # the only value that is no mask
        y[0, at] = what
        bad.append(y)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = llp.beam_candidates(rows16(np.concatenate([good, *bad, good]), dtype), 5, status=st)
    assert int(st) == llp.STATUS_BITS["VALUE_NOT_FINITE"]
    s = host(got["sum"])
    assert (s[1:-1] == -1).all() and s[0] > 0 and s[-1] == s[0]
    assert (host(got["token"])[1:-1] == -1).all() and (host(got["value"])[1:-1] == -np.inf).all()
    assert (host(got["token"])[[0, -1]] >= 0).all() and (host(got["max"])[1:-1] == -np.inf).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beam_candidates_of_the_widest_shard(llp, dtype):
    V = 1 << 21
    say(f"beam_candidates V={V} {dtype}")
    x = np.random.default_rng(12).standard_normal((1, V)) * 2
    z = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    got = llp.beam_candidates(z, 64)
    check_candidates(got, host(z.float()), 64, 1.0)
    # Equal values everywhere: every piece reaches the bar, the first columns win.
    z.fill_(1.5)
    check_candidates(llp.beam_candidates(z, 64), host(z.float()), 64, 1.0)


def test_beam_select_takes_no_token_that_is_none(llp):
    # Ids that no vocabulary holds, as a caller's own candidates might have them.
    part = dict(value=torch.tensor([[3.0, 2.0, 1.0, 0.0]], device="cuda"),
                token=torch.tensor([[1 << 40, 5, -7, 1 << 62]], device="cuda"),
                max=torch.tensor([3.0], device="cuda"), sum=torch.tensor([2.0], dtype=torch.float64, device="cuda"))
    got = llp.beam_select([part], torch.zeros(1, 1, device="cuda"), 4)
    assert host(got["token"]).tolist() == [[5, -1, -1, -1]] and host(got["parent"]).tolist() == [[0, -1, -1, -1]]


def step(llp, z, B, K, num, tau, scores, shards, real, finished=None, end=None, status=None):
    pad = z.shape[1]
    cuts = [min(pad, i * (-(-pad // shards) + 8) // 8 * 8) for i in range(shards)] + [pad]
    parts = []
    for r in range(shards):
        a, b = cuts[r], cuts[r + 1]
        parts.append(llp.beam_candidates(z[:, a:b], num, temperature=tau, offset=a, real_vocab=real, padded_vocab=pad,
                                         rank=r, world=shards, status=status))
    return llp.beam_select(parts, scores, num, temperature=tau, finished=finished, end_id=end, status=status)


@pytest.mark.parametrize("B,K,num,V,shards,dtype", [
    (1, 1, 1, 7, 1, torch.float32), (1, 4, 8, 5000, 1, torch.float32), (3, 5, 10, 4111, 4, torch.bfloat16),
    (2, 64, 64, 300, 1, torch.float32), (5, 3, 64, 50, 2, torch.float32), (40, 2, 4, 2500, 3, torch.bfloat16),
    (2, 16, 32, 2049, 8, torch.float32), (1, 2, 60, 20, 1, torch.float32)])
def test_beam_select(llp, B, K, num, V, shards, dtype):
    say(f"beam_select B={B} K={K} num={num} V={V} shards={shards}")
    g = np.random.default_rng(B * 1000 + K)
    x = g.standard_normal((B * K, V + 13)) * 3
    x[:, V:] = 50                                    # padding
    z = rows16(x, dtype)
    scores = (-g.uniform(0, 8, (B, K))).astype(np.float32)
    if K > 2:
        scores[0, 1] = -np.inf
    done = (g.uniform(size=(B, K)) < 0.3).astype(np.uint8)
    for tau, finished in ((1.0, None), (0.7, done)):
        c = float(np.float32(1.0 / np.float32(tau).astype(np.float64)))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = step(llp, z, B, K, num, tau, dev(scores), shards, V, None if finished is None else dev(finished), 2, st)
        token, parent, score = O.beam_select(host(z.float())[:, :V].reshape(B, K, V), scores, num, c, finished, 2)
        assert np.array_equal(host(got["parent"]), parent)
        assert np.array_equal(host(got["token"]), token)
        s = host(got["score"]).astype(np.float64)
        fin = np.isfinite(score)
        assert np.array_equal(np.isfinite(s), fin) and (s[~fin] == -np.inf).all()
        # The log of a sum that is off by 80 half steps of fp32 (check_candidates), one rounding.
        assert (np.abs(s[fin] - score[fin]) <= 2.0 ** -24 * (80 + np.abs(score[fin]))).all()
        assert int(st) == 0


def test_beam_select_ties_and_what_is_not_there(llp):
    # Equal beams: bits decide nothing, the lowest beam and token come first.
    x = np.tile(np.float32([1, 5, 5, 2, 5, 0, -1, 3]), (6, 1))
    z = rows16(x, torch.float32)
    got = step(llp, z, 2, 3, 5, 1.0, torch.zeros((2, 3), device="cuda"), 1, 8)
    assert host(got["token"]).tolist() == [[1, 2, 4, 1, 2]] * 2
    assert host(got["parent"]).tolist() == [[0, 0, 0, 1, 1]] * 2
    # A finished beam ties with another finished one; their tokens are the caller's.
    done = torch.ones((2, 3), dtype=torch.uint8, device="cuda")
    got = step(llp, z, 2, 3, 5, 1.0, torch.full((2, 3), -2.0, device="cuda"), 1, 8, done, -7)
    assert host(got["parent"]).tolist() == [[0, 1, 2, -1, -1]] * 2
    assert host(got["token"]).tolist() == [[-7, -7, -7, -1, -1]] * 2
    assert host(got["score"]).tolist() == [[-2.0, -2.0, -2.0, -math.inf, -math.inf]] * 2
    # The first step: one beam is there.
    s = torch.tensor([[0.0, -math.inf, -math.inf], [-math.inf, 0.0, -math.inf]], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = step(llp, z, 2, 3, 3, 1.0, s, 2, 8, status=st)
    assert host(got["parent"]).tolist() == [[0, 0, 0], [1, 1, 1]] and int(st) == 0
    # A broken score or row takes its beam out; a masked row has nothing to offer.
    s = torch.tensor([[0.0, math.nan, 0.0], [0.0, 0.0, math.inf]], device="cuda")
    x[0, 3] = np.nan
    x[3] = -np.inf
    z = rows16(x, torch.float32)
    got = step(llp, z, 2, 3, 2, 1.0, s, 2, 8, status=st)
    assert host(got["parent"]).tolist() == [[2, 2], [1, 1]] and int(st) == llp.STATUS_BITS["VALUE_NOT_FINITE"]
    # Nobody left.
    got = step(llp, z, 2, 3, 2, 1.0, torch.full((2, 3), -math.inf, device="cuda"), 1, 8)
    assert (got["parent"] == -1).all() and (got["token"] == -1).all() and (got["score"] == -math.inf).all()


def test_beam_select_of_rows_at_the_lowest_value(llp):
    # Every logit of a beam at the type's lowest value is a uniform distribution over it.
    x = np.full((2, 40), np.finfo(np.float32).min, np.float32)
    x[1] = 0
    z = rows16(x, torch.float32)
    got = step(llp, z, 1, 2, 3, 0.5, torch.tensor([[0.0, -1.0]], device="cuda"), 2, 40)
    assert host(got["parent"]).tolist() == [[0, 0, 0]] and host(got["token"]).tolist() == [[0, 1, 2]]
    assert np.allclose(host(got["score"]), -math.log(40), rtol=1e-6, atol=0)


DTYPES = [torch.bfloat16, torch.float32, torch.uint8, torch.int64, torch.float8_e4m3fn]


@pytest.mark.parametrize("B,K,shape", [(1, 1, (3,)), (1, 2, ()), (2, 4, (5, 7, 16)), (3, 5, (2, 9, 3)), (1, 8, (1, 33, 128)),
                                       (2, 16, (4, 10, 64)), (2, 17, (3, 2, 8)), (1, 33, (2, 5, 40)), (2, 64, (2, 3, 24))])
def test_beam_reorder_in_place(llp, B, K, shape):
    g = np.random.default_rng(B * 100 + K)
    parents = g.integers(-1, K, (B, K)).astype(np.int32)
    for dt in DTYPES:
        x = torch.from_numpy(g.integers(0, 100, (B * K, *shape))).to(torch.float32).to(dt)
        raw = x.view(torch.uint8) if dt == torch.float8_e4m3fn else x
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        d = x.cuda()
        assert llp.beam_reorder(d, dev(parents), status=st) is d
        rows = torch.from_numpy(np.arange(B * K).reshape(B, K))
        take = torch.where(dev(parents).cpu() >= 0, dev(parents).cpu() + torch.arange(B)[:, None] * K, rows).reshape(-1)
        got = d.view(torch.uint8) if dt == torch.float8_e4m3fn else d
        assert torch.equal(got.cpu(), raw[take]) and int(st) == 0, dt
        # A view: the last but one dim cut, what lies behind the cut untouched.
        if len(shape) == 3:
            room = torch.zeros((B * K, shape[0], shape[1] + 3, shape[2]), dtype=torch.uint8).fill_(9)
            room[:, :, :shape[1]] = x.to(torch.float32).to(torch.uint8)
            dr = room.cuda()
            llp.beam_reorder([dr[:, :, :shape[1]]], dev(parents))
            assert torch.equal(dr[:, :, :shape[1]].cpu(), room[:, :, :shape[1]][take])
            assert (dr[:, :, shape[1]:] == 9).all()


def test_beam_reorder_many_states_and_layouts(llp):
    g = np.random.default_rng(8)
    B, K = 2, 4
    parents = g.integers(0, K, (B, K)).astype(np.int32)
    take = torch.from_numpy((parents + np.arange(B)[:, None] * K).reshape(-1)).cuda()

    def r(*s):
        return torch.from_numpy(g.standard_normal(s).astype(np.float32)).cuda()

    kv = r(B * K, 2, 3, 10, 16)                       # keys and values side by side
    heads_first = r(3, B * K, 10, 16)                 # rows within heads
    states = [r(B * K, 5, 64) for _ in range(70)]     # more than one launch takes
    states += [kv[:, 0], kv[:, 1], kv[:, 0, :, :7][:, :, :0], heads_first.transpose(0, 1), r(B * K), r(B * K, 3).t()[1],
               r(B * K, 12)[:, ::3]]
    want = [s[take] for s in states]
    llp.beam_reorder(states, dev(parents))
    for i, (s, w) in enumerate(zip(states, want)):
        assert torch.equal(s, w), i
    # Into other tensors: K beams become N, one prompt row many beams, rows expanded.
    prompt = r(B, 6, 8)
    out = [torch.full((B * 5, 6, 8), 7.0, device="cuda")]
    p = torch.tensor([[0, 0, -1, 0, 0], [0, 0, 0, 0, -1]], dtype=torch.int32, device="cuda")
    assert llp.beam_reorder([prompt], p, out=out) is out
    w = prompt.repeat_interleave(5, dim=0)
    w[2], w[9] = 7.0, 7.0
    assert torch.equal(out[0], w)
    one = r(1, 6, 8).expand(B * K, 6, 8)
    o = torch.zeros((B * K, 6, 8), device="cuda")
    assert torch.equal(llp.beam_reorder(one, dev(parents), out=o), one)


def test_beam_reorder_of_parents_past_the_beams(llp):
    x = torch.arange(24, device="cuda", dtype=torch.float32).reshape(6, 4)
    p = torch.tensor([[1, 3, 0], [-2, 2, 1]], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = llp.beam_reorder(x.clone(), p, status=st)
    assert torch.equal(y, x[[1, 1, 0, 3, 5, 4]]) and int(st) == llp.STATUS_BITS["PARENT_INVALID"]


def test_beam_reorder_of_nothing(llp):
    p = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 4), device="cuda")
    assert llp.beam_reorder(x, p) is x
    p = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    assert llp.beam_reorder([], p) == []
    x = torch.empty((2, 0, 4), device="cuda")
    assert llp.beam_reorder([x], p)[0] is x
