"""A forward of few rows ends in a combine of its own: its rows have the bits they have in a large
batch, with entropy and without, and in the library's own scratch."""
import pytest
import torch

from tests._gpu import LOGP_ATOL, bytes_equal, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def _inputs(T, H, V, pad, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(pad, H, generator=g, device="cuda") * 0.3).bfloat16()
    tg = torch.randint(0, V, (T,), generator=g, device="cuda")
    b = torch.randn(pad, generator=g, device="cuda")
    return h, w, tg, b


# 3 tiles, 79, a whole head's 593; 2048 and 2049 tiles, where the few-row combine ends.
@pytest.mark.parametrize("V", [700, 20001, 151669, 524288, 524289])
def test_rows_of_a_small_batch_have_the_bits_of_a_large_one(llp, V):
    T, H, pad = 300, 64, (V + 63) // 64 * 64
    h, w, tg, b = _inputs(T, H, V, pad, V)
    kw = dict(temperature=0.7, real_vocab=V, padded_vocab=pad, bias=b)
    whole = llp.forward(h, w, tg, **kw)
    z = (h.double() @ w[:V].double().t() + b[:V].double()) / 0.7
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    assert float((whole["lse"].double() - lse).abs().max()) <= LOGP_ATOL
    assert float((whole["entropy"].double() - (lse - (p * z).sum(1))).abs().max()) <= LOGP_ATOL
    for rows in ([0], [299], [7, 3], list(range(17)), list(range(100, 133)), list(range(200, 264)),
                 list(range(299, 170, -2))):
        say(f"few rows V={V} n={len(rows)}")
        i = torch.tensor(rows, device="cuda")
        part = llp.forward(h[i], w, tg[i], **kw)
        for k in whole:
            assert bytes_equal(part[k], whole[k][i]), (k, len(rows))
        bare = llp.forward(h[i], w, tg[i], want_entropy=False, **kw)
        for k in ("logp", "lse", "target_logit", "in_range"):
            assert bytes_equal(bare[k], whole[k][i]), (k, len(rows))
    i = torch.arange(40, 104, device="cuda")
    mask = (torch.arange(64, device="cuda") % 3 != 1).to(torch.uint8)
    part = llp.forward(h[i], w, tg[i], loss_mask=mask, **kw)
    on = mask.bool()
    for k in whole:
        assert bytes_equal(part[k][on], whole[k][i][on]), k
        assert not part[k][~on].any(), k
    out = {k: torch.empty_like(v[i]) for k, v in whole.items()}
    llp.forward_noalloc(h[i], w, tg[i], out=out, **kw)
    for k in whole:
        assert bytes_equal(out[k], whole[k][i]), k


def test_few_rows_of_far_logits_and_empty_shards_bitwise(llp):
    # Maxima that differ by hundreds between tiles (sums of 0 in most chains), and a shard whose real
    # columns are none.
    T, H, V, pad = 128, 64, 30000, 30016
    h, w, tg, b = _inputs(T, H, V, pad, 5)
    b = b * 300
    kw = dict(temperature=1.0, real_vocab=V, padded_vocab=2 * pad, bias=b, world=2)
    for off in (0, pad):
        whole = llp.forward(h, w, tg, rank=1 if off else 0, offset=off, **kw)
        part = llp.forward(h[20:50], w, tg[20:50], rank=1 if off else 0, offset=off, **kw)
        for k in whole:
            assert bytes_equal(part[k], whole[k][20:50]), (k, off)
        if off:
            assert torch.isneginf(whole["lse"]).all() and not whole["entropy"].any()
