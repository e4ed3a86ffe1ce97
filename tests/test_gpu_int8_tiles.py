"""int8 scoring where a worker of the wide tile takes several tiles one after another (an even number
of 128-column steps, more tiles than compute units): values against the oracle, and the bits of the
few-row form, which has no such workers."""
import numpy as np
import pytest
import torch

from oracle import ops as O
from tests._gpu import bytes_equal, dev, need_gpu, say
from tests.test_gpu_int8 import _case, _close, _dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


# Scored tiles of 256 rows x 256 columns: 940, 470 and 940; and 3 tiles per worker of 4 K steps.
@pytest.mark.parametrize("T,K,V,bias", [(1100, 256, 60001, "f32"), (300, 256, 60001, "bf16"),
                                        (1100, 256, 60000, None), (700, 512, 66000, "f32")])
def test_workers_with_several_tiles(llp, T, K, V, bias):
    say(f"int8 tiles T={T} K={K} V={V} bias={bias}")
    pad = V + 40
    c = _case(T, K, V, pad, seed=T + K, bias=bias, mask_frac=0.1)
    d = _dev(c)
    kw = dict(temperature=0.7, bias=d["b"], real_vocab=V, padded_vocab=pad)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], loss_mask=d["mask"], status=st, **kw)
    b = None if c["b"] is None else c["b"].float().numpy()
    z = O.int8_logits(c["hq"], c["hs"], c["wq"], c["ws"], b, 0.7, V)
    _close(out, O.score(z, c["tg"], c["mask"]), z)
    assert int(st) == 0
    again = llp.forward_int8(d["hq"], d["hs"], d["wq"], d["ws"], d["tg"], loss_mask=d["mask"], **kw)
    for k in out:
        assert bytes_equal(out[k], again[k]), k
    on = np.nonzero(c["mask"])[0]
    for rows in (on[:1], on[-48:], on[len(on) // 2:len(on) // 2 + 64], on[::29]):
        i = dev(rows[:64])
        part = llp.forward_int8(d["hq"][i], d["hs"][i], d["wq"], d["ws"], d["tg"][i], **kw)
        for k in out:
            assert bytes_equal(part[k], out[k][i]), (k, len(rows))
