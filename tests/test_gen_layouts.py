"""Which states beam_reorder takes together (CPU only): every set whose bytes lie apart as parts of one buffer's rows do,
whatever the parts' widths, and none that share a byte."""
import itertools

import numpy as np
import pytest
import torch

import lm_head_linear_logp_amd as llp

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="a GPU is present: the tensors are not on it")
P = torch.zeros(2, 4, dtype=torch.int32)


def taken(states, **kw):
    """Whether the checks let the states through (to the missing GPU)."""
    try:
        llp.beam_reorder(states, P, **kw)
    except RuntimeError as e:
        assert "gfx950" in str(e)
        return True
    except ValueError as e:
        assert "overlap" in str(e), e
        return False
    raise AssertionError("nothing to move")


def test_parts_of_rows_of_different_widths_are_taken():
    wide = torch.zeros(8, 20, 576, dtype=torch.bfloat16)      # a latent of 512 and 64 columns beside it
    assert taken([wide[:, :, :512], wide[:, :, 512:]]) and taken([wide[:, :, 512:], wide[:, :, :512]])
    assert taken([wide[:, :13, :512], wide[:, :13, 512:]]) and taken([wide[:, :13], wide[:, 13:]])
    assert taken([wide[:, :13, :100], wide[:, 13:]]) and taken([wide[:, 0, :7], wide[:, 1:, 3:], wide[:, 0, 7:]])
    flat = torch.zeros(8, 1000)
    assert taken([flat[:, :300], flat[:, 300:301], flat[:, 301:]])
    assert taken([flat[:, :10].view(torch.uint8), flat[:, 10:20].view(torch.int16)])
    heads = torch.zeros(3, 8, 10, 24)                         # rows within heads
    assert taken([heads.transpose(0, 1)[:, :, :4], heads.transpose(0, 1)[:, :, 4:]])
    assert taken([heads[0], heads[1], heads[2]])


def test_parts_that_share_a_byte_are_refused():
    wide = torch.zeros(8, 20, 576, dtype=torch.bfloat16)
    assert not taken([wide[:, :, :513], wide[:, :, 512:]]) and not taken([wide[:, :14], wide[:, 13:]])
    assert not taken([wide[:, :13], wide[:, 12:, 575:]]) and not taken([wide[:, 0], wide])
    flat = torch.zeros(8, 1000)
    assert not taken([flat[:, :300], flat[:, 299:]]) and not taken([flat, flat[:, 999:]])


def test_no_states_that_share_a_byte_are_taken():
    g = np.random.default_rng(0)
    room = torch.zeros(1 << 14, dtype=torch.uint8)
    apart = n = 0
    for _ in range(6000):
        views, places = [], []
        outer, row = int(g.integers(1, 5)), int(g.choice([64, 96, 200]))
        for _ in range(int(g.integers(2, 4))):
            inner, do = int(g.integers(1, 24)), int(g.choice([8, 16, 24, 32]))
            dr = int(g.choice([row, row, row + 8]))
            if g.random() < 0.3:
                dr, do = int(g.choice([16, 24, 40])), 8 * row
            at = int(g.integers(0, 2 * row))
            v = torch.as_strided(room, (8, outer, inner), (dr, do, 1), at)
            views.append(v)
            places.append((np.arange(8)[:, None, None] * dr + np.arange(outer)[:, None] * do + np.arange(inner) + at).reshape(-1))
        if any(len(np.unique(p)) < len(p) for p in places):
            continue                                          # a state that overlaps itself
        share = any(len(np.intersect1d(a, b)) for a, b in itertools.combinations(places, 2))
        got = taken(views)
        apart += not share
        n += got
        assert not (got and share), [(tuple(v.shape), v.stride(), v.storage_offset()) for v in views]
    assert apart > 300 and n > apart // 2
