"""Reordering of states that fill a launch, on the GPU."""
import pytest
import torch

from tests._gpu import need_gpu, say

pytestmark = pytest.mark.gpu


def test_beam_reorder_of_states_that_fill_a_launch():
    # 64 states of 1024 sequences of 2 beams, a byte a thread: 2^32 threads together, more than a launch holds.
    need_gpu()
    import lm_head_linear_logp_amd as llp
    n, B, K, W = 64, 1024, 2, 65535
    say(f"beam_reorder {n} states of {B * K} x {W} bytes")
    g = torch.Generator(device="cuda").manual_seed(1)
    room = torch.randint(0, 256, (n, B * K, W), generator=g, device="cuda", dtype=torch.uint8)
    parents = torch.randint(0, K, (B, K), generator=g, device="cuda").to(torch.int32)
    take = (parents + K * torch.arange(B, device="cuda", dtype=torch.int32)[:, None]).reshape(-1).long()
    sums = [room[i].long().sum(1)[take] for i in range(n)]
    first, last = room[0][take], room[n - 1][take]
    llp.beam_reorder(list(room), parents)
    for i in range(n):
        assert torch.equal(room[i].long().sum(1), sums[i]), i
    assert torch.equal(room[0], first) and torch.equal(room[n - 1], last)


def test_beam_reorder_of_parts_of_one_buffers_rows():
    need_gpu()
    import lm_head_linear_logp_amd as llp
    g = torch.Generator(device="cuda").manual_seed(2)
    parents = torch.randint(0, 4, (3, 4), generator=g, device="cuda").to(torch.int32)
    take = (parents + 4 * torch.arange(3, device="cuda", dtype=torch.int32)[:, None]).reshape(-1).long()
    for split, used in ((512, 20), (512, 13), (301, 13)):
        wide = torch.randn(12, 20, 576, generator=g, device="cuda").to(torch.bfloat16)
        want = wide.clone()
        want[:, :used] = wide[take, :used]
        llp.beam_reorder([wide[:, :used, :split], wide[:, :used, split:]], parents)
        assert torch.equal(wide, want)
