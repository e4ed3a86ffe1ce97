"""What the decoding calls write into a caller's tensors counts as changed in place: autograd refuses a backward
pass that saved it before."""
import pytest
import torch

from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def changed(call, *tensors):
    before = [t._version for t in tensors]
    call()
    return all(t._version > b for t, b in zip(tensors, before))


def test_written_tensors_count_as_changed(llp):
    x = torch.randn(40, 256, device="cuda")
    xq, xs = llp.quantize_blocks(x)
    assert changed(lambda: llp.quantize_blocks(x, out=(xq, xs)), xq, xs)
    wq, ws = llp.quantize_blocks(torch.randn(128, 256, device="cuda"), rows=128)
    y = llp.linear_fp8(xq, xs, wq, ws, out_dtype=torch.float32)
    assert changed(lambda: llp.linear_fp8(xq, xs, wq, ws, out=y), y)
    dw = torch.zeros(128, 40, device="cuda")
    for overwrite in (False, True):
        assert changed(lambda: llp.dweight_fp8(wq, ws, xq, xs, dweight=dw, overwrite=overwrite), dw)
    parts = llp.beam_candidates(y, 4)
    assert changed(lambda: llp.beam_candidates(y, 4, out=parts), *parts.values())
    scores = torch.zeros(10, 4, device="cuda")
    step = llp.beam_select([parts], scores)
    assert changed(lambda: llp.beam_select([parts], scores, out=step), *step.values())
    states = [torch.randn(40, 3, 8, device="cuda"), torch.arange(40, device="cuda")]
    assert changed(lambda: llp.beam_reorder(states, step["parent"]), *states)
    out = [torch.empty_like(s) for s in states]
    before = [s._version for s in states]
    assert changed(lambda: llp.beam_reorder(states, step["parent"], out=out), *out)
    assert [s._version for s in states] == before
    assert not changed(lambda: llp.linear_fp8(xq, xs, wq, ws), xq, xs, wq, ws)


def test_a_backward_pass_that_saved_a_reordered_state_is_refused(llp):
    w = torch.randn(8, device="cuda", requires_grad=True)
    state = torch.randn(4, 8, device="cuda")
    parents = torch.tensor([[1, 0, 3, 2]], dtype=torch.int32, device="cuda")
    loss = (state * w).sum()
    llp.beam_reorder(state, parents)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # A view shares its base's count.
    room = torch.randn(4, 3, 8, device="cuda")
    loss = (room * w).sum()
    llp.beam_reorder([room[:, 1]], parents)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_have_no_count(llp):
    parents = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    with torch.inference_mode():
        x = torch.arange(6, device="cuda").reshape(2, 3)
        assert llp.beam_reorder(x, parents) is x and x[:, 0].tolist() == [3, 0]
        y = llp.linear_fp8(*llp.quantize_blocks(torch.ones(2, 128, device="cuda")),
                           *llp.quantize_blocks(torch.ones(8, 128, device="cuda"), rows=128))
        assert (y == 128).all()
    assert llp.beam_reorder(x, parents) is x and x[:, 0].tolist() == [0, 3]
