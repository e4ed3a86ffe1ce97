"""The fp8 and beam-search operators as a program uses them: decoding steps from hidden states to
reordered states, a training step, both captured and replayed, and calls on several streams at once."""
import numpy as np
import pytest
import torch

from oracle import gen as O
from tests._gpu import bytes_equal, dev, host, need_gpu, say

pytestmark = pytest.mark.gpu
V, VP, H, B, K = 1000, 1024, 256, 3, 4


@pytest.fixture(scope="module")
def llp():
    need_gpu()
    import lm_head_linear_logp_amd as m
    m.open(0)
    return m


def model(llp, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn(VP, H, generator=g, device="cuda").to(torch.bfloat16)
    head = (torch.randn(VP, H, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    return table, head, llp.quantize_blocks(head, rows=128)


def decode(llp, table, weight, state, shards):
    """One step: logits of every beam, the choice, and everything kept per beam in its new place."""
    z = llp.linear_fp8(*llp.quantize_blocks(state["h"]), *weight, out_dtype=torch.float32)
    cuts = [VP * i // shards for i in range(shards + 1)]
    parts = [llp.beam_candidates(z[:, a:b], 2 * K, temperature=0.7, offset=a, real_vocab=V, padded_vocab=VP, rank=r,
                                 world=shards) for r, (a, b) in enumerate(zip(cuts, cuts[1:]))]
    got = llp.beam_select(parts, state["score"], K, temperature=0.7, finished=state["done"], end_id=0)
    llp.beam_reorder([state["cache"], state["tokens"], state["h"], state["done"].view(-1)], got["parent"])
    state["tokens"][:, state["at"]] = got["token"].reshape(-1)
    state["cache"][:, :, state["at"]] = state["h"].reshape(B * K, 4, -1)
    state["score"].copy_(got["score"])
    state["done"].copy_(torch.logical_or(state["done"] != 0, got["token"] < 120))
    state["h"].copy_((state["h"] * 0.5 + llp.embedding_forward(got["token"].reshape(-1), table, real_vocab=V)))
    state["at"] += 1
    return z, got


def fresh(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    score = torch.full((B, K), -float("inf"), device="cuda")
    score[:, 0] = 0
    return dict(h=torch.randn(B * K, H, generator=g, device="cuda").to(torch.bfloat16), score=score, at=0,
                cache=torch.zeros(B * K, 4, 12, H // 4, device="cuda", dtype=torch.bfloat16),
                tokens=torch.zeros(B * K, 12, dtype=torch.int64, device="cuda"),
                done=torch.zeros(B, K, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("shards", [1, 2, 4])
def test_decoding_steps_against_the_oracle(llp, shards):
    table, head, weight = model(llp)
    s = fresh(5)
    c = float(np.float32(1.0 / np.float64(np.float32(0.7))))
    wv = O.values(*O.quantize_blocks(host(head.float()), 128), 128)
    for step in range(6):
        before = {k: v.clone() for k, v in s.items() if k != "at"}
        z, got = decode(llp, table, weight, s, shards)
        say(f"step {step}: scores {host(got['score'])[0]}")
        hv = O.values(*O.quantize_blocks(host(before["h"].float())), 1)
        ref, size = O.linear(hv, wv)
        assert (np.abs(host(z) - ref) <= size * 2.0 ** -24 * (2 * 128 + 2 * 2 + 4) + np.abs(ref) * 2.0 ** -24).all()
        token, parent, score = O.beam_select(host(z)[:, :V].reshape(B, K, V), host(before["score"]), K, c,
                                             host(before["done"]), 0)
        assert np.array_equal(host(got["token"]), token) and np.array_equal(host(got["parent"]), parent)
        fin = np.isfinite(score)
        assert (np.abs(host(got["score"]) - score)[fin] <= 2.0 ** -24 * (80 + np.abs(score[fin]))).all()
        # What is kept follows: histories and caches are those of the parents, then the step's own.
        for k in ("tokens", "cache"):
            kept = host(before[k].float())
            want = O.beam_reorder(kept, parent)
            assert np.array_equal(host(s[k].float())[..., :step, :] if k == "cache" else host(s[k])[:, :step],
                                  want[..., :step, :] if k == "cache" else want[:, :step])
        # A beam's score is its parent's and the log-probability that the logits' own forward gives.
        live = fin & (np.take_along_axis(host(before["done"]), np.maximum(parent, 0).astype(np.int64), 1) == 0)
        rows = torch.arange(B, device="cuda")[:, None] * K + got["parent"].clamp_min(0)
        lp = llp.forward_logits(z[rows.reshape(-1)].contiguous(), got["token"].reshape(-1), temperature=0.7,
                                real_vocab=V, padded_vocab=VP)["logp"].reshape(B, K)
        old = np.take_along_axis(host(before["score"]), np.maximum(parent, 0).astype(np.int64), 1)
        assert np.allclose((old + host(lp))[live], host(got["score"])[live], rtol=0, atol=2e-5)


def test_a_captured_step_replays_as_the_eager_one(llp):
    table, head, weight = model(llp, 2)
    h = torch.zeros(B * K, H, dtype=torch.bfloat16, device="cuda")
    score = torch.zeros(B, K, device="cuda")
    cache = torch.zeros(B * K, 4, 9, 16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(out=None):
        z = llp.linear_fp8(*llp.quantize_blocks(h), *weight, out_dtype=torch.float32)
        p = llp.beam_candidates(z, K, real_vocab=V, status=status)
        got = llp.beam_select([p], score, status=status)
        llp.beam_reorder(cache[:, :, :7], got["parent"], status=status)
        return z, got

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h.copy_(torch.randn(B * K, H, generator=g, device="cuda"))
        score.copy_(torch.randn(B, K, generator=g, device="cuda"))
        cache.copy_(torch.randn(cache.shape, generator=g, device="cuda"))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill(0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, got = step()
    for seed in (1, 2, 3, 4):
        fill(seed)
        ez, egot = step()
        want = [ez.clone(), *(v.clone() for v in egot.values()), cache.clone()]
        torch.cuda.synchronize()
        fill(seed)
        graph.replay()
        assert all(bytes_equal(a, b) for a, b in zip([z, *got.values(), cache], want)), seed
        torch.cuda.synchronize()
    assert int(status) == 0


def test_a_captured_training_step_replays_as_the_eager_one(llp):
    T, H2, V2 = 200, 320, 640
    x = torch.zeros(T, H2, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(V2, H2, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(T, V2, dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros(V2, H2, device="cuda")

    def step():
        y = llp.linear_fp8(*llp.quantize_blocks(x), *llp.quantize_blocks(w, rows=128))
        dx = llp.linear_fp8(*llp.quantize_blocks(dy), *llp.quantize_blocks(w, rows=128, transpose=True))
        a = (*llp.quantize_blocks(dy, rows=128, transpose=True), *llp.quantize_blocks(x, transpose=True))
        dw = llp.dweight_fp8(*a, out_dtype=torch.bfloat16)
        llp.dweight_fp8(*a, dweight=acc)
        return y, dx, dw

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        acc.zero_()

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        fill(seed)
        want = [t.clone() for t in step()] + [acc.clone()]
        # The autograd node gives the same bits.
        xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = llp.fp8_linear(xl, wl)
        dx, dw = torch.autograd.grad(y, (xl, wl), dy)
        assert all(bytes_equal(a, b) for a, b in zip((y.detach(), dx, dw), want))
        fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        assert all(bytes_equal(a, b) for a, b in zip([*out, acc], want)), seed
        torch.cuda.synchronize()


def test_calls_on_several_streams_at_once(llp):
    table, head, weight = model(llp, 3)
    g = torch.Generator(device="cuda").manual_seed(9)
    work = [dict(h=torch.randn(n, H, generator=g, device="cuda").to(torch.bfloat16), k=k) for n, k in
            ((4, 4), (40, 5), (300, 3), (2100, 2), (8, 8))]

    def run(w):
        z = llp.linear_fp8(*llp.quantize_blocks(w["h"]), *weight, out_dtype=torch.float32)
        p = llp.beam_candidates(z, 2 * w["k"], real_vocab=V)
        got = llp.beam_select([p], torch.zeros(z.shape[0] // w["k"], w["k"], device="cuda"))
        h = llp.beam_reorder(w["h"].clone(), got["parent"])
        return z, got["token"], got["score"], h

    want = [run(w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        got = []
        for w, s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(run(w))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(bytes_equal(x, y) for x, y in zip(a, b))


def test_the_smallest_and_odd_decoding(llp):
    # One row, one column; a vocabulary smaller than the beams; beams without a candidate stay -1 and their
    # states stay where they are.
    q, s = llp.quantize_blocks(torch.ones(1, 1, device="cuda"))
    y = llp.linear_fp8(q, s, *llp.quantize_blocks(torch.full((1, 1), 3.0, device="cuda"), rows=128), out_dtype=torch.float32)
    # 448 * 448 exactly, times scales of 1 and 3 by fl(1/448): five roundings.
    assert abs(float(y) - 3.0) <= 3.0 * 5 * 2.0 ** -24
    z = torch.tensor([[1.0, 0.0, 0.0, 0.0]] * 4, device="cuda")
    p = llp.beam_candidates(z, 4, real_vocab=1, padded_vocab=4)
    sc = torch.tensor([[-1.0, -2.0, -float("inf"), -float("inf")]], device="cuda")
    got = llp.beam_select([p], sc)
    assert host(got["parent"]).tolist() == [[0, 1, -1, -1]] and host(got["token"]).tolist() == [[0, 0, -1, -1]]
    x = torch.arange(8.0, device="cuda").reshape(4, 2)
    assert torch.equal(llp.beam_reorder(x.clone(), got["parent"]), x)


def test_a_captured_autograd_step_replays_as_the_eager_one(llp):
    # Forward and backward of the autograd node recorded together, its leaves' gradients taken, not accumulated.
    T, H2, V2 = 150, 256, 400
    x = torch.zeros(T, H2, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.zeros(V2, H2, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    dy = torch.zeros(T, V2, dtype=torch.bfloat16, device="cuda")

    def step():
        y = llp.fp8_linear(x, w)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        with torch.no_grad():
            for t in (x, w, dy):
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill(0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        assert all(bytes_equal(a, b) for a, b in zip(out, want)), seed
        torch.cuda.synchronize()
