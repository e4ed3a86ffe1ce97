"""The operators that decode and train with a head in 8-bit floating point refuse malformed calls before
anything reaches a device: the C ABI with its documented status, the binding with ValueError or TypeError.
Struct layouts and constants match the header. Runs on the CPU."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import lm_head_linear_logp_amd as llp
from lm_head_linear_logp_amd import _capi as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "llp.h")
FAKE = 0x100000
BAD = (ValueError, TypeError)
INV, UNS = A.LLP_ERR_INVALID_ARGUMENT, A.LLP_ERR_UNSUPPORTED

needs_lib = pytest.mark.skipif(not os.path.exists(A.LIB_PATH), reason="libllp.so not built")
STRUCTS = ["llp_fp8_quant_request", "llp_fp8_linear_request", "llp_beam_request", "llp_beam_parts",
           "llp_beam_select_request", "llp_beam_out", "llp_beam_reorder_request"]


def test_structs_and_constants_match_the_header(tmp_path):
    names = ["LLP_FP8_BLOCK", "LLP_MAX_BEAMS", "LLP_STATUS_PARENT_INVALID", "LLP_STATUS_VALUE_NOT_FINITE"]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "llp.h"', "int main(void){"]
    for s in STRUCTS:
        src.append(f'printf("{s} size %zu\\n", sizeof({s}));')
        src += [f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));' for f, _ in getattr(A, s)._fields_]
    src += [f'printf("const {n} %d\\n", (int){n});' for n in names] + ["return 0;}"]
    c, exe = tmp_path / "p.c", tmp_path / "p"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(c), "-o", str(exe)], check=True)
    for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        s, f, v = ln.split()
        want = getattr(A, f) if s == "const" else (
            C.sizeof(getattr(A, s)) if f == "size" else getattr(getattr(A, s), f).offset)
        assert int(v) == want, ln


# ---- C ABI ----------------------------------------------------------------------------------
def quant(**over):
    r = A.llp_fp8_quant_request(FAKE, A.LLP_DTYPE_BF16, 1, 256, 10, 200, 0, 0, FAKE, 256, FAKE, 256)
    for k, v in over.items():
        setattr(r, k, v)
    return A.load().llp_quantize_blocks(C.byref(r), None)


def linear(grad=False, **over):
    r = A.llp_fp8_linear_request(FAKE, 256, FAKE, 300, FAKE, 256, FAKE, 2, None, 0, A.LLP_DTYPE_F32, FAKE, 500,
                                 300, 400, 256, 0, 0)
    for k, v in over.items():
        setattr(r, k, v)
    return getattr(A.load(), "llp_dweight_fp8" if grad else "llp_linear_fp8")(C.byref(r), None)


def candidates(out=None, **over):
    r = A.llp_beam_request()
    r.logits, r.logits_dtype, r.num, r.logits_stride, r.num_rows, r.temperature = FAKE, A.LLP_DTYPE_F32, 8, 1000, 12, 0.7
    r.vocab.local_size = r.vocab.real_vocab = r.vocab.padded_vocab = 1000
    r.vocab.world = 1
    for k, v in over.items():
        if k in ("offset", "local_size", "real_vocab", "padded_vocab", "rank", "world"):
            setattr(r.vocab, k, v)
        else:
            setattr(r, k, v)
    o = A.llp_beam_parts(FAKE, FAKE, FAKE, FAKE) if out is None else out
    return A.load().llp_beam_candidates(C.byref(r), C.byref(o), None)


def select(parts=None, out=None, **over):
    p = (A.llp_beam_parts * 2)(*(parts or [A.llp_beam_parts(FAKE, FAKE, FAKE, FAKE)] * 2))
    r = A.llp_beam_select_request(2, 8, p, 3, 4, 8, FAKE, None, 0, 1.0, 0, None)
    for k, v in over.items():
        setattr(r, k, v)
    o = A.llp_beam_out(FAKE, FAKE, FAKE) if out is None else out
    return A.load().llp_beam_select(C.byref(r), C.byref(o), None)


def reorder(src=(FAKE,), dst=(FAKE,), **over):
    n = len(src)
    r = A.llp_beam_reorder_request((C.c_void_p * n)(*src), (C.c_void_p * n)(*dst), n, 4, 4, 0, 2, 3, 64, 256, 64, 256,
                                   64, FAKE, None)
    for k, v in over.items():
        setattr(r, k, v)
    return A.load().llp_beam_reorder(C.byref(r), None)


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(x_dtype=3), INV), (dict(block_rows=64), INV), (dict(x_stride=199), INV), (dict(rows=-1), INV),
    (dict(cols=-1), INV), (dict(rows=1 << 31), INV), (dict(q_stride=240), INV), (dict(q_stride=264), INV),
    (dict(scale_stride=9), INV), (dict(transpose=1, q_stride=112), INV), (dict(transpose=1, scale_stride=199), INV),
    (dict(block_rows=128, scale_stride=1), INV), (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV),
    (dict(x=FAKE + 1), INV), (dict(q=FAKE + 8), INV), (dict(scale=FAKE + 2), INV),
    (dict(rows=1 << 30, scale_stride=1 << 30), UNS)])
def test_quantize_refusals(over, want):
    assert quant(**over) == want, llp.last_error()


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(depth=100), INV), (dict(depth=-128), INV), (dict(depth=(1 << 23) + 128), UNS), (dict(rows=-1), INV),
    (dict(cols=-1), INV), (dict(rows=1 << 23, x_scale_stride=1 << 23), UNS), (dict(cols=1 << 23, out_stride=1 << 23), UNS),
    (dict(x_stride=128), INV), (dict(x_stride=264), INV), (dict(weight_stride=240), INV), (dict(x_stride=1 << 24), UNS),
    (dict(weight_stride=1 << 24), UNS), (dict(x_stride=(1 << 23) + 16), UNS), (dict(weight_stride=(1 << 23) + 16), UNS), (dict(x_scale_stride=299), INV), (dict(weight_scale_stride=1), INV),
    (dict(x=None), INV), (dict(x_scale=None), INV), (dict(weight=None), INV), (dict(weight_scale=None), INV),
    (dict(x=FAKE + 8), INV), (dict(weight=FAKE + 4), INV), (dict(x_scale=FAKE + 1), INV), (dict(out=None), INV),
    (dict(out=FAKE + 2), INV), (dict(out_stride=399), INV), (dict(out_dtype=0), INV), (dict(flags=1), INV),
    (dict(flags=2), INV), (dict(bias=FAKE, bias_dtype=9), INV), (dict(bias=FAKE + 2, bias_dtype=A.LLP_DTYPE_F32), INV),
    (dict(rows=(1 << 22), cols=1 << 22, x_scale_stride=1 << 22, out_stride=1 << 22), UNS)])
def test_linear_refusals(over, want):
    assert linear(**over) == want, llp.last_error()


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(bias=FAKE, bias_dtype=A.LLP_DTYPE_F32), INV), (dict(flags=4), INV), (dict(out_stride=299), INV),
    (dict(out_dtype=A.LLP_DTYPE_BF16), INV), (dict(depth=64), INV), (dict(out_stride=1 << 24), UNS)])
def test_dweight_refusals(over, want):
    assert linear(True, **over) == want, llp.last_error()


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(num=0), INV), (dict(num=65), INV), (dict(num_rows=-1), INV), (dict(num_rows=1 << 22), INV),
    (dict(logits_dtype=5), INV), (dict(logits_stride=999), INV), (dict(logits_stride=1001), INV), (dict(logits=None), INV),
    (dict(logits=FAKE + 8), INV), (dict(temperature=0.0), INV), (dict(temperature=float("nan")), INV),
    (dict(temperature=1e-39), INV), (dict(offset=-1), INV), (dict(world=0), INV), (dict(real_vocab=0), INV),
    (dict(local_size=1 << 23, padded_vocab=1 << 23, real_vocab=1 << 23, logits_stride=1 << 23), UNS),
    (dict(local_size=(1 << 21) + 8, padded_vocab=(1 << 21) + 8, real_vocab=1 << 21, logits_stride=1 << 22), UNS),
    (dict(local_size=1000, padded_vocab=1 << 41, world=2), UNS),
    (dict(temperature=2.0 ** -65), INV), (dict(temperature=2.0 ** 65), INV),
    (dict(out=A.llp_beam_parts(FAKE, FAKE, FAKE, None)), INV)])
def test_candidates_refusals(over, want):
    assert candidates(**over) == want, llp.last_error()


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(world=0), INV), (dict(world=65), INV), (dict(num=0), INV), (dict(num=65), INV), (dict(num=7), INV),
    (dict(num_out=0), INV), (dict(num_beams=0), INV), (dict(num_beams=65), INV), (dict(num_seqs=-1), INV),
    (dict(num_seqs=1 << 22), INV), (dict(temperature=0.0), INV), (dict(temperature=1e-39), INV), (dict(scores=None), INV),
    (dict(out=A.llp_beam_out(FAKE, None, FAKE)), INV),
    (dict(parts=[A.llp_beam_parts(FAKE, FAKE, FAKE, FAKE), A.llp_beam_parts(FAKE, FAKE, None, FAKE)]), INV)])
def test_select_refusals(over, want):
    assert select(**over) == want, llp.last_error()


@needs_lib
@pytest.mark.parametrize("over,want", [
    (dict(num_src=0), INV), (dict(num_out=65), INV), (dict(num_seqs=-1), INV), (dict(outer=-1), INV), (dict(inner=-1), INV),
    (dict(num_states=-1), INV), (dict(parents=None), INV), (dict(src=(None,)), INV), (dict(dst=(None,)), INV),
    (dict(src_row_stride=-1), INV), (dict(dst_outer_stride=1 << 41), INV), (dict(num_src=3), INV),
    (dict(src_row_stride=512), INV), (dict(src=(FAKE, FAKE), dst=(FAKE, FAKE)), INV),
    (dict(src=(FAKE, FAKE * 2), dst=(FAKE, FAKE * 3)), INV), (dict(src_row_stride=128, dst_row_stride=128), INV),
    (dict(src_outer_stride=63, dst_outer_stride=63), INV), (dict(num_seqs=1 << 22), INV),
    (dict(outer=1 << 30, src_outer_stride=64, dst_outer_stride=64, src_row_stride=1 << 36, dst_row_stride=1 << 36), UNS)])
def test_reorder_refusals(over, want):
    assert reorder(**over) == want, llp.last_error()


@needs_lib
def test_null_requests():
    lib = A.load()
    assert lib.llp_quantize_blocks(None, None) == INV
    assert lib.llp_quantize_both(None, None, None) == INV
    assert lib.llp_linear_fp8(None, None) == INV and lib.llp_dweight_fp8(None, None) == INV
    assert lib.llp_beam_candidates(None, None, None) == INV
    assert lib.llp_beam_select(None, None, None) == INV
    assert lib.llp_beam_reorder(None, None) == INV


@needs_lib
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="a GPU is present: the pointers are not real")
def test_well_formed_requests_pass_validation():
    # On a machine without a GPU they are refused at the device, with their own message.
    for st in (quant(), quant(transpose=1, scale_stride=200), quant(block_rows=128), linear(), linear(True), candidates(),
               select(), reorder(), reorder(src=(FAKE, FAKE * 2)[:1], dst=(FAKE * 4,), num_src=2),
               linear(True, flags=2, out_dtype=A.LLP_DTYPE_BF16), linear(depth=0, x=None, weight=None)):
        assert st in (A.LLP_ERR_INVALID_ARGUMENT, A.LLP_ERR_HIP), llp.last_error()
        assert "llp_open" in llp.last_error() or "hipGetDevice" in llp.last_error(), llp.last_error()


# ---- Binding --------------------------------------------------------------------------------
T, K, V = 6, 256, 300
F8 = torch.float8_e4m3fn


def f8(*s):
    return torch.zeros(s, dtype=torch.uint8).view(F8)


def lin(**over):
    a = dict(x=f8(T, K), x_scale=torch.zeros(2, T).t(), weight=f8(V, K), weight_scale=torch.zeros(3, 2))
    kw = {}
    for k, v in over.items():
        (a if k in a else kw)[k] = v
    return llp.linear_fp8(**a, **kw)


def dw(**over):
    a = dict(dout_t=f8(V, K), dout_scale=torch.zeros(3, 2), x_t=f8(T, K), x_scale=torch.zeros(2, T).t())
    kw = {}
    for k, v in over.items():
        (a if k in a else kw)[k] = v
    return llp.dweight_fp8(**a, **kw)


def reaches_library(f, **over):
    with pytest.raises(RuntimeError) as e:
        f(**over)
    assert not isinstance(e.value, BAD)


def test_quantize_binding():
    x = torch.zeros(5, 200)
    reaches_library(lambda: llp.quantize_blocks(x))
    reaches_library(lambda: llp.quantize_blocks(x, out=(f8(5, 256), torch.zeros(2, 5).t())))
    for bad in (dict(rows=2), dict(out=(f8(5, 200), torch.zeros(2, 5).t())), dict(out=(f8(5, 256), torch.zeros(5, 2))),
                dict(out=(f8(5, 256), torch.zeros(5, 3).t())), dict(rows=128, out=(f8(5, 256), torch.zeros(2, 3).t())),
                dict(rows=128, out=(f8(5, 256), torch.zeros(2, 2).t()[:1]), transpose=True),
                dict(out=(torch.zeros(5, 256, dtype=torch.uint8), torch.zeros(2, 5).t()))):
        with pytest.raises(BAD):
            llp.quantize_blocks(x, **bad)
    reaches_library(lambda: llp.quantize_both(x))
    for t in (x.half(), x[0], x.t(), x.to(torch.float64), None):
        with pytest.raises(BAD):
            llp.quantize_blocks(t)
        with pytest.raises(BAD):
            llp.quantize_both(t)


@pytest.mark.parametrize("over", [
    dict(x=f8(T, K - 128)), dict(x=f8(T, 200), weight=f8(V, 200)), dict(x=torch.zeros(T, K)), dict(weight=f8(V, K).t()),
    dict(x_scale=torch.zeros(T, 2)), dict(x_scale=torch.zeros(2, T)), dict(x_scale=torch.zeros(2, T).half().t()),
    dict(weight_scale=torch.zeros(2, 2)), dict(weight_scale=torch.zeros(2, 3).t()), dict(bias=torch.zeros(V - 1)),
    dict(bias=torch.zeros(V, dtype=torch.float64)), dict(out_dtype=torch.float16), dict(out=torch.zeros(T, V + 1)),
    dict(out=torch.zeros(T, V, dtype=torch.float16)), dict(out=torch.zeros(V, T).t())])
def test_linear_binding(over):
    reaches_library(lin)
    with pytest.raises(BAD):
        lin(**over)


@pytest.mark.parametrize("over", [
    dict(dout_t=f8(V, 128)), dict(dout_scale=torch.zeros(2, 3).t()), dict(x_scale=torch.zeros(T, 2)),
    dict(dweight=torch.zeros(V, T, dtype=torch.bfloat16)), dict(dweight=torch.zeros(T, V)),
    dict(dweight=torch.zeros(V, T, dtype=torch.float16), overwrite=True), dict(out_dtype=torch.int8)])
def test_dweight_binding(over):
    reaches_library(dw)
    reaches_library(dw, dweight=torch.zeros(V, T, dtype=torch.bfloat16), overwrite=True)
    with pytest.raises(BAD):
        dw(**over)


def test_scales_may_be_parameters():
    p = torch.nn.Parameter
    reaches_library(lin, x_scale=p(torch.zeros(2, T).t(), requires_grad=False),
                    weight_scale=p(torch.zeros(-(-V // 128), 2), requires_grad=False))


def test_fp8_linear_binding():
    reaches_library(lambda: llp.fp8_linear(torch.zeros(2, 3, 64), torch.zeros(10, 64)))
    for x, w in ((torch.zeros(3, 63), torch.zeros(10, 64)), (torch.zeros(3, 64).half(), torch.zeros(10, 64)),
                 (torch.zeros(3, 64), torch.zeros(10, 64).half()), (torch.zeros(3, 64), torch.zeros(64)),
                 (torch.zeros(()), torch.zeros(10, 64)), (None, torch.zeros(10, 64))):
        with pytest.raises(BAD):
            llp.fp8_linear(x, w)


def part(rows=12, num=8):
    return dict(value=torch.zeros(rows, num), token=torch.zeros(rows, num, dtype=torch.int64), max=torch.zeros(rows),
                sum=torch.zeros(rows, dtype=torch.float64))


def test_candidates_binding():
    z = torch.zeros(12, 1000)
    reaches_library(lambda: llp.beam_candidates(z, 8, out=part()))
    for bad in (dict(num=0), dict(num=65), dict(num=2.0), dict(out=part(11)), dict(out=part(12, 9)),
                dict(out=dict(part(), sum=torch.zeros(12))), dict(out=dict(part(), value=torch.zeros(8, 12).t())),
                dict(status=torch.zeros(1)), dict(world=2)):
        with pytest.raises(BAD):
            llp.beam_candidates(z, **{"num": 8, **bad})
    for t in (z.half(), z[0], z.t()):
        with pytest.raises(BAD):
            llp.beam_candidates(t, 8)


def test_select_binding():
    s = torch.zeros(3, 4)
    reaches_library(lambda: llp.beam_select([part(), part()], s, 8))
    reaches_library(lambda: llp.beam_select([part()], s, finished=torch.zeros(3, 4, dtype=torch.uint8), end_id=5))
    for parts, kw in (([], {}), ([part(11)], {}), ([part(12, 3)], {}), ([part(), part(12, 9)], {}),
                      ([dict(part(), sum=torch.zeros(12))], {}), ([part()], dict(num=9)), ([part()], dict(num=0)),
                      ([part()], dict(finished=torch.zeros(3, 4, dtype=torch.uint8))),
                      ([part()], dict(finished=torch.zeros(3, 4), end_id=1)),
                      ([part()], dict(finished=torch.zeros(4, 3, dtype=torch.uint8).t(), end_id=1)),
                      ([part()], dict(out=dict(token=torch.zeros(3, 4), parent=torch.zeros(3, 4), score=torch.zeros(3, 4)))),
                      ([part()] * 65, {}), (part(), {})):
        with pytest.raises(BAD):
            llp.beam_select(parts, s, **kw)
    for t in (s.double(), s[0], torch.zeros(4, 3).t(), torch.zeros(3, 0), torch.zeros(1, 65)):
        with pytest.raises(BAD):
            llp.beam_select([part()], t)


def test_reorder_binding():
    p = torch.zeros(2, 4, dtype=torch.int32)
    x = torch.zeros(8, 3, 10, 16)
    reaches_library(lambda: llp.beam_reorder(x, p))
    reaches_library(lambda: llp.beam_reorder([x[:, :, :7], torch.zeros(8)], p))
    kv = torch.zeros(8, 2, 3, 10, 16)
    reaches_library(lambda: llp.beam_reorder([kv[:, 0], kv[:, 1], kv[:, 0, :, :0]], p))
    pairs = torch.zeros(8, 6, 16)
    reaches_library(lambda: llp.beam_reorder([pairs[:, ::2], pairs[:, 1::2]], p))
    reaches_library(lambda: llp.beam_reorder(torch.zeros(2, 5).expand(2, 5), p, out=torch.zeros(8, 5)))
    for states, kw in ((torch.zeros(7, 3), {}), (torch.zeros(4, 3), {}), (torch.zeros(1, 3).expand(8, 3), {}),
                       ([x, x], {}), ([x, x[:, :, 1:5]], {}), ([x[:, :, :5], x[:, :, 4:9]], {}),
                       ([kv[:, 0], kv[:, 0:1].reshape(8, 3, 10, 16)], dict(out=[x])),
                       (torch.zeros(8, 4, 6, 10)[:, ::2, ::2, ::2], {}), (x, dict(out=x[:, :, :5])),
                       (x, dict(out=x.to(torch.int64))), (x, dict(out=torch.zeros(9, 3, 10, 16))),
                       (x[:, :, :5], dict(out=x[:, :, 3:8])), (x, dict(status=torch.zeros(1))),
                       ([x, torch.zeros(8, 5)], dict(out=[torch.zeros(8, 3, 10, 16), x.reshape(8, -1)[:, :5]]))):
        with pytest.raises(BAD):
            llp.beam_reorder(states, p, **kw)
    for q in (p.long(), p[0], torch.zeros(4, 2, dtype=torch.int32).t(), torch.zeros(2, 65, dtype=torch.int32)):
        with pytest.raises(BAD):
            llp.beam_reorder(x, q)
