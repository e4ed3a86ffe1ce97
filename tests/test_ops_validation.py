"""The operators around the linear log-prob refuse malformed calls before anything reaches a
device: the C ABI with its documented status, the binding with ValueError or TypeError. Struct
layouts and constants match the header. Runs on the CPU."""
import ctypes as C
import os
import re
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
STRUCTS = ["llp_quant_request", "llp_int8_request", "llp_policy_request", "llp_policy_out",
           "llp_pref_request", "llp_pref_out", "llp_embedding_request"]


def test_structs_and_constants_match_the_header(tmp_path):
    names = ["LLP_INT8_COLUMNS", "LLP_KL_K1", "LLP_KL_K2", "LLP_KL_K3", "LLP_REDUCE_TOKEN_MEAN",
             "LLP_REDUCE_SEQ_MEAN", "LLP_REDUCE_SUM", "LLP_LOG_RATIO_MAX", "LLP_POLICY_STATS",
             "LLP_PREF_SIGMOID", "LLP_PREF_HINGE", "LLP_PREF_IPO",
             "LLP_STATUS_TOKEN_OUT_OF_RANGE", "LLP_STATUS_VALUE_NOT_FINITE"]
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
def vocab(v, V=1000, Vr=1000):
    v.offset, v.local_size, v.real_vocab, v.padded_vocab, v.rank, v.world = 0, V, Vr, V, 0, 1


def quant(**over):
    r = A.llp_quant_request(FAKE, A.LLP_DTYPE_BF16, 0, 256, 10, 256, FAKE, 256, FAKE)
    for k, v in over.items():
        setattr(r, k, v)
    return A.load().llp_quantize_rows(C.byref(r), None)


def int8(ws=1 << 40, wsp=FAKE, out=None, **over):
    r = A.llp_int8_request()
    r.hidden, r.hidden_stride, r.hidden_scale = FAKE, 256, FAKE
    r.weight, r.weight_stride, r.weight_scale = FAKE, 256, FAKE
    r.hidden_size, r.target_ids, r.temperature, r.flags = 256, FAKE, 0.7, 1
    vocab(r.vocab)
    r.layout.num_tokens = 100
    _set(r, over)
    o = A.llp_partials(FAKE, FAKE, FAKE, FAKE, FAKE) if out is None else out
    return A.load().llp_forward_int8(C.byref(r), C.byref(o), wsp, ws, None)


def _set(r, over):
    for k, v in over.items():
        if k in ("T", "seqs", "cu", "mask"):
            setattr(r.layout, dict(T="num_tokens", seqs="num_seqs", cu="cu_seqlens", mask="loss_mask")[k], v)
        elif k in ("V", "Vr"):
            vocab(r.vocab, V=over.get("V", 1000), Vr=over.get("Vr", over.get("V", 1000)))
        else:
            setattr(r, k, v)


def policy(ws=1 << 30, wsp=FAKE, out=None, **over):
    r = A.llp_policy_request()
    r.logp = r.old_logp = r.advantages = r.ref_logp = r.entropy = FAKE
    r.clip_low, r.clip_high, r.kl_coef, r.entropy_coef = 0.2, 0.2, 0.1, 0.1
    r.kl_kind, r.reduction = A.LLP_KL_K3, A.LLP_REDUCE_TOKEN_MEAN
    r.layout.num_tokens, r.layout.num_seqs, r.layout.cu_seqlens = 100, 4, FAKE
    _set(r, over)
    o = A.llp_policy_out(FAKE, FAKE, None, FAKE, FAKE) if out is None else out
    return A.load().llp_policy_loss(C.byref(r), C.byref(o), wsp, ws, None)


def pref(ws=1 << 30, wsp=FAKE, out=None, **over):
    r = A.llp_pref_request()
    r.logp = r.ref_logp = FAKE
    r.beta, r.kind, r.reduction = 0.1, A.LLP_PREF_SIGMOID, A.LLP_REDUCE_TOKEN_MEAN
    r.layout.num_tokens, r.layout.num_seqs, r.layout.cu_seqlens = 100, 4, FAKE
    _set(r, over)
    o = A.llp_pref_out(FAKE, FAKE, FAKE, FAKE, None, FAKE) if out is None else out
    return A.load().llp_preference_loss(C.byref(r), C.byref(o), wsp, ws, None)


def emb(backward=False, ptr=FAKE, out=FAKE, dt=A.LLP_DTYPE_BF16, ld=64, ldo=64, ws=1 << 40, wsp=FAKE, **over):
    r = A.llp_embedding_request()
    r.token_ids, r.num_tokens, r.hidden_size, r.scale = FAKE, 10, 64, 1.0
    vocab(r.vocab)
    _set(r, over)
    lib = A.load()
    if backward:
        return lib.llp_embedding_backward(C.byref(r), ptr, dt, ld, out, ldo, wsp, ws, None)
    return lib.llp_embedding(C.byref(r), ptr, dt, ld, out, ldo, None)


NAN, INF = float("nan"), float("inf")


@needs_lib
@pytest.mark.parametrize("call,over,want", [
    (quant, dict(rows=-1), INV), (quant, dict(rows=1 << 31), INV), (quant, dict(cols=0), INV),
    (quant, dict(cols=(1 << 20) + 1), INV), (quant, dict(x_dtype=7), INV), (quant, dict(x_stride=255), INV),
    (quant, dict(q_stride=240), INV), (quant, dict(q_stride=264), INV), (quant, dict(cols=129, q_stride=128), INV),
    (quant, dict(x=None), INV), (quant, dict(q=None), INV), (quant, dict(scale=None), INV),
    (quant, dict(x=FAKE + 1), INV), (quant, dict(q=FAKE + 8), INV),
    (int8, dict(T=-1), INV), (int8, dict(T=1 << 23), UNS), (int8, dict(hidden_size=0), INV),
    (int8, dict(hidden_size=64, hidden_stride=64, weight_stride=64), UNS),
    (int8, dict(hidden_size=1 << 17, hidden_stride=1 << 17, weight_stride=1 << 17), UNS),
    (int8, dict(hidden_stride=128), INV), (int8, dict(weight_stride=264), INV),
    (int8, dict(hidden_stride=1 << 24), UNS), (int8, dict(weight_stride=1 << 24), UNS),
    (int8, dict(T=1 << 20, hidden_stride=2048), UNS), (int8, dict(V=1 << 23), UNS),
    (int8, dict(hidden=None), INV), (int8, dict(hidden_scale=None), INV), (int8, dict(weight=None), INV),
    (int8, dict(weight_scale=None), INV), (int8, dict(weight_scale=FAKE + 2), INV), (int8, dict(hidden_scale=FAKE + 1), INV),
    (int8, dict(hidden=FAKE + 8), INV), (int8, dict(weight=FAKE + 8), INV), (int8, dict(target_ids=None), INV),
    (int8, dict(bias=FAKE, bias_dtype=9), INV), (int8, dict(bias=FAKE + 2, bias_dtype=2), INV), (int8, dict(bias=FAKE + 1, bias_dtype=1), INV),
    (int8, dict(temperature=0.0), INV), (int8, dict(temperature=NAN), INV), (int8, dict(flags=2), INV),
    (int8, dict(ws=100), INV), (int8, dict(wsp=None), INV), (int8, dict(wsp=FAKE + 16), INV),
    (int8, dict(out=A.llp_partials(FAKE, FAKE, FAKE, None, FAKE)), INV),
    (int8, dict(cu=FAKE, seqs=-1), INV),
    (int8, dict(T=1 << 20, V=1 << 21, hidden_size=128), UNS),       # 2^25 tiles, each a workgroup
    (policy, dict(T=-1), INV), (policy, dict(T=1 << 31), INV), (policy, dict(seqs=-1), INV), (policy, dict(seqs=(1 << 23) + 1), UNS),
    (policy, dict(reduction=0), INV), (policy, dict(reduction=4), INV), (policy, dict(clip_low=-0.1), INV),
    (policy, dict(clip_low=1.1), INV), (policy, dict(clip_low=NAN), INV), (policy, dict(clip_high=-0.1), INV),
    (policy, dict(clip_high=INF), INV), (policy, dict(dual_clip=1.0), INV), (policy, dict(dual_clip=-2.0), INV),
    (policy, dict(dual_clip=NAN), INV), (policy, dict(kl_coef=NAN), INV), (policy, dict(entropy_coef=INF), INV),
    (policy, dict(kl_kind=0), INV), (policy, dict(ref_logp=None), INV), (policy, dict(entropy=None), INV),
    (policy, dict(logp=None), INV), (policy, dict(old_logp=None), INV), (policy, dict(advantages=None), INV),
    (policy, dict(reduction=2, cu=None), INV), (policy, dict(reduction=2, seqs=0), INV),
    (policy, dict(reduction=3, denominator=FAKE), INV), (policy, dict(T=9000, ws=16), INV), (policy, dict(T=9000, wsp=None), INV),
    (policy, dict(out=A.llp_policy_out(None, FAKE, None, FAKE, FAKE)), INV),
    (policy, dict(entropy=None, entropy_coef=0.0), INV),           # dentropy without entropy
    (pref, dict(T=-1), INV), (pref, dict(cu=None), INV), (pref, dict(seqs=3), INV), (pref, dict(seqs=(1 << 23) + 2), UNS), (pref, dict(seqs=0), INV),
    (pref, dict(logp=None), INV), (pref, dict(kind=0), INV), (pref, dict(kind=4), INV), (pref, dict(reduction=2), INV),
    (pref, dict(beta=0.0), INV), (pref, dict(beta=NAN), INV), (pref, dict(gamma=INF), INV),
    (pref, dict(kind=3, gamma=0.5), INV), (pref, dict(label_smoothing=1.0), INV),
    (pref, dict(label_smoothing=-0.1), INV), (pref, dict(kind=2, label_smoothing=0.1), INV),
    (pref, dict(T=9000, ws=8), INV), (pref, dict(T=9000, wsp=FAKE + 8), INV),
    (pref, dict(out=A.llp_pref_out(None, None, None, None, None, None)), INV),
    (emb, dict(num_tokens=-1), INV), (emb, dict(num_tokens=1 << 23), UNS), (emb, dict(V=1 << 23), UNS),
    (emb, dict(hidden_size=0), INV), (emb, dict(hidden_size=60), UNS), (emb, dict(hidden_size=(1 << 20) + 8), UNS),
    (emb, dict(token_ids=None), INV), (emb, dict(scale=NAN), INV), (emb, dict(flags=2), INV), (emb, dict(dt=0), INV),
    (emb, dict(ld=56), INV), (emb, dict(ld=68), INV), (emb, dict(ldo=60), INV), (emb, dict(ptr=None), INV),
    (emb, dict(ptr=FAKE + 8), INV), (emb, dict(out=None), INV), (emb, dict(out=FAKE + 4), INV),
    (emb, dict(backward=True, flags=1), INV), (emb, dict(backward=True, ld=60), INV),
    (emb, dict(backward=True, out=None), INV), (emb, dict(backward=True, ptr=None), INV),
    (emb, dict(backward=True, ldo=66), INV), (emb, dict(backward=True, ws=64), INV),
    (emb, dict(backward=True, wsp=FAKE + 128), INV)])
def test_abi_refuses(call, over, want):
    assert call(**over) == want, A.load().llp_last_error()


@needs_lib
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="a GPU is present: the pointers are not real")
@pytest.mark.parametrize("call,kw", [(quant, {}), (int8, {}), (policy, {}), (pref, {}), (emb, {}),
                                     (emb, dict(backward=True, flags=2))])
def test_abi_accepts_well_formed_up_to_the_device(call, kw):
    st = call(**kw)
    assert st in (A.LLP_ERR_INVALID_ARGUMENT, A.LLP_ERR_HIP)
    msg = A.load().llp_last_error()
    assert b"llp_open" in msg or b"hipGetDevice" in msg


@needs_lib
def test_null_requests():
    lib, n = A.load(), C.c_size_t(0)
    for st in (lib.llp_quantize_rows(None, None), lib.llp_forward_int8(None, None, None, 0, None),
               lib.llp_policy_loss(None, None, None, 0, None), lib.llp_preference_loss(None, None, None, 0, None),
               lib.llp_embedding(None, None, 1, 8, None, 8, None),
               lib.llp_embedding_backward(None, None, 1, 8, None, 8, None, 0, None),
               lib.llp_int8_workspace_bytes(None, C.byref(n)), lib.llp_policy_workspace_bytes(None, C.byref(n)),
               lib.llp_preference_workspace_bytes(None, C.byref(n)),
               lib.llp_embedding_workspace_bytes(None, C.byref(n))):
        assert st == INV


# ---- Binding --------------------------------------------------------------------------------
T, H, V, P = 12, 128, 40, 3


def f32(*s):
    return torch.zeros(*s)


def i64(n):
    return torch.zeros(n, dtype=torch.int64)


def cu(*v):
    return torch.tensor(v, dtype=torch.int32)


def b_quant(x=f32(T, H), **kw):
    return llp.quantize_rows(x, **kw)


def b_int8(hidden=torch.zeros(T, H, dtype=torch.int8), hs=f32(T), weight=torch.zeros(V, H, dtype=torch.int8),
           ws=f32(V), tg=i64(T), temperature=0.7, **kw):
    return llp.forward_int8(hidden, hs, weight, ws, tg, temperature=temperature, **kw)


def b_policy(logp=f32(T), old=f32(T), adv=f32(T), **kw):
    return llp.policy_grads(logp, old, adv, **kw)


def b_pref(logp=f32(T), c=cu(0, 1, 2, 3, 4, 5, T), **kw):
    return llp.preference_grads(logp, c, **kw)


def b_embed(ids=i64(T), w=torch.zeros(V, H, dtype=torch.bfloat16), **kw):
    return llp.embedding_forward(ids, w, **kw)


def b_egrad(ids=i64(T), dout=torch.zeros(T, H, dtype=torch.bfloat16), **kw):
    return llp.embedding_backward(ids, dout, **kw)


u8 = torch.ones(T, dtype=torch.uint8)
PO = dict(loss=f32(1), stats=f32(8), dlogp=f32(T), dentropy=f32(T))
QO = dict(loss=f32(1), pair_loss=f32(P), chosen=f32(P), rejected=f32(P), dlogp=f32(T))


@pytest.mark.parametrize("call,kw", [
    (b_quant, dict(x=[1])), (b_quant, dict(x=f32(T))), (b_quant, dict(x=torch.zeros(T, H, dtype=torch.float16))),
    (b_quant, dict(x=f32(H, T).t())), (b_quant, dict(x=f32(T, 0))),
    (b_quant, dict(out=(torch.zeros(T, H, dtype=torch.int8), f32(T - 1)))),
    (b_quant, dict(x=f32(T, 130), out=(torch.zeros(T, 130, dtype=torch.int8), f32(T)))),
    (b_int8, dict(hidden=f32(T, H))), (b_int8, dict(hidden=None)), (b_int8, dict(hs=f32(T - 1))),
    (b_int8, dict(hs=f32(T, 1))), (b_int8, dict(weight=torch.zeros(V, H + 128, dtype=torch.int8))),
    (b_int8, dict(ws=f32(V + 1))), (b_int8, dict(ws=f32(V).double())), (b_int8, dict(tg=i64(T + 1))),
    (b_int8, dict(bias=f32(V - 1))), (b_int8, dict(bias=torch.zeros(V, dtype=torch.int8))),
    (b_int8, dict(loss_mask=u8[:-1])), (b_int8, dict(loss_mask=u8.bool())), (b_int8, dict(world=2)),
    (b_int8, dict(out=dict(target_logit=f32(T), in_range=u8, lse=f32(T), entropy=None, logp=f32(T)))),
    (b_int8, dict(workspace=f32(100))), (b_int8, dict(status=f32(1))),
    (b_policy, dict(logp=f32(T).double())), (b_policy, dict(logp=f32(T, 1))), (b_policy, dict(logp=None)),
    (b_policy, dict(old=f32(T + 1))), (b_policy, dict(adv=f32(T - 1))), (b_policy, dict(adv=f32(2 * T)[::2])),
    (b_policy, dict(ref_logp=f32(T - 1))), (b_policy, dict(entropy=f32(T + 2))), (b_policy, dict(loss_mask=u8.bool())),
    (b_policy, dict(cu_seqlens=torch.zeros(3))), (b_policy, dict(cu_seqlens=cu())), (b_policy, dict(kl="k4")),
    (b_policy, dict(reduction="mean")), (b_policy, dict(reduction="seq_mean")), (b_policy, dict(kl_coef=0.1)),
    (b_policy, dict(entropy_coef=0.1)), (b_policy, dict(denominator=f32(2))), (b_policy, dict(denominator=3.0)),
    (b_policy, dict(dloss=f32(1).double())), (b_policy, dict(out=dict(PO, dlogp=f32(T - 1)))),
    (b_policy, dict(out=dict(PO, stats=f32(7)))), (b_policy, dict(entropy=f32(T), out=dict(PO, dentropy=f32(1)))),
    (b_pref, dict(logp=f32(T, 1))), (b_pref, dict(c=cu(0, 4, 8, T))), (b_pref, dict(c=cu(0))),
    (b_pref, dict(c=torch.zeros(7, dtype=torch.int64))), (b_pref, dict(c=None)), (b_pref, dict(ref_logp=f32(T - 1))),
    (b_pref, dict(loss_mask=u8[1:])), (b_pref, dict(pair_weight=f32(P + 1))), (b_pref, dict(kind="dpo")),
    (b_pref, dict(reduction="token_mean")), (b_pref, dict(dloss=f32(2))), (b_pref, dict(out=dict(QO, chosen=f32(P + 1)))),
    (b_pref, dict(out=dict(QO, dlogp=f32(T + 1)))),
    (b_embed, dict(ids=torch.zeros(T, dtype=torch.int32))), (b_embed, dict(ids=i64(T).reshape(3, 4))),
    (b_embed, dict(w=torch.zeros(V, H, dtype=torch.float16))), (b_embed, dict(w=f32(H, V).t())),
    (b_embed, dict(token_mask=u8[1:])), (b_embed, dict(out=f32(T, H))), (b_embed, dict(world=2)),
    (b_embed, dict(out=torch.zeros(T - 1, H, dtype=torch.bfloat16))),
    (b_egrad, dict()), (b_egrad, dict(local_size=-1)), (b_egrad, dict(dweight=f32(V, H + 8))),
    (b_egrad, dict(dweight=torch.zeros(V, H, dtype=torch.bfloat16))), (b_egrad, dict(local_size=V + 1, dweight=f32(V, H))),
    (b_egrad, dict(ids=i64(T - 1), local_size=V)), (b_egrad, dict(dout=f32(H, T).t(), local_size=V)),
    (b_egrad, dict(dout=torch.zeros(T, H, dtype=torch.float16), local_size=V)),
    (b_egrad, dict(local_size=V, workspace=f32(8)))])
def test_binding_refuses(call, kw):
    with pytest.raises(BAD):
        call(**kw)


@pytest.mark.parametrize("call,kw", [
    (b_quant, {}), (b_int8, dict(loss_mask=u8, bias=f32(V), status=torch.zeros(1, dtype=torch.int32))),
    (b_policy, dict(ref_logp=f32(T), entropy=f32(T), kl_coef=0.1, entropy_coef=0.1, loss_mask=u8,
                    cu_seqlens=cu(0, T), reduction="seq_mean", denominator=f32(1), dloss=f32(1), out=PO)),
    (b_pref, dict(ref_logp=f32(T), pair_weight=f32(P), out=QO)), (b_embed, dict(token_mask=u8)),
    (b_egrad, dict(local_size=V)), (b_egrad, dict(dweight=f32(V, H)))])
def test_binding_needs_a_gpu_tensor(call, kw):
    # Well formed, on the CPU: refused before a host pointer could reach a kernel.
    with pytest.raises(RuntimeError) as e:
        call(**kw)
    assert not isinstance(e.value, BAD)


def test_names_are_public():
    for n in ("quantize_rows", "forward_int8", "policy_grads", "policy_loss", "preference_grads", "preference_loss",
              "embedding_forward", "embedding_backward", "embedding"):
        assert n in llp.__all__ and callable(getattr(llp, n))
    src = open(HEADER).read()
    for n in re.findall(r"\bllp_\w+(?=\()", src):
        assert n in A.SIGNATURES
