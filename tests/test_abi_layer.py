"""Refusals of the operators around the attention: the C entry points answer
bad arguments before any CUDA work, the binding refuses tensors of the wrong
kind.  (No call here passes the checks: the pointers are not memory.)"""
import ctypes

import pytest
import torch

from sparse_bit_attention_smoothing_b200 import build as sbuild

F, P, LL = ctypes.c_float, ctypes.c_void_p, ctypes.c_longlong
A, B_, M8 = P(0x10000), P(0x20000), P(0x10008)
INVALID, MISALIGNED = -1, -2


@pytest.fixture(scope="module")
def sg():
    sbuild.build()
    import sparse_bit_attention_smoothing_b200 as s
    return s


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def with_(base, **kw):
    d = dict(base)
    assert set(kw) <= set(d)
    d.update(kw)
    return list(d.values())


# ------------------------------------------------------- W8A8, token/channel
QUANT = dict(a=A, dtype=0, rows=4, cols=64, lda=64, codes=A, scales=B_, st=None)
GEMM = dict(xq=A, sx=B_, wq=A, sw=B_, bias=None, y=A, dtype=0, M=4, N=5, K=64, st=None)
LINEAR = dict(x=A, ldx=64, wq=A, sw=B_, bias=None, y=A, dtype=0, M=4, N=5, K=64, ws=A, nb=LL(1 << 20), st=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(a=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(cols=72), INVALID),
    (dict(cols=131072, lda=131072), INVALID), (dict(lda=56), INVALID), (dict(lda=-64), INVALID),
    (dict(rows=2147483647, cols=65536, lda=65536), INVALID), (dict(lda=68), MISALIGNED), (dict(a=M8), MISALIGNED),
    (dict(codes=M8), MISALIGNED), (dict(scales=P(0x20002)), MISALIGNED)])
def test_token_quant(sg, kw, rc):
    assert sg.lib().sagesla_w8a8_token_quant(*with_(QUANT, **kw)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(xq=None), INVALID), (dict(sx=None), INVALID), (dict(wq=None), INVALID), (dict(sw=None), INVALID),
    (dict(y=None), INVALID), (dict(dtype=2), INVALID), (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(K=24), INVALID), (dict(K=131072), INVALID), (dict(M=8388481), INVALID), (dict(N=8388481), INVALID),
    (dict(M=8388480, N=8388480), INVALID), (dict(xq=M8), MISALIGNED),
    (dict(wq=M8), MISALIGNED), (dict(y=M8), MISALIGNED), (dict(sx=P(0x20001)), MISALIGNED),
    (dict(sw=P(0x20002)), MISALIGNED), (dict(bias=P(0x20001)), MISALIGNED)])
def test_token_gemm(sg, kw, rc):
    assert sg.lib().sagesla_w8a8_token_gemm(*with_(GEMM, **kw)) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), INVALID), (dict(ws=None), INVALID), (dict(nb=LL(255)), INVALID), (dict(nb=LL(-1)), INVALID),
    (dict(ldx=32), INVALID), (dict(M=0), INVALID), (dict(K=8), INVALID), (dict(dtype=2), INVALID),
    (dict(ldx=65), MISALIGNED), (dict(x=M8), MISALIGNED), (dict(ws=M8), MISALIGNED), (dict(y=M8), MISALIGNED)])
def test_token_linear(sg, kw, rc):
    assert sg.lib().sagesla_w8a8_token_linear(*with_(LINEAR, **kw)) == rc


def test_token_workspace(sg):
    n = LL(0)
    assert sg.lib().sagesla_w8a8_token_workspace(3, 64, ctypes.byref(n)) == 0 and n.value >= 3 * 64 + 3 * 4
    for M, K in ((0, 64), (1, 0), (1, 72), (1, 131072)):
        assert sg.lib().sagesla_w8a8_token_workspace(M, K, ctypes.byref(n)) == INVALID
    assert sg.lib().sagesla_w8a8_token_workspace(3, 64, None) == INVALID
    assert sg.sagesla_w8a8_token_workspace(3, 64) >= 204


# ---------------------------------------------------------- norm and rotation
S12 = arr(*(512, 128, 64) * 4)
S18 = arr(*(512, 128, 64) * 6)
ROPE = dict(q=A, k=A, gq=A, gk=A, eps=F(1e-6), cos=A, sin=A, pos=None, qo=B_, ko=B_, dtype=0, B=2, N=4, Hq=2, Hk=2,
            d=64, rot=64, T=4, il=1, strides=S12, st=None)
BWD = dict(dqo=A, dko=A, q=A, k=A, gq=A, gk=A, eps=F(1e-6), cos=A, sin=A, pos=None, dq=B_, dk=B_, dgq=B_, dgk=B_,
           dtype=0, B=2, N=4, Hq=2, Hk=2, d=64, rot=64, T=4, il=1, strides=S18, ws=A, nb=LL(1 << 30), st=None)
BAD_ROPE = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(gq=None), INVALID), (dict(gk=None), INVALID),
    (dict(cos=None), INVALID), (dict(sin=None), INVALID), (dict(strides=None), INVALID), (dict(eps=F(-1)), INVALID),
    (dict(eps=F(2)), INVALID), (dict(eps=F(float("nan"))), INVALID), (dict(dtype=3), INVALID), (dict(il=2), INVALID),
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(d=0), INVALID),
    (dict(d=72), INVALID), (dict(d=272), INVALID), (dict(rot=80), INVALID), (dict(rot=8), INVALID), (dict(rot=-16), INVALID),
    (dict(T=0), INVALID), (dict(T=3), INVALID), (dict(B=65536, N=65536, pos=A), INVALID),
    (dict(B=30000, N=30000, Hq=64, pos=A), INVALID), (dict(Hq=65536), INVALID), (dict(q=M8), MISALIGNED),
    (dict(gq=M8), MISALIGNED), (dict(gk=M8), MISALIGNED), (dict(cos=M8), MISALIGNED), (dict(sin=M8), MISALIGNED),
    (dict(pos=P(0x10002)), MISALIGNED)]


@pytest.mark.parametrize("kw,rc", BAD_ROPE + [
    (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(qo=M8), MISALIGNED),
    (dict(strides=arr(512, 128, 60, *(512, 128, 64) * 3)), MISALIGNED),
    (dict(strides=arr(-512, 128, 64, *(512, 128, 64) * 3)), INVALID),
    # rows of an output on top of one another: repeated heads, tokens inside a head, sequences inside a token
    (dict(strides=arr(*(512, 128, 64) * 2, 512, 128, 0, 512, 128, 64)), INVALID),
    (dict(strides=arr(*(512, 128, 64) * 2, 512, 64, 64, 512, 128, 64)), INVALID),
    (dict(strides=arr(*(512, 128, 64) * 3, 64, 128, 64)), INVALID)])
def test_qk_norm_rope(sg, kw, rc):
    assert sg.lib().sagesla_qk_norm_rope(*with_(ROPE, **kw)) == rc


@pytest.mark.parametrize("kw,rc", BAD_ROPE + [
    (dict(dqo=None), INVALID), (dict(dko=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dgq=None), INVALID), (dict(dgk=None), INVALID), (dict(ws=None), INVALID), (dict(ws=M8), MISALIGNED),
    (dict(dqo=M8), MISALIGNED), (dict(dq=M8), MISALIGNED), (dict(dgq=P(0x20002)), MISALIGNED),
    (dict(strides=arr(*(512, 128, 64) * 4, 512, 128, 0, 512, 128, 64)), INVALID)])
def test_qk_norm_rope_bwd(sg, kw, rc):
    assert sg.lib().sagesla_qk_norm_rope_bwd(*with_(BWD, **kw)) == rc


def test_qk_norm_rope_bwd_workspace(sg):
    n = LL(0)
    for a in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, -1, 64), (1, 1, 1, 1, 8), (1, 1, 1, 1, 512)):
        assert sg.lib().sagesla_qk_norm_rope_bwd_workspace(*a, ctypes.byref(n)) == INVALID
    assert sg.lib().sagesla_qk_norm_rope_bwd_workspace(1, 1, 1, 1, 64, None) == INVALID


# ------------------------------------------- linear attention with a decay
DECAY = dict(q=A, k=A, v=A, ld=B_, s0=None, lens=None, scale=F(1), out=A, s1=None, B=2, N=4, H=2, Hk=2, d=64,
             strides=S12, ws=None, nb=LL(0), st=None)
STEP = dict(q=A, k=A, v=A, ld=B_, s0=A, scale=F(1), out=A, s1=A, B=2, H=2, Hk=2, d=64, strides=arr(*(128, 64) * 4), st=None)
BAD_DECAY = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ld=None), INVALID),
    (dict(out=None), INVALID), (dict(strides=None), INVALID), (dict(scale=F(float("inf"))), INVALID),
    (dict(scale=F(float("nan"))), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(H=3), INVALID), (dict(d=96), INVALID), (dict(d=32), INVALID), (dict(B=400, H=400), INVALID),
    (dict(q=M8), MISALIGNED), (dict(k=M8), MISALIGNED), (dict(v=M8), MISALIGNED), (dict(out=M8), MISALIGNED),
    (dict(s0=M8), MISALIGNED), (dict(s1=M8), MISALIGNED), (dict(ld=P(0x20002)), MISALIGNED)]


@pytest.mark.parametrize("kw,rc", BAD_DECAY + [
    (dict(N=0), INVALID), (dict(N=(1 << 30) + 1), INVALID), (dict(lens=P(0x20001)), MISALIGNED),
    (dict(strides=arr(512, 0, 64, *(512, 128, 64) * 3)), INVALID),
    (dict(strides=arr(512, 128, 36, *(512, 128, 64) * 3)), MISALIGNED),
    (dict(strides=arr(*(512, 128, 64) * 3, 512, 64, 64)), INVALID)])
def test_linear_decay(sg, kw, rc):
    assert sg.lib().sagesla_linear_decay(*with_(DECAY, **kw)) == rc


@pytest.mark.parametrize("kw,rc", BAD_DECAY + [
    (dict(s0=None), INVALID), (dict(s1=None), INVALID), (dict(strides=arr(*(128, 64) * 3, 64, 64)), INVALID),
    (dict(strides=arr(128, -64, *(128, 64) * 3)), INVALID), (dict(strides=arr(132, 64, *(128, 64) * 3)), MISALIGNED)])
def test_linear_decay_step(sg, kw, rc):
    assert sg.lib().sagesla_linear_decay_step(*with_(STEP, **kw)) == rc


def test_linear_decay_workspace(sg):
    n = LL(0)
    for a in ((0, 1, 1, 64), (1, 0, 1, 64), (1, 1, 0, 64), (1, 1, 1, 96), (400, 1, 400, 64)):
        assert sg.lib().sagesla_linear_decay_workspace(*a, ctypes.byref(n)) == INVALID
    assert sg.lib().sagesla_linear_decay_workspace(1, 1, 1, 64, None) == INVALID


# ---------------------------------------------------------------- the binding
def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda s: s.sagesla_w8a8_token_quant(t(2, 32)),  # not on a GPU
    lambda s: s.sagesla_w8a8_token_quant(t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_w8a8_token_quant(t(2, 2, 32)),
    lambda s: s.sagesla_w8a8_token_quant(t(32, 2).t()),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 16, dtype=torch.int8), t(4, dtype=torch.float32)),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 32), t(4, dtype=torch.float32)),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 32, dtype=torch.int8), t(4)),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 32, dtype=torch.int8), t(3, dtype=torch.float32)),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 32, dtype=torch.int8), t(4, dtype=torch.float32), bias=t(4, dtype=torch.float16)),
    lambda s: s.sagesla_w8a8_token_linear(t(2, 32), t(4, 32, dtype=torch.int8), t(4, dtype=torch.float32)),
    lambda s: s.sagesla_w8a8_token_gemm(t(2, 32), t(2, dtype=torch.float32), t(4, 32, dtype=torch.int8), t(4, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), t(1, 2, 3, 32), t(64), t(64), t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), None, t(32), None, t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), t(1, 2, 3, 64), t(64), None, t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), None, t(64), None, t(2, 32), t(2, 32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), None, t(64), None, t(2, 32, dtype=torch.float32), t(3, 32, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), None, t(64), None, t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32), pos=t(1, 2, dtype=torch.int64)),
    lambda s: s.sagesla_qk_norm_rope(t(1, 2, 3, 64), None, t(64), None, t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_qk_norm_rope_bwd(t(1, 2, 2, 64), None, t(1, 2, 3, 64), None, t(64), None, t(2, 32, dtype=torch.float32), t(2, 32, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay(t(1, 2, 3, 64), t(1, 2, 3, 64), t(1, 2, 1, 64), t(3, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay(t(1, 2, 3, 64), t(1, 2, 3, 64), t(1, 2, 3, 64), t(2, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay(t(1, 2, 3, 64), t(1, 2, 3, 64), t(1, 2, 3, 64), t(3, dtype=torch.float32), t(1, 3, 64, 64)),
    lambda s: s.sagesla_linear_decay(t(1, 2, 3, 64, dtype=torch.float16), t(1, 2, 3, 64), t(1, 2, 3, 64), t(3, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay_step(t(1, 3, 64), t(1, 3, 64), t(1, 3, 64), t(3, dtype=torch.float32), t(1, 3, 64, 32, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay_step(t(1, 3, 64), t(1, 3, 64), t(1, 2, 64), t(3, dtype=torch.float32), t(1, 3, 64, 64, dtype=torch.float32)),
    lambda s: s.sagesla_linear_decay_step(t(1, 3, 64), t(1, 3, 64), t(1, 3, 64), t(3, dtype=torch.float32), t(1, 3, 64, 64, dtype=torch.float32)),
])
def test_binding_refuses(sg, call):
    with pytest.raises(ValueError):
        call(sg)


@pytest.mark.parametrize("N", [(1 << 30) + 1, (1 << 31) - 1])
def test_linear_decay_workspace_too_long(sg, N):
    n = LL(0)
    assert sg.lib().sagesla_linear_decay_workspace(1, N, 1, 64, ctypes.byref(n)) == INVALID
