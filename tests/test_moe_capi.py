"""Refusals of the mixture-of-experts operators, at the C ABI and in the binding: every
argument error is found on the host (the fake pointers are never dereferenced), and calls
of size zero return MXQ_OK without a launch."""
import math

import pytest
import torch

import mxfp8_quantization_moe_mx_b200 as mxq
from mxfp8_quantization_moe_mx_b200 import build as mxq_build

OK, NULL, SHAPE, ALIGN, ARG = 0, 1, 2, 3, 4
P, P8, P2 = 0x10000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def L():
    mxq_build.build()
    return mxq.lib()


def _route(L, logits=P, ty=0, T=4, E=64, bias=None, score=0, n=1, top=1, gt=1, k=4, renorm=0, scale=1.0, w=P, i=P):
    return L.moe_route(logits, ty, T, E, bias, score, n, top, gt, k, renorm, scale, w, i, None)


def test_moe_route_argument_errors(L):
    for kw in (dict(ty=2), dict(score=2), dict(score=-1), dict(n=0), dict(n=33, E=66), dict(n=4, top=5),
               dict(n=4, top=0), dict(n=4, gt=0), dict(n=4, gt=3), dict(scale=math.inf), dict(scale=math.nan)):
        assert _route(L, **kw) == ARG, kw
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=3, k=4), dict(n=5, top=1),
               dict(T=2 ** 60)):
        assert _route(L, **kw) == SHAPE, kw
    for kw in (dict(logits=None), dict(w=None), dict(i=None)):
        assert _route(L, **kw) == NULL, kw
    for kw in (dict(logits=P + 1), dict(logits=P2, ty=1), dict(bias=P2), dict(w=P2), dict(i=P2)):
        assert _route(L, **kw) == ALIGN, kw
    assert _route(L, T=0, logits=None, w=None, i=None) == OK


def test_moe_route_backward_argument_errors(L):
    f = L.moe_route_backward
    ok = [P, 0, 4, 64, P, 4, P, 0, 0, 1.0, P, None]

    def go(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    assert go(a1=7) == ARG and go(a7=2) == ARG and go(a9=math.nan) == ARG
    assert go(a2=-1) == SHAPE and go(a3=2000) == SHAPE and go(a5=0) == SHAPE and go(a5=65) == SHAPE
    for i in (0, 4, 6, 10):
        assert go(**{f"a{i}": None}) == NULL
    assert go(a0=P + 1) == ALIGN and go(a4=P2) == ALIGN and go(a6=P2) == ALIGN and go(a10=P + 1) == ALIGN
    assert go(a1=1, a0=P2) == ALIGN and go(a1=1, a10=P2) == ALIGN
    assert f(None, 0, 0, 64, None, 4, None, 0, 0, 1.0, None, None) == OK


def test_moe_plan_argument_errors(L):
    f = L.moe_plan
    assert f(P, -1, 4, P, P, P, P, None) == SHAPE
    assert f(P, 2 ** 31, 4, P, P, P, P, None) == SHAPE
    assert f(P, 8, 0, P, P, P, P, None) == SHAPE
    assert f(P, 8, 1025, P, P, P, P, None) == SHAPE
    assert f(None, 8, 4, P, P, P, P, None) == NULL
    assert f(P, 8, 4, None, P, P, P, None) == NULL
    assert f(P, 8, 4, P, None, P, P, None) == NULL
    assert f(P, 8, 4, P, P, None, P, None) == NULL
    assert L.moe_plan_workspace_bytes(1 << 20, 4) > 0
    assert f(P, 1 << 20, 4, P, P, P, None, None) == NULL
    assert f(P, 8, 4, P2, P, P, P, None) == ALIGN
    assert f(P, 1 << 20, 4, P, P, P, P2, None) == ALIGN
    assert L.moe_plan_workspace_bytes(-1, 4) == -1 and L.moe_plan_workspace_bytes(4, 0) == -1
    assert L.moe_plan_workspace_bytes(8, 4) == 0


def test_rmsnorm_argument_errors(L):
    f = L.rmsnorm_mx_quantize

    def go(x=P, r=None, w=P, ty=0, M=4, D=64, eps=1e-5, ro=None, y=None, q=P, s=P, t=None):
        return f(x, r, w, ty, M, D, eps, ro, y, q, s, t, None)
    for kw in (dict(ty=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)):
        assert go(**kw) == ARG, kw
    for kw in (dict(M=-1), dict(D=48), dict(D=16416), dict(D=-32), dict(M=2 ** 60)):
        assert go(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(q=None), dict(s=None)):
        assert go(**kw) == NULL, kw
    for kw in (dict(x=P8), dict(r=P8), dict(w=P8), dict(ro=P8), dict(y=P8), dict(q=P8), dict(t=P2)):
        assert go(**kw) == ALIGN, kw
    assert go(M=0, x=None, w=None, q=None, s=None) == OK and go(D=0) == OK


def test_rmsnorm_backward_argument_errors(L):
    f = L.rmsnorm_backward

    def go(g=P, h=P, w=P, ty=0, r=P, e=None, M=4, D=64, x=P, d=P, ws=P):
        return f(g, h, w, ty, r, e, M, D, x, d, ws, None)
    assert go(ty=3) == ARG
    for kw in (dict(M=-1), dict(D=40), dict(D=32768)):
        assert go(**kw) == SHAPE, kw
    for kw in (dict(g=None), dict(h=None), dict(w=None), dict(r=None), dict(x=None), dict(d=None), dict(ws=None)):
        assert go(**kw) == NULL, kw
    for kw in (dict(g=P8), dict(h=P8), dict(w=P8), dict(r=P2), dict(e=P8), dict(x=P8), dict(d=P8), dict(ws=P8)):
        assert go(**kw) == ALIGN, kw
    assert go(D=0) == OK
    assert L.rmsnorm_backward_workspace_bytes(4, 40) == -1
    assert L.rmsnorm_backward_workspace_bytes(0, 64) == 0


def test_mxfp4_argument_errors(L):
    f = L.mxfp4_quantize

    def go(x=P, b=1, r=64, c=64, q=P, s=P, sf=None, o=None, G=0):
        return f(x, b, r, c, q, s, sf, o, G, None)
    for kw in (dict(b=-1), dict(r=-1), dict(c=48), dict(G=-1), dict(b=2, G=2, o=P, sf=P), dict(r=2 ** 50, c=2 ** 20)):
        assert go(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(G=2, sf=P), dict(G=2, o=P)):
        assert go(**kw) == NULL, kw
    for kw in (dict(x=P8), dict(q=P8), dict(sf=P8), dict(sf=P, o=P2, G=2)):
        assert go(**kw) == ALIGN, kw
    assert go(r=0, x=None, q=None, s=None) == OK
    d = L.mxfp4_dequantize
    assert d(P, P, 4, 48, P, None) == SHAPE and d(P, P, -4, 64, P, None) == SHAPE
    assert d(None, P, 4, 64, P, None) == NULL and d(P, None, 4, 64, P, None) == NULL
    assert d(P8, P, 4, 64, P, None) == ALIGN and d(P, P, 4, 64, P8, None) == ALIGN
    assert d(None, None, 0, 64, None, None) == OK


def test_mxfp4_grouped_gemm_argument_errors(L):
    f = L.mxfp4_grouped_gemm
    ok = [P, P, P, P, P, 4, 128, 256, 128, P, None]

    def go(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    assert go(8, 64) == SHAPE and go(7, 128) == SHAPE and go(6, -1) == SHAPE and go(5, 70000) == SHAPE
    assert go(6, 2 ** 31) == SHAPE
    for i in (0, 1, 2, 3, 4, 9):
        assert go(i, None) == NULL
    for i in (0, 1, 2, 3, 9):
        assert go(i, P8) == ALIGN
    assert go(4, P2) == ALIGN
    for i in (5, 6, 7, 8):
        assert go(i, 0) == OK


def test_binding_refuses_host_and_wrong_tensors(L):
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    f32 = lambda *s: torch.zeros(*s)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    calls = [
        lambda: mxq.moe_route(x, f32(8, 2), i32(8, 2)),
        lambda: mxq.moe_route(x[0], f32(8, 2), i32(8, 2)),
        lambda: mxq.moe_route(x.double(), f32(8, 2), i32(8, 2)),
        lambda: mxq.moe_route_backward(x, i32(8, 2), f32(8, 2), x),
        lambda: mxq.moe_plan(i32(8), i32(4), i32(8), i32(8)),
        lambda: mxq.rmsnorm_mx_quantize(x, x[0], 1e-5, u8(8, 64), u8(8, 2)),
        lambda: mxq.rmsnorm_backward(x, x, x[0], f32(8), x, f32(64), u8(4096)),
        lambda: mxq.mxfp4_quantize(x, u8(8, 32), u8(8, 2)),
        lambda: mxq.mxfp4_dequantize(u8(8, 32), u8(8, 2), x),
        lambda: mxq.mxfp4_grouped_gemm(u8(8, 64), u8(512), u8(2, 256, 64), u8(4096), i32(2), x),
        lambda: mxq.mxfp4_grouped_gemm(u8(8, 64), u8(512), u8(2, 256, 32), u8(4096), i32(2), x),
    ]
    for call in calls:
        with pytest.raises(mxq.MxqError):
            call()
    with pytest.raises(mxq.MxqError):
        mxq.moe_plan_workspace_bytes(-1, 4)
    with pytest.raises(mxq.MxqError):
        mxq.rmsnorm_backward_workspace_bytes(4, 20)


def test_the_layer_forms_refuse_host_and_misshapen_tensors(L):
    from mxfp8_quantization_moe_mx_b200 import moe
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.route(x, 2), lambda: moe.route(x[0], 2), lambda: moe.plan(torch.zeros(4, dtype=torch.int32), 2),
                 lambda: moe.rmsnorm(x, x[0].float()), lambda: moe.rmsnorm(x, x[0], residual=x[:2]),
                 lambda: moe.rmsnorm(x[0], x[0]), lambda: moe.Mxfp4Experts(x),
                 lambda: moe.Mxfp4Experts(torch.zeros(2, 256, 128, dtype=torch.bfloat16))):
        with pytest.raises(mxq.MxqError):
            call()
