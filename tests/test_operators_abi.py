"""Refusals of the router's and the gradients' entry points that need no
GPU: invalid calls return their status before anything is enqueued, and the
binding refuses host tensors."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 20  # 16-byte aligned, never dereferenced by a refused call


@pytest.fixture(scope="module")
def mxq():
    import fp8_mx_activation_amd as m
    if not os.path.exists(m.LIB_PATH):
        from fp8_mx_activation_amd import build
        build.build(verbose=False)
    m.lib()
    return m


def test_route_validation(mxq):
    ok = dict(x=FAKE, dt=1, ld=64, T=4, E=64, K=4, score=0, bias=None, G=1,
              g=1, renorm=1, scale=1.0, ids=FAKE, w=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_route(
            a["x"], a["dt"], a["ld"], a["T"], a["E"], a["K"], a["score"],
            a["bias"], a["G"], a["g"], a["renorm"],
            ctypes.c_float(a["scale"]), a["ids"], a["w"], None)

    assert call(T=0) == 0
    assert call(dt=2) == UNSUPPORTED
    assert call(score=2) == UNSUPPORTED
    assert call(E=1025, ld=1025) == UNSUPPORTED
    assert call(G=128, E=128, ld=128) == INVALID       # K > E / G * g
    assert call(G=128, g=128, E=128, ld=128) == UNSUPPORTED
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=65), dict(G=0),
                dict(G=3), dict(g=0), dict(G=8, g=9), dict(ld=63),
                dict(x=None), dict(ids=None), dict(w=None),
                dict(G=32, g=1, K=4), dict(E=2, K=3)):
        assert call(**bad) == INVALID, bad


def test_route_backward_validation(mxq):
    ok = dict(g=FAKE, x=FAKE, dt=1, ld=64, ids=FAKE, T=4, E=64, K=4, score=0,
              renorm=1, scale=1.0, out=FAKE, ldo=64)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_route_backward(
            a["g"], a["x"], a["dt"], a["ld"], a["ids"], a["T"], a["E"],
            a["K"], a["score"], a["renorm"], ctypes.c_float(a["scale"]),
            a["out"], a["ldo"], None)

    assert call(T=0) == 0
    assert call(dt=5) == UNSUPPORTED
    assert call(score=7) == UNSUPPORTED
    assert call(E=1025, ld=1025, ldo=1025) == UNSUPPORTED
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=65), dict(ld=63),
                dict(ldo=63), dict(g=None), dict(x=None), dict(ids=None),
                dict(out=None)):
        assert call(**bad) == INVALID, bad


def test_scatter_rows_backward_validation(mxq):
    ok = dict(r=FAKE, dt=0, ld=64, rows=8, s=FAKE, T=4, K=2, H=64, x=FAKE,
              ldx=64, xdt=0)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_scatter_rows_backward(
            a["r"], a["dt"], a["ld"], a["rows"], a["s"], a["T"], a["K"],
            a["H"], a["x"], a["ldx"], a["xdt"], None)

    assert call(T=0) == 0
    assert call(dt=2) == UNSUPPORTED
    assert call(xdt=2) == UNSUPPORTED
    for bad in (dict(T=-1), dict(K=-1), dict(K=65), dict(H=0), dict(H=60),
                dict(rows=-1), dict(rows=1 << 31), dict(ld=56),
                dict(ld=68), dict(ldx=56), dict(ldx=68), dict(r=None),
                dict(r=FAKE + 8), dict(x=None), dict(x=FAKE + 2),
                dict(s=None)):
        assert call(**bad) == INVALID, bad


def test_combine_backward_validation(mxq):
    ok = dict(g=FAKE, dt=0, ldg=64, y=FAKE, ldy=64, rows=8, s=FAKE, w=FAKE,
              T=4, K=2, H=64, gy=FAKE, ldgy=64, gw=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_combine_backward(
            a["g"], a["dt"], a["ldg"], a["y"], a["ldy"], a["rows"], a["s"],
            a["w"], a["T"], a["K"], a["H"], a["gy"], a["ldgy"], a["gw"],
            None)

    assert call(T=0) == 0
    assert call(K=0) == 0
    assert call(dt=2) == UNSUPPORTED
    assert call(H=32776, ldg=32776, ldy=32776, ldgy=32776) == UNSUPPORTED
    for bad in (dict(T=-1), dict(K=-1), dict(K=65), dict(H=0), dict(H=60),
                dict(rows=-1), dict(g=None), dict(g=FAKE + 4), dict(ldg=56),
                dict(ldg=68), dict(y=None), dict(y=FAKE + 2), dict(ldy=56),
                dict(ldy=68), dict(s=None), dict(w=None),
                dict(gy=None, gw=None), dict(gy=FAKE + 8), dict(ldgy=56),
                dict(ldgy=68)):
        assert call(**bad) == INVALID, bad


def test_binding_refuses_host_tensors(mxq):
    l = torch.zeros((4, 16))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((4, 2))
    y = torch.zeros((8, 64), dtype=torch.bfloat16)
    g = torch.zeros((4, 64), dtype=torch.bfloat16)
    for c in (lambda: mxq.moe_route(l, 2),
              lambda: mxq.moe_route_backward(w, l, ids),
              lambda: mxq.moe_scatter_rows_backward(y, ids),
              lambda: mxq.moe_combine_backward(g, y, ids, w)):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            c()


def test_expert_matmul_validation(mxq):
    ok = dict(q=FAKE, ldq=256, s=FAKE, lds=2, rows=8, fmt=0, w=FAKE, ws=FAKE,
              E=2, N=256, H=256, off=FAKE, cnt=FAKE, bias=None, act=0,
              res=None, ldr=0, m=4, out=FAKE, ldo=256)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_expert_matmul(
            a["q"], a["ldq"], a["s"], a["lds"], a["rows"], a["fmt"], a["w"],
            a["ws"], a["E"], a["N"], a["H"], a["off"], a["cnt"], a["bias"],
            a["act"], a["res"], a["ldr"], a["m"], a["out"], a["ldo"], None)

    assert call(rows=0) == 0
    assert call(fmt=2) == UNSUPPORTED
    assert call(act=3) == UNSUPPORTED
    assert call(H=32896, ldq=32896, lds=257) == UNSUPPORTED
    assert call(ldq=(1 << 22) + 16) == UNSUPPORTED
    for bad in (dict(E=0), dict(E=1025), dict(N=0), dict(H=0), dict(H=192),
                dict(H=16, fmt=1), dict(rows=-1), dict(rows=1 << 31),
                dict(m=-1), dict(N=255, act=2), dict(N=254),
                dict(N=260, act=2, ldo=127), dict(q=None), dict(s=None),
                dict(w=None), dict(ws=None), dict(off=None), dict(cnt=None),
                dict(out=None), dict(q=FAKE + 8), dict(ldq=264),
                dict(ldq=240), dict(lds=1), dict(w=FAKE + 8),
                dict(out=FAKE + 4), dict(ldo=252), dict(ldo=258),
                dict(res=FAKE + 4, ldr=256), dict(res=FAKE, ldr=252),
                dict(res=FAKE, ldr=258)):
        assert call(**bad) == INVALID, bad


def test_expert_matmul_quant_validation(mxq):
    ok = dict(q=FAKE, ldq=256, s=FAKE, lds=2, rows=8, fmt=0, w=FAKE, ws=FAKE,
              E=2, N=256, H=256, off=FAKE, cnt=FAKE, bias=None, act=0, m=4,
              of=0, out=FAKE, ldo=256, so=FAKE, ldso=8)

    def call(**kw):
        a = dict(ok, **kw)
        return mxq.lib().moe_expert_matmul_quant(
            a["q"], a["ldq"], a["s"], a["lds"], a["rows"], a["fmt"], a["w"],
            a["ws"], a["E"], a["N"], a["H"], a["off"], a["cnt"], a["bias"],
            a["act"], a["m"], a["of"], a["out"], a["ldo"], a["so"],
            a["ldso"], None)

    assert call(rows=0) == 0
    assert call(of=2) == UNSUPPORTED
    for bad in (dict(N=192), dict(N=128, act=2), dict(N=48, of=1),
                dict(so=None), dict(out=None), dict(out=FAKE + 8),
                dict(ldo=264), dict(ldo=240), dict(ldso=1),
                dict(of=1, ldso=7)):
        assert call(**bad) == INVALID, bad


def test_expert_matmul_refuses_row_counts_near_int32(mxq):
    """Row counts are rounded up to whole tiles in 32 bits."""
    def call(rows):
        return mxq.lib().moe_expert_matmul(
            FAKE, 256, FAKE, 2, rows, 0, FAKE, FAKE, 2, 256, 256, FAKE, FAKE,
            None, 0, None, 0, 4, FAKE, 256, None)

    assert call((1 << 31) - (1 << 16) + 1) == UNSUPPORTED
    assert call((1 << 31) - 1) == UNSUPPORTED
