"""Refusals of the entry points of the balance loss and of the microscaled
4-bit floats that need no GPU: invalid calls return their status before
anything is enqueued, and the binding refuses host tensors."""
import os

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
FAKE = 1 << 20  # 16-byte aligned, never dereferenced by a refused call


@pytest.fixture(scope="module")
def mxq():
    import fp8_mx_activation_amd as m
    if not os.path.exists(m.LIB_PATH):
        from fp8_mx_activation_amd import build
        build.build(verbose=False)
    m.lib()
    return m


def caller(fn, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return fn(*{**ok, **kw}.values(), None)
    return call


def test_balance_loss(mxq):
    call = caller(mxq.lib().moe_balance_loss, dict(
        x=FAKE, dt=1, ld=64, ids=FAKE, T=4000, E=64, K=4, score=0, off=FAKE,
        lens=None, S=3, loss=FAKE, z=None, counts=FAKE, probs=FAKE, ws=FAKE,
        size=1 << 30))
    assert call(dt=2) == UNSUPPORTED
    assert call(score=2) == UNSUPPORTED
    assert call(E=1025, ld=1025) == UNSUPPORTED
    assert call(T=1 << 30, K=2) == UNSUPPORTED
    assert call(S=(1 << 31) - 1) == UNSUPPORTED
    need = mxq.moe_balance_loss_workspace_bytes(4000, 64, 3)
    assert need > 0 and call(size=need - 1) == WORKSPACE
    assert call(T=1 << 31, K=1) == UNSUPPORTED
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=65),
                dict(S=0), dict(off=None), dict(ld=63), dict(x=None),
                dict(ids=None), dict(loss=None), dict(counts=None),
                dict(probs=None), dict(ws=None), dict(ws=FAKE + 8)):
        assert call(**bad) == INVALID, bad


def test_balance_loss_workspace(mxq):
    f = mxq.moe_balance_loss_workspace_bytes
    assert f(256, 256, 1) == 0 and f(1024, 16, 1000) == 0
    assert f(257, 256, 1) > 0 and f(1025, 16, 1) > 0
    assert f(0, 8, 1) == 0 and f(-1, 8, 1) == 0 and f(9, 1025, 1) == 0
    # no more with more tokens, once every block has some
    assert f(1 << 20, 256, 4) == f(1 << 30, 256, 4) < 1 << 21
    assert f(1 << 20, 256, 5) > f(1 << 20, 256, 4)


def test_balance_loss_backward(mxq):
    call = caller(mxq.lib().moe_balance_loss_backward, dict(
        g=FAKE, gz=FAKE, x=FAKE, dt=1, ld=64, counts=FAKE, T=4000, E=64,
        score=0, off=FAKE, lens=None, S=3, add=FAKE, lda=64, out=FAKE,
        ldo=64))
    assert call(T=0) == 0
    assert call(dt=2) == UNSUPPORTED
    assert call(score=2) == UNSUPPORTED
    assert call(E=1025, ld=1025, lda=1025, ldo=1025) == UNSUPPORTED
    assert call(T=1 << 31) == UNSUPPORTED
    for bad in (dict(T=-1), dict(E=0), dict(S=0),
                dict(off=None), dict(ld=63), dict(lda=63), dict(ldo=63),
                dict(x=None), dict(out=None), dict(counts=None),
                dict(g=None, gz=None)):
        assert call(**bad) == INVALID, bad


def test_quant_rows(mxq):
    call = caller(mxq.lib().mxfp4_quant_rows, dict(
        x=FAKE, dt=0, ldx=64, rows=8, H=64, rule=0, q=FAKE, ldq=32, s=FAKE,
        lds=2))
    assert call(rows=0) == 0
    assert call(dt=2) == UNSUPPORTED
    assert call(rule=2) == UNSUPPORTED
    # one row to a block of 256 threads: 2^32 of them
    assert call(rows=1 << 24, H=8192, ldx=8192, ldq=4096, lds=256) == \
        UNSUPPORTED
    for bad in (dict(rows=-1), dict(H=0), dict(H=48), dict(ldx=56),
                dict(ldx=68), dict(ldq=16), dict(ldq=40), dict(lds=1),
                dict(x=None), dict(x=FAKE + 8), dict(q=None),
                dict(q=FAKE + 4), dict(s=None)):
        assert call(**bad) == INVALID, bad


def test_scatter(mxq):
    call = caller(mxq.lib().moe_scatter_quant_mxfp4, dict(
        x=FAKE, ldx=64, T=8, H=64, src=FAKE, K=2, rule=0, q=FAKE, ldq=32,
        s=FAKE, lds=2, rows=16))
    assert call(T=0) == 0 and call(K=0) == 0 and call(rows=0) == 0
    assert call(rule=2) == UNSUPPORTED
    assert call(H=32800, ldx=32800, ldq=16400, lds=1025) == UNSUPPORTED
    assert call(T=1 << 26) == UNSUPPORTED
    for bad in (dict(T=-1), dict(H=0), dict(H=48), dict(K=-1), dict(K=65),
                dict(rows=-1), dict(rows=1 << 31), dict(ldx=56),
                dict(ldx=68), dict(ldq=16), dict(ldq=40), dict(lds=1),
                dict(x=None), dict(x=FAKE + 8), dict(src=None), dict(q=None),
                dict(q=FAKE + 4), dict(s=None)):
        assert call(**bad) == INVALID, bad


def test_back(mxq):
    call = caller(mxq.lib().mxfp4_to_e4m3, dict(
        q=FAKE, ldq=32, rows=8, H=64, out=FAKE, ldo=64))
    assert call(rows=0) == 0
    for bad in (dict(rows=-1), dict(H=0), dict(H=48), dict(ldq=16),
                dict(ldq=40), dict(ldo=48), dict(ldo=72), dict(q=None),
                dict(q=FAKE + 8), dict(out=None), dict(out=FAKE + 8)):
        assert call(**bad) == INVALID, bad
    call = caller(mxq.lib().upscale_mxfp4_to_bf16, dict(
        q=FAKE, ldq=32, s=FAKE, lds=2, rows=8, H=64, out=FAKE, ldo=64))
    assert call(rows=0) == 0
    for bad in (dict(rows=-1), dict(H=0), dict(H=48), dict(ldq=16),
                dict(ldq=40), dict(lds=1), dict(ldo=56), dict(ldo=68),
                dict(q=None), dict(s=None), dict(q=FAKE + 8), dict(out=None),
                dict(out=FAKE + 8)):
        assert call(**bad) == INVALID, bad


@pytest.mark.parametrize("fmt,pay", [(2, 64), (1, 128)])
def test_expert_matmul(mxq, fmt, pay):
    call = caller(mxq.lib().moe_expert_matmul_mxfp4, dict(
        q=FAKE, ldq=pay, s=FAKE, lds=4, rows=8, fmt=fmt, w=FAKE, ws=FAKE,
        ldws=4, E=4, N=64, H=128, off=FAKE, counts=FAKE, bias=None, act=0,
        res=None, ldr=0, m=1, out=FAKE, ldo=64))
    assert call(rows=0) == 0
    assert call(fmt=0) == UNSUPPORTED and call(fmt=3) == UNSUPPORTED
    assert call(act=3) == UNSUPPORTED
    assert call(H=32800, ldq=32800, lds=1025, ldws=1028) == UNSUPPORTED
    assert call(N=1 << 24) == UNSUPPORTED              # N * H
    assert call(ldws=1 << 26) == UNSUPPORTED           # N * ld_ws
    assert call(rows=(1 << 31) - 1) == UNSUPPORTED
    assert call(ldq=(1 << 22) + 16) == UNSUPPORTED
    assert call(lds=(1 << 22) + 1) == UNSUPPORTED
    # 2^32 threads: blocks of weight rows, tiles
    assert call(E=1024, N=1 << 24, H=32, ldq=32, lds=1,
                ldo=1 << 24) == UNSUPPORTED
    for m in (200, 1 << 30):
        assert call(rows=(1 << 31) - (1 << 16), E=1024, N=1024, H=32, ldq=32,
                    lds=1, m=m, ldo=1024) == UNSUPPORTED
    for bad in (dict(E=0), dict(E=1025), dict(N=0), dict(H=0), dict(H=48),
                dict(rows=-1), dict(m=-1), dict(N=62), dict(act=2, N=65),
                dict(act=2, N=4), dict(ldq=pay - 16), dict(ldq=pay + 8),
                dict(lds=3), dict(ldws=0), dict(ldws=6), dict(ws=FAKE + 2),
                dict(w=FAKE + 8), dict(q=FAKE + 8), dict(ldo=60),
                dict(ldo=66), dict(out=FAKE + 4), dict(res=FAKE, ldr=60),
                dict(res=FAKE + 4, ldr=64), dict(q=None), dict(s=None),
                dict(w=None), dict(ws=None), dict(off=None),
                dict(counts=None), dict(out=None)):
        assert call(**bad) == INVALID, bad


@pytest.mark.parametrize("out_fmt", [1, 2])
def test_expert_matmul_quant(mxq, out_fmt):
    call = caller(mxq.lib().moe_expert_matmul_mxfp4_quant, dict(
        q=FAKE, ldq=64, s=FAKE, lds=4, rows=8, fmt=2, w=FAKE, ws=FAKE,
        ldws=4, E=4, N=64, H=128, off=FAKE, counts=FAKE, bias=None, act=0,
        m=1, of=out_fmt, out=FAKE, ldo=64, so=FAKE, lso=2))
    assert call(rows=0) == 0
    assert call(of=0) == UNSUPPORTED and call(of=3) == UNSUPPORTED
    for bad in (dict(N=48), dict(act=2, N=32), dict(ldo=16), dict(ldo=72),
                dict(out=FAKE + 8), dict(so=None), dict(lso=1),
                dict(out=None)):
        assert call(**bad) == INVALID, bad


def test_the_format_is_none_of_the_8_bit_calls(mxq):
    L = mxq.lib()
    assert L.moe_scatter_quant(FAKE, 64, 8, 64, FAKE, 1, 2, FAKE, 64, FAKE, 2,
                               8, None) == UNSUPPORTED
    assert L.moe_expert_matmul(
        FAKE, 128, FAKE, 4, 8, 2, FAKE, FAKE, 4, 64, 128, FAKE, FAKE, None, 0,
        None, 0, 1, FAKE, 64, None) == UNSUPPORTED
    assert L.moe_expert_matmul_quant(
        FAKE, 128, FAKE, 4, 8, 1, FAKE, FAKE, 4, 64, 128, FAKE, FAKE, None, 0,
        1, 2, FAKE, 64, FAKE, 2, None) == UNSUPPORTED


def test_binding_refuses_host_tensors(mxq):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q = torch.zeros((4, 32), dtype=torch.uint8)
    s = torch.zeros((4, 2), dtype=torch.uint8)
    w = torch.zeros((2, 8, 32), dtype=torch.uint8)
    ws = torch.zeros((2, 8, 4), dtype=torch.uint8)[:, :, :2]
    i = torch.zeros((4, 2), dtype=torch.int32)
    l = torch.zeros((4, 8))
    for f in (lambda: mxq.moe_balance_loss(l, i),
              lambda: mxq.moe_balance_loss_backward(torch.ones(1), l,
                                                    i[:1].repeat(1, 4)),
              lambda: mxq.mxfp4_quant_rows(x),
              lambda: mxq.moe_scatter_quant_mxfp4(x, i, 8),
              lambda: mxq.mxfp4_to_e4m3(q),
              lambda: mxq.upscale_mxfp4_to_bf16(q, s),
              lambda: mxq.moe_expert_matmul_mxfp4(q, s, w, ws, i[0], i[0]),
              lambda: mxq.moe_expert_matmul_mxfp4_quant(q, s, w, ws, i[0],
                                                        i[0])):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            f()
