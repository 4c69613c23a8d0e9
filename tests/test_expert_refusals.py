"""Refusals of the expert products, their combination and the 8-bit products:
host checks that return before any HIP call, so they need no GPU."""
import ctypes

import pytest
import torch

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")

FAKE = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced (checks fail first)
MIS = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned
INV, UNS, OK = B.OMNI_ERR_INVALID_ARG, B.OMNI_ERR_UNSUPPORTED, B.OMNI_OK


def test_expert_matmul_argument_checks():
    f = B.lib().omni_expert_matmul

    def call(dt=1, M=4, E=2, n=8, k=16, R=4, Ro=4, x=FAKE, xr=None, w=FAKE, off=FAKE, tr=0,
             act=0, out=FAKE, orow=None):
        return f(dt, M, E, n, k, R, Ro, x, xr, w, off, tr, act, out, orow, None)
    for bad in (dict(dt=2), dict(M=-1), dict(E=0), dict(n=0), dict(k=0), dict(R=-1),
                dict(Ro=-1), dict(x=None), dict(w=None), dict(off=None), dict(out=None),
                dict(x=MIS), dict(w=MIS), dict(out=MIS), dict(act=2), dict(act=1, tr=1),
                dict(R=3), dict(Ro=3)):
        assert call(**bad) == INV, bad
    assert call(k=12) == UNS                       # bf16 rows of 8
    assert call(dt=0, k=6) == UNS                  # float32 rows of 4
    assert call(n=12, tr=1) == UNS
    assert call(M=1 << 30, R=1 << 30, Ro=1 << 30, n=1 << 20) == UNS  # work-items past 32 bits
    assert call(n=(1 << 22) + 1) == UNS
    assert call(k=(1 << 22) + 8) == UNS
    assert call(M=0, R=0, Ro=0, x=None, out=None) == OK


def test_expert_weight_grad_argument_checks():
    f = B.lib().omni_expert_weight_grad

    def call(dt=1, M=4, E=2, n=8, k=16, R=4, Ry=4, x=FAKE, xr=None, dy=FAKE, yr=None, off=FAKE,
             dw=FAKE, ws=None, nws=0):
        return f(dt, M, E, n, k, R, Ry, x, xr, dy, yr, off, dw, ws, nws, None)
    for bad in (dict(dt=2), dict(M=-1), dict(E=0), dict(n=0), dict(k=0), dict(x=None),
                dict(dy=None), dict(off=None), dict(dw=None), dict(x=MIS), dict(dy=MIS),
                dict(dw=MIS), dict(R=3), dict(Ry=3)):
        assert call(**bad) == INV, bad
    assert call(n=12) == UNS
    assert call(k=12) == UNS
    assert call(dt=0, n=6) == UNS
    assert call(E=1 << 30, n=1 << 15, k=1 << 15) == UNS
    assert call(n=(1 << 22) + 8) == UNS
    assert call(k=(1 << 22) + 8) == UNS
    # few tiles, many tasks: partial sums in a workspace
    need = B.lib().omni_expert_weight_grad_workspace
    assert need(1, 4, 2, 8, 16) == 0 and need(2, 4, 2, 8, 16) == 0 and need(1, 4, 2, 0, 16) == 0
    assert need(1, 65536, 64, 1408, 2048) == 0
    big = dict(M=8192, E=1, n=512, k=512, R=8192, Ry=8192)
    n = need(1, 8192, 1, 512, 512)
    assert n >= 2 * 512 * 512 * 4
    for bad in (dict(), dict(ws=FAKE, nws=n - 1), dict(ws=ctypes.c_void_p((1 << 20) + 16), nws=n)):
        assert call(**big, **bad) == B.OMNI_ERR_WORKSPACE, bad


def test_combine_argument_checks():
    f = B.lib().omni_expert_combine

    def call(dt=1, L=4, K=2, n=16, o=FAKE, g=None, y=FAKE):
        return f(dt, L, K, n, o, g, y, 0, None)
    for bad in (dict(dt=2), dict(L=-1), dict(K=0), dict(n=0), dict(o=None), dict(y=None),
                dict(o=MIS), dict(y=MIS), dict(L=1 << 30, K=2)):
        assert call(**bad) == INV, bad
    assert call(n=12) == UNS
    assert call(dt=0, n=6) == UNS
    assert call(L=1 << 28, K=1, n=1 << 20) == UNS
    assert call(L=0, o=None, y=None) == OK
    f2 = B.lib().omni_expert_combine_backward

    def back(dt=1, L=4, K=2, n=16, o=FAKE, g=None, dy=FAKE, do=FAKE, dg=FAKE):
        return f2(dt, L, K, n, o, g, dy, do, dg, None)
    for bad in (dict(dt=2), dict(K=0), dict(o=None), dict(dy=None), dict(do=None), dict(o=MIS),
                dict(dy=MIS), dict(do=MIS)):
        assert back(**bad) == INV, bad
    assert back(n=12) == UNS
    assert back(L=0, o=None, dy=None, do=None, dg=None) == OK


def test_quantized_argument_checks():
    f = B.lib().omni_quantize_rows

    def quant(dt=1, R=4, k=32, x=FAKE, q=FAKE, s=FAKE):
        return f(dt, R, k, x, q, s, None)
    for bad in (dict(dt=2), dict(R=-1), dict(k=0), dict(x=None), dict(q=None), dict(s=None),
                dict(x=MIS), dict(q=MIS)):
        assert quant(**bad) == INV, bad
    assert quant(k=24) == UNS
    assert quant(R=1 << 26) == UNS
    assert quant(R=0, x=None, q=None, s=None) == OK
    g = B.lib().omni_quantized_matmul

    def dense(dt=1, M=4, n=8, k=32, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, act=0, out=FAKE):
        return g(dt, M, n, k, xq, xs, wq, ws, act, out, None)
    for bad in (dict(dt=2), dict(M=-1), dict(n=0), dict(k=0), dict(xq=None), dict(xs=None),
                dict(wq=None), dict(ws=None), dict(out=None), dict(xq=MIS), dict(wq=MIS),
                dict(out=MIS), dict(act=3)):
        assert dense(**bad) == INV, bad
    assert dense(k=24) == UNS
    assert dense(k=131072) == UNS                  # the integer sum could pass 31 bits
    assert dense(M=0, xq=None, xs=None, out=None) == OK
    h = B.lib().omni_quantized_expert_matmul

    def expert(dt=1, M=4, E=2, n=8, k=32, R=4, Ro=4, xq=FAKE, xs=FAKE, xr=None, wq=FAKE,
               ws=FAKE, off=FAKE, act=0, out=FAKE, orow=None):
        return h(dt, M, E, n, k, R, Ro, xq, xs, xr, wq, ws, off, act, out, orow, None)
    for bad in (dict(off=None), dict(R=3), dict(Ro=3), dict(xs=None), dict(ws=None), dict(E=0)):
        assert expert(**bad) == INV, bad
    assert expert(k=24) == UNS


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 16), torch.zeros(2, 8, 16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        B.expert_matmul(x, w, off)
    with pytest.raises(ValueError, match=r"\[E, n, k\]"):
        B.expert_matmul(x, w[0], off)
    with pytest.raises(ValueError, match=r"\[E, n, k\]"):
        B.expert_matmul(x, torch.zeros(2, 7, 16), off, swiglu=True)
    with pytest.raises(ValueError, match="not a multiple"):
        B.expert_combine(x, 3)
    with pytest.raises(ValueError, match="device tensor"):
        B.quantize_rows(x)
