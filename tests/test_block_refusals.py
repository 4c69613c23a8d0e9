"""Refusals of routing, residual norms and 4-bit rows: host checks that return
before any HIP call, so they need no GPU."""
import ctypes

import pytest
import torch

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")

FAKE = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced (checks fail first)
MIS = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned
ODD = ctypes.c_void_p((1 << 20) + 2)  # not 4-byte aligned
INV, UNS, OK = B.OMNI_ERR_INVALID_ARG, B.OMNI_ERR_UNSUPPORTED, B.OMNI_OK
NAN, INF = float("nan"), float("inf")


def test_route_argument_checks():
    f = B.lib().omni_expert_route

    def call(dt=1, L=4, E=16, K=2, z=FAKE, b=None, fn=0, g=1, tg=1, gb=2, rn=1, sc=1.0, i=FAKE,
             w=FAKE, s=None):
        return f(dt, L, E, K, z, b, fn, g, tg, gb, rn, sc, i, w, s, None)
    for bad in (dict(dt=2), dict(L=-1), dict(E=0), dict(K=0), dict(K=17), dict(fn=2),
                dict(fn=-1), dict(g=0), dict(g=3), dict(g=4, tg=5), dict(tg=0), dict(gb=0),
                dict(gb=3), dict(sc=NAN), dict(sc=INF), dict(z=None), dict(i=None), dict(w=None),
                dict(g=4, tg=1, K=5), dict(L=1 << 25, K=64, E=64)):
        assert call(**bad) == INV, bad
    assert call(K=65, E=128) == UNS
    assert call(E=1025) == UNS
    assert call(E=256, g=128, tg=128) == UNS
    assert call(L=1 << 26) == UNS
    assert call(L=0, z=None, i=None, w=None) == OK
    assert call(L=0, E=17, g=4, tg=4) == INV


def test_route_backward_argument_checks():
    f = B.lib().omni_expert_route_backward

    def call(dt=1, L=4, E=16, K=2, z=FAKE, i=FAKE, dg=FAKE, fn=0, rn=1, sc=1.0, ds=None, sh=0,
             dz=FAKE):
        return f(dt, L, E, K, z, i, dg, fn, rn, sc, ds, sh, dz, None)
    for bad in (dict(dt=2), dict(L=-1), dict(E=0), dict(K=0), dict(fn=2), dict(sc=INF),
                dict(z=None), dict(i=None), dict(dg=None), dict(dz=None)):
        assert call(**bad) == INV, bad
    assert call(K=65) == UNS and call(E=1025) == UNS and call(L=1 << 26) == UNS
    assert call(L=0, z=None, i=None, dg=None, dz=None) == OK


def test_norm_argument_checks():
    f = B.lib().omni_residual_norm

    def call(dt=1, yt=0, L=4, d=64, r=FAKE, y=FAKE, post=0, pw=None, g=None, gk=0, al=1.0,
             eps=1e-6, ro=FAKE, w=FAKE, x=FAKE):
        return f(dt, yt, L, d, r, y, post, pw, g, gk, al, eps, ro, w, x, None)
    for bad in (dict(dt=2), dict(yt=2), dict(dt=0, yt=1), dict(L=-1), dict(d=0), dict(r=None),
                dict(ro=None), dict(x=None), dict(pw=FAKE), dict(post=1, pw=MIS), dict(g=FAKE),
                dict(gk=1), dict(gk=4, g=FAKE), dict(gk=-1, g=FAKE), dict(gk=1, g=MIS),
                dict(gk=2, g=ctypes.c_void_p((1 << 20) + 1)), dict(dt=0, gk=2, g=ODD),
                dict(al=NAN), dict(eps=NAN), dict(eps=-1.0), dict(eps=INF), dict(r=MIS),
                dict(y=MIS), dict(ro=MIS), dict(w=MIS), dict(x=MIS), dict(y=None),
                dict(y=None, ro=None, post=1), dict(y=None, ro=None, g=FAKE, gk=1),
                dict(y=None, ro=None, x=None, w=None)):
        assert call(**bad) == INV, bad
    assert call(d=60) == UNS and call(dt=0, d=62) == UNS and call(d=16392) == UNS
    assert call(L=1 << 22) == UNS
    assert call(L=0, r=None, y=None, ro=None, x=None) == OK


def test_norm_backward_argument_checks():
    f, need = B.lib().omni_residual_norm_backward, B.lib().omni_residual_norm_backward_workspace

    def call(dt=1, yt=0, xt=0, L=200, d=64, r=FAKE, y=FAKE, post=0, pw=None, g=None, gk=0,
             al=1.0, eps=1e-6, w=FAKE, dro=FAKE, dx=FAKE, dr=FAKE, dy=FAKE, dg=None, dw=None, dpw=None,
             ws=None, n=0):
        return f(dt, yt, xt, L, d, r, y, post, pw, g, gk, al, eps, w, dro, dx, dr, dy, dg, dw,
                 dpw, ws, n, None)
    for bad in (dict(dt=2), dict(yt=2), dict(xt=2), dict(dt=0, xt=1), dict(dt=0, yt=1),
                dict(L=-1), dict(d=0), dict(r=None), dict(dr=None), dict(dx=None, dro=None),
                dict(dx=None), dict(dx=None, w=None, dw=FAKE), dict(y=None),
                dict(dg=FAKE), dict(dpw=FAKE), dict(pw=FAKE), dict(gk=1), dict(g=FAKE),
                dict(r=MIS), dict(y=MIS), dict(w=MIS), dict(dro=MIS), dict(dx=MIS), dict(dr=MIS),
                dict(dy=MIS), dict(dw=MIS), dict(gk=1, g=FAKE, dg=MIS), dict(gk=2, g=FAKE, dg=ODD),
                dict(eps=-1.0), dict(al=INF)):
        assert call(**bad) == INV, bad
    assert call(d=60) == UNS and call(d=16392) == UNS and call(L=1 << 22) == UNS
    n = need(1, 200, 64)
    assert n > 0 and need(2, 200, 64) == 0 and need(1, -1, 64) == 0 and need(1, 200, 1 << 20) == 0
    assert need(1, 32, 64) == 0 < need(1, 33, 64) and need(0, 4, 16384) == 0 < need(0, 5, 16384)
    for bad in (dict(), dict(ws=FAKE, n=n - 1), dict(ws=MIS, n=n)):
        assert call(dw=FAKE, **bad) == B.OMNI_ERR_WORKSPACE
        assert call(post=1, dpw=FAKE, **bad) == B.OMNI_ERR_WORKSPACE
        assert call(gk=1, g=FAKE, dg=FAKE, **bad) == B.OMNI_ERR_WORKSPACE
    assert call(L=0, r=None, y=None, dro=None, dx=None, dr=None, dy=None) == OK


def test_microscale_argument_checks():
    f = B.lib().omni_microscale_rows

    def rows(dt=1, R=4, k=64, x=FAKE, q=FAKE, s=FAKE):
        return f(dt, R, k, x, q, s, None)
    for bad in (dict(dt=2), dict(R=-1), dict(k=0), dict(x=None), dict(q=None), dict(s=None),
                dict(x=MIS), dict(q=MIS), dict(s=ODD)):
        assert rows(**bad) == INV, bad
    assert rows(k=48) == UNS and rows(R=1 << 28) == UNS and rows(R=1 << 24, k=2048) == UNS
    assert rows(R=0, x=None, q=None, s=None) == OK
    for grouped in (False, True):
        g = B.lib().omni_microscaled_expert_matmul if grouped else B.lib().omni_microscaled_matmul

        def call(dt=1, M=4, E=2, n=8, k=64, R=4, Ro=4, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, off=FAKE,
                 act=0, out=FAKE):
            if grouped:
                return g(dt, M, E, n, k, R, Ro, x, xs, None, w, ws, off, act, out, None, None)
            return g(dt, M, n, k, x, xs, w, ws, act, out, None)
        cases = [dict(dt=2), dict(M=-1), dict(n=0), dict(k=0), dict(x=None), dict(xs=None),
                 dict(w=None), dict(ws=None), dict(out=None), dict(x=MIS), dict(w=MIS),
                 dict(out=MIS), dict(xs=ODD), dict(ws=ODD), dict(act=2)]
        if grouped:
            cases += [dict(E=0), dict(R=3), dict(Ro=3), dict(R=-1), dict(off=None)]
        for bad in cases:
            assert call(**bad) == INV, bad
        assert call(k=48) == UNS and call(n=(1 << 22) + 1) == UNS and call(k=(1 << 22) + 32) == UNS
        assert call(M=1 << 30, R=1 << 30, Ro=1 << 30, n=1 << 20) == UNS
        assert call(act=1, n=1 << 17, k=1 << 16) == UNS and call(act=1, n=1 << 22, k=2048) == UNS
        assert call(M=0, R=0, Ro=0, x=None, xs=None, out=None) == OK


def test_python_calls_refuse_what_does_not_fit():
    z, f32 = torch.zeros(4, 8), torch.float32
    with pytest.raises(ValueError):
        B.expert_route(z, 2)                                   # not on a device
    with pytest.raises(ValueError):
        B.expert_route_backward(z, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        B.residual_norm(z)
    with pytest.raises(ValueError):
        B.residual_norm_backward(z, dx=z)
    with pytest.raises(ValueError):
        B.microscale_rows(z)
    u8 = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.microscaled_matmul(u8, u8, u8, u8)
    with pytest.raises(ValueError):
        B.microscaled_expert_matmul(u8, u8, u8[None], u8[None], u8)
    assert f32 == z.dtype


@pytest.mark.gpu
def test_python_calls_refuse_mismatched_arguments():
    d = "cuda"
    z = torch.zeros(4, 8, device=d)
    with pytest.raises(ValueError, match="scores"):
        B.expert_route(z, 2, scores="relu")
    with pytest.raises(TypeError, match="bias"):
        B.expert_route(z, 2, bias=torch.zeros(8, device=d, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        B.expert_route(torch.zeros(4, 16, device=d)[:, ::2], 2)
    with pytest.raises(TypeError, match="unsupported"):
        B.expert_route(z.half(), 2)
    with pytest.raises(B.OmniError):
        B.expert_route(z, 9)
    with pytest.raises(ValueError, match="dscore"):
        B.expert_route_backward(z, torch.zeros(4, 2, device=d, dtype=torch.int32),
                                torch.zeros(4, 2, device=d), dscore=torch.zeros(7, device=d))
    with pytest.raises(ValueError, match="need y"):
        B.residual_norm(z, post=True)
    with pytest.raises(ValueError, match="r_out is r"):
        B.residual_norm(z, r_out=torch.zeros_like(z))
    with pytest.raises(ValueError, match="gate has shape"):
        B.residual_norm(z, y=z, gate=torch.zeros(4, 3, device=d))
    with pytest.raises(TypeError, match="weight"):
        B.residual_norm(z, weight=torch.zeros(8, device=d, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="wanted"):
        B.residual_norm(z, want_x=False)
    with pytest.raises(ValueError, match="one of dx"):
        B.residual_norm_backward(z)
    with pytest.raises(ValueError, match="belongs to x"):
        B.residual_norm_backward(z, dr_out=z, weight=torch.zeros(8, device=d))
    with pytest.raises(ValueError, match="does not give"):
        B.residual_norm_backward(z, dx=z, out={"dy": torch.zeros_like(z)})
    with pytest.raises(B.OmniError):
        B.microscale_rows(torch.zeros(4, 48, device=d))
    q, s = B.microscale_rows(torch.zeros(4, 64, device=d))
    with pytest.raises(ValueError, match="x_scale"):
        B.microscaled_matmul(q, s[:, :2].contiguous(), q, s)
    with pytest.raises(TypeError, match="wq"):
        B.microscaled_matmul(q, s, q.to(torch.int8), s)
    with pytest.raises(ValueError, match="even"):
        B.microscaled_matmul(q, s, q[:3].contiguous(), s[:3].contiguous(), swiglu=True)


@pytest.mark.parametrize("more", [1, 2, 3])
def test_route_of_more_tokens_than_a_launch_holds(more):
    """Four tokens a workgroup of 256: from 2^26 - 3 on they are 2^24 workgroups, 2^32
    work-items, one more than a launch takes."""
    L = (1 << 26) - 4 + more
    assert (L + 3) // 4 * 256 == 1 << 32 and (L - more + 3) // 4 * 256 < 1 << 32
    for E, K in ((16, 2), (128, 17), (520, 1), (1024, 1)):
        assert B.lib().omni_expert_route(1, L, E, K, FAKE, None, 0, 1, 1, 1, 1, 1.0, FAKE, FAKE,
                                         None, None) == UNS
        assert B.lib().omni_expert_route_backward(1, L, E, K, FAKE, FAKE, FAKE, 0, 1, 1.0, None, 0,
                                                  FAKE, None) == UNS
