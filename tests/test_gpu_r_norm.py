"""The residual norms and their gradients against the float64 oracle.

Tolerances.  A sum of squares of d <= 16384 columns over 64 lanes or more (32 up to 256) runs at
most 32 + 6 + 16 additions deep for its partial sums (each 2^-24 of a positive
sum), its root halves that, the root itself adds 2^-22, and each product 2^-24:
c = 40 x 2^-23 of every term of r_out.  x also carries r_out's error, directly and
through the mean of its squares.  The gradients hold up to three such factors and
two more row sums: 100 x 2^-23 of the sum of the absolute terms; a sum over L rows
adds at most L + 32 additions.  A rounding to bfloat16 adds 2^-8 of the value, to
float32 2^-24."""
import itertools

import numpy as np
import pytest
import torch

from oracle import omni_blocks as OB
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from tests.gpu_helpers import dev, host

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C = 40 * 2.0 ** -23
NAMES = ("dr", "dweight", "dgate", "dpost_weight", "dy")


def arr(rng, shape, dt, scale=1.0, shift=0.0):
    a = (rng.standard_normal(shape) * scale + shift).astype(np.float32)
    return f32_to_bf16_bits(a) if dt == "bf16" else a


def close(got, want, tol, what):
    got = bf16_bits_to_f32(got) if got.dtype == np.uint16 else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], want[bad][:3], np.broadcast_to(tol, want.shape)[bad][:3])


def make(rng, L, d, dt, yt, post, gate):
    a = {"r": arr(rng, (L, d), dt, 2.0), "weight": arr(rng, (d,), dt, 0.3, 1.0)}
    if yt:
        a["y"] = arr(rng, (L, d), yt)
    if post == "weight":
        a["post_weight"] = arr(rng, (d,), dt, 0.3, 1.0)
    if gate:
        a["gate"] = arr(rng, {"column": (d,), "token": (L, 1), "full": (L, d)}[gate], dt, 0.5, 0.5)
    return a


def forward_close(a, dt, post, alpha, eps, r_out, x):
    w1, wx, mass = OB.residual_norm(a["r"], a.get("y"), a.get("weight"), a.get("post_weight"), post,
                                    a.get("gate"), alpha, eps)
    if "y" in a:
        close(host(r_out), w1, C * mass + HALF[dt] * 1.001 * np.abs(w1) + 1e-37, "r_out")
    if x is None:
        return
    ms = (w1 * w1).mean(axis=1, keepdims=True) + eps
    inv = 1 / np.sqrt(ms)
    w = 1.0 if a.get("weight") is None else np.abs(OB.widen(a["weight"]))
    rel = C * (1 + (np.abs(w1) * mass).mean(axis=1, keepdims=True) / ms)
    close(host(x), wx, (C * mass * inv + rel * np.abs(w1) * inv) * w
          + HALF[dt] * 1.001 * np.abs(wx) + 1e-37, "x")


WIDTHS = {"bf16": [8, 64, 200, 512, 520, 1000, 1024, 2048, 2056, 4096, 5632, 8192, 8200, 16384],
          "f32": [4, 64, 100, 256, 260, 512, 1000, 1024, 1028, 2048, 4096, 8192, 8196, 16384]}


@pytest.mark.parametrize("dt,d", [(t, d) for t in WIDTHS for d in WIDTHS[t]])
@pytest.mark.parametrize("L", [1, 7])
def test_norm_widths(dt, d, L):
    rng = np.random.default_rng(d + L)
    for yt, post, gate in ((None, "none", None), ("f32", "weight", "column"), (dt, "ones", "token"),
                           ("f32", "none", "full")):
        a = make(rng, L, d, dt, yt, post, gate)
        t = {k: dev(v) for k, v in a.items()}
        r_out, x = B.residual_norm(**t, post=post != "none", alpha=0.7, eps=1e-5)
        forward_close(a, dt, post != "none", 0.7, 1e-5, r_out, x)
        if yt is None:
            assert r_out is t["r"]


@pytest.mark.parametrize("yt,post,gate", itertools.product(
    ["f32", "same"], ["none", "ones", "weight"], [None, "column", "token", "full"]))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_forms(dt, yt, post, gate):
    rng = np.random.default_rng(9)
    L, d = 37, 328
    a = make(rng, L, d, dt, dt if yt == "same" else yt, post, gate)
    t = {k: dev(v) for k, v in a.items()}
    r_out, x = B.residual_norm(**t, post=post != "none")
    forward_close(a, dt, post != "none", 1.0, 1e-6, r_out, x)
    # without the weight, without x, and into r itself
    del t["weight"]
    w = a.pop("weight")
    r2, x2 = B.residual_norm(**t, post=post != "none", alpha=-2.0)
    forward_close(a, dt, post != "none", -2.0, 1e-6, r2, x2)
    r3, x3 = B.residual_norm(**t, post=post != "none", alpha=-2.0, want_x=False)
    assert x3 is None and torch.equal(r3, r2)
    r4, x4 = B.residual_norm(**t, post=post != "none", alpha=-2.0, r_out=t["r"],
                             weight=dev(w))
    assert r4 is t["r"] and torch.equal(r4, r2)


def test_norm_rows_do_not_depend_on_the_batch():
    rng = np.random.default_rng(3)
    a = {k: dev(v) for k, v in make(rng, 300, 1000, "bf16", "f32", "weight", "full").items()}
    dx, dr = dev(arr(rng, (300, 1000), "f32")), dev(arr(rng, (300, 1000), "bf16"))
    r1, x = B.residual_norm(**a)
    g = B.residual_norm_backward(r1, dx=dx, dr_out=dr, **{k: v for k, v in a.items() if k != "r"})
    for lo, hi in ((0, 1), (17, 40), (299, 300)):
        s = {k: v[lo:hi] if v.dim() == 2 else v for k, v in a.items()}
        r2, x2 = B.residual_norm(**s)
        h = B.residual_norm_backward(r1[lo:hi], dx=dx[lo:hi], dr_out=dr[lo:hi],
                                     **{k: v for k, v in s.items() if k != "r"})
        assert torch.equal(r2, r1[lo:hi]) and torch.equal(x2, x[lo:hi])
        for name in ("dr", "dy", "dgate"):
            assert torch.equal(h[name], g[name][lo:hi]), name


def test_norm_of_zeros_nan_and_no_rows():
    """A row of zeros gives zeros (with eps), NaN and infinity stay in their rows."""
    z = torch.zeros((4, 64), device="cuda")
    z[1, 3], z[2, 5] = float("nan"), float("inf")
    z[3] = torch.arange(64.0)
    r1, x = B.residual_norm(torch.zeros_like(z), y=z, post=True)
    assert (x[0] == 0).all() and (r1[0] == 0).all() and torch.isnan(x[1]).all()
    assert torch.isnan(r1[2, 5]) and torch.isfinite(x[3]).all()
    g = B.residual_norm_backward(torch.zeros_like(z), dx=torch.ones_like(z), y=z, post=True)
    assert torch.isfinite(g["dr"]).all() and torch.isnan(g["dy"][1]).all()
    assert torch.isfinite(g["dy"][[0, 3]]).all()
    e, w = torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda")
    r1, x = B.residual_norm(e, y=e, weight=w, post_weight=w, gate=w)
    assert r1.shape == x.shape == (0, 64)
    g = B.residual_norm_backward(e, dx=e, y=e, weight=w, post_weight=w, gate=w,
                                 out={"dweight": torch.full((64,), 7.0, device="cuda")})
    for name in ("dweight", "dpost_weight", "dgate"):
        assert g[name].shape == (64,) and (g[name] == 0).all()


def backward_close(a, dt, xt, post, alpha, eps, dx, dr_out, got):
    kw = {k: a.get(k) for k in ("y", "post_weight", "gate")}
    want = OB.residual_norm_backward(a["r"], dx, dr_out, kw["y"],
                                     a.get("weight") if dx is not None else None,
                                     kw["post_weight"], post, kw["gate"], alpha, eps)
    L = a["r"].shape[0]
    for name, g in got.items():
        w, mass = want[name]
        t = host(g)
        steps = 100 + (L + 32 if name in ("dweight", "dpost_weight") or
                       (name == "dgate" and kw["gate"].ndim == 1) else 0)
        half = 2.0 ** -8 if t.dtype == np.uint16 else 2.0 ** -24
        close(t, w, steps * 2.0 ** -23 * mass + half * 1.001 * np.abs(w) + 1e-36, name)


@pytest.mark.parametrize("dt,d", [(t, d) for t in WIDTHS for d in WIDTHS[t]])
@pytest.mark.parametrize("L", [1, 5])
def test_norm_backward_widths(dt, d, L):
    rng = np.random.default_rng(d + L)
    for yt, post, gate, xt in ((None, "none", None, "f32"), ("f32", "weight", "column", dt),
                               (dt, "ones", "token", "f32"), ("f32", "weight", "full", "f32")):
        a = make(rng, L, d, dt, yt, post, gate)
        dx, dr = arr(rng, (L, d), xt), arr(rng, (L, d), dt)
        t = {k: dev(v) for k, v in a.items()}
        got = B.residual_norm_backward(t.pop("r"), dx=dev(dx), dr_out=dev(dr), **t,
                                       post=post != "none", alpha=0.7, eps=1e-5)
        backward_close(a, dt, xt, post != "none", 0.7, 1e-5, dx, dr, got)


@pytest.mark.parametrize("yt,post,gate", itertools.product(
    ["f32", "same"], ["none", "ones", "weight"], [None, "column", "token", "full"]))
@pytest.mark.parametrize("dt,xt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm_backward_forms(dt, xt, yt, post, gate):
    rng = np.random.default_rng(21)
    L, d = 41, 264
    a = make(rng, L, d, dt, dt if yt == "same" else yt, post, gate)
    dx, dr = arr(rng, (L, d), xt), arr(rng, (L, d), dt)
    t = {k: dev(v) for k, v in a.items()}
    r = t.pop("r")
    p = post != "none"
    both = B.residual_norm_backward(r, dx=dev(dx), dr_out=dev(dr), **t, post=p)
    expected = {"dr", "dy", "dweight"} | ({"dgate"} if gate else set()) | \
        ({"dpost_weight"} if post == "weight" else set())
    assert set(both) == expected
    backward_close(a, dt, xt, p, 1.0, 1e-6, dx, dr, both)
    only_dx = B.residual_norm_backward(r, dx=dev(dx), **t, post=p, alpha=0.5)
    backward_close(a, dt, xt, p, 0.5, 1e-6, dx, None, only_dx)
    w = t.pop("weight")
    only_dr = B.residual_norm_backward(r, dr_out=dev(dr), **t, post=p, alpha=0.5)
    assert "dweight" not in only_dr
    backward_close(a, dt, xt, p, 0.5, 1e-6, None, dr, only_dr)
    # no sums, and in place: dr over dr_out, dy over y
    y2, dr2 = t["y"].clone(), dev(dr)
    few = B.residual_norm_backward(r, dx=dev(dx), dr_out=dr2, **{**t, "y": y2}, weight=w, post=p,
                                   want_sums=False, out={"dr": dr2, "dy": y2})
    assert set(few) == {"dr", "dy"}
    assert torch.equal(few["dr"], both["dr"]) and torch.equal(few["dy"], both["dy"])


@pytest.mark.parametrize("L,d,dt", [(700, 64, "bf16"), (2600, 512, "f32"), (515, 1024, "bf16"),
                                    (1500, 2048, "bf16"), (513, 8192, "f32")])
def test_norm_backward_sums_over_many_rows(L, d, dt):
    rng = np.random.default_rng(L)
    a = make(rng, L, d, dt, "f32", "weight", "column")
    dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), dt)
    t = {k: dev(v) for k, v in a.items()}
    r = t.pop("r")
    got = B.residual_norm_backward(r, dx=dev(dx), dr_out=dev(dr), **t)
    backward_close(a, dt, "f32", True, 1.0, 1e-6, dx, dr, got)
    again = B.residual_norm_backward(r, dx=dev(dx), dr_out=dev(dr), **t)
    for name in got:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("post,gate", [("none", None), ("weight", "column"), ("ones", "token"),
                                       ("weight", "full")])
def test_norm_gradient_against_differences(post, gate):
    """Against differences of the forward itself, along random directions."""
    rng = np.random.default_rng(8)
    L, d, h = 3, 64, 2.0 ** -7
    a = make(rng, L, d, "f32", "f32", post, gate)
    dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), "f32")
    p = post != "none"

    def run(a):
        return B.residual_norm(**{k: dev(v) for k, v in a.items()}, post=p)
    r1, _ = run(a)
    t = {k: dev(v) for k, v in a.items()}
    t.pop("r")
    g = B.residual_norm_backward(r1, dx=dev(dx), dr_out=dev(dr), **t, post=p)

    def loss(a):
        r1, x = run(a)
        return (host(r1).astype(np.float64) * dr).sum() + (host(x).astype(np.float64) * dx).sum()
    grads = {"r": "dr", "y": "dy", "weight": "dweight", "gate": "dgate",
             "post_weight": "dpost_weight"}
    for name in a:
        v = rng.standard_normal(a[name].shape).astype(np.float32)
        hi, lo = dict(a), dict(a)
        hi[name], lo[name] = a[name] + np.float32(h) * v, a[name] - np.float32(h) * v
        step = (hi[name].astype(np.float64) - lo[name]) / (2 * h)
        diff = (loss(hi) - loss(lo)) / (2 * h)
        want = (host(g[grads[name]]).astype(np.float64) * step).sum()
        # third derivatives of unit-sized rows along unit directions, h^2 of each of
        # the L d terms, and float32 outputs over 2 h
        tol = (h * h + 2.0 ** -21 / h) * (np.abs(dr).sum() + np.abs(dx).sum())
        assert abs(diff - want) <= tol, (name, diff, want, tol)


def test_norm_into_given_arrays_leaves_the_rest():
    rng = np.random.default_rng(2)
    L, d = 9, 72
    a = {k: dev(v) for k, v in make(rng, L + 2, d, "bf16", "bf16", "weight", "token").items()}
    cut = {k: v[:L] if v.dim() == 2 else v for k, v in a.items()}
    out = torch.full((4, L + 2, d), -7.0, device="cuda").to(torch.bfloat16)
    dg = torch.full((L + 2, 1), -7.0, device="cuda")
    B.residual_norm(**cut, r_out=out[0, :L], x=out[1, :L])
    cut.pop("r")
    B.residual_norm_backward(out[0, :L], dx=out[1, :L], **cut,
                             out={"dr": out[2, :L], "dy": out[3, :L], "dgate": dg[:L]})
    assert (out[:, L:] == -7).all() and (dg[L:] == -7).all() and not (out[:, :L] == -7).any()


def test_norm_captured_and_workspaces():
    """Captured forward and backward replay as they run; a workspace of the caller's."""
    rng = np.random.default_rng(6)
    L, d = 90, 1024
    a = {k: dev(v) for k, v in make(rng, L, d, "bf16", "f32", "weight", "column").items()}
    ins = [dev(arr(rng, (L, d), "bf16")) for _ in range(3)]
    dx = dev(arr(rng, (L, d), "f32"))
    r1, x = torch.empty_like(a["r"]), torch.empty_like(a["r"])
    rest = {k: v for k, v in a.items() if k != "r"}
    ws = torch.empty(B.lib().omni_residual_norm_backward_workspace(1, L, d), dtype=torch.uint8,
                     device="cuda")
    out = B.residual_norm_backward(a["r"], dx=dx, **rest, workspace=ws)

    def step():
        B.residual_norm(**a, r_out=r1, x=x)
        B.residual_norm_backward(r1, dx=dx, dr_out=x, **rest, out=out, workspace=ws)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for v in ins:
        a["r"].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        got = [r1.clone(), x.clone()] + [out[n].clone() for n in out]
        ws.fill_(255)
        step()
        for p, q in zip(got, [r1, x] + [out[n] for n in out]):
            assert torch.equal(p, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2, x2 = B.residual_norm(**a, stream=s)
    o2 = B.residual_norm_backward(r2, dx=dx, dr_out=x2, **rest, stream=s)
    s.synchronize()
    assert torch.equal(r2, r1) and torch.equal(x2, x)
    for n in out:
        assert torch.equal(out[n], o2[n])


# a width of each kernel that holds a row its own way
CLASSES = {"bf16": [64, 256, 512, 1000, 2048, 4096, 8192, 16384],
           "f32": [64, 256, 508, 1024, 2048, 4096, 8192, 16384]}


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("L", [1, 5, 33])
@pytest.mark.parametrize("dt,d", [(t, d) for t in CLASSES for d in CLASSES[t]])
def test_norm_backward_sums_with_little_eps(dt, d, L, eps):
    """Places that a workgroup has beyond the last row add nothing to the sums over the
    rows: there the mean of the squares is eps alone, its root 0 or next to it."""
    rng = np.random.default_rng(d + L)
    for yt, post, gate in ((None, "none", None), ("f32", "weight", "column")):
        a = make(rng, L, d, dt, yt, post, gate)
        dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), dt)
        t = {k: dev(v) for k, v in a.items()}
        got = B.residual_norm_backward(t.pop("r"), dx=dev(dx), dr_out=dev(dr), **t, eps=eps)
        backward_close(a, dt, "f32", post != "none", 1.0, eps, dx, dr, got)


@pytest.mark.parametrize("power", [50, -50])
@pytest.mark.parametrize("dt,d", [(t, d) for t in CLASSES for d in CLASSES[t]])
def test_norm_backward_of_large_and_small_rows(dt, d, power):
    """Rows of 2^50 and 2^-50, whose inverse root's cube is no float32, without eps; dr_out
    of the size of dx over them, so that every term counts."""
    rng = np.random.default_rng(d)
    L = 5
    for yt, post, gate in ((None, "none", None), ("f32", "weight", "column"), (dt, "ones", "token")):
        a = make(rng, L, d, dt, yt, post, gate)
        a["r"] = arr(rng, (L, d), dt, 2.0 ** power)
        if yt:
            a["y"] = arr(rng, (L, d), yt, 2.0 ** power)
        dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), dt, 2.0 ** -power)
        t = {k: dev(v) for k, v in a.items()}
        got = B.residual_norm_backward(t.pop("r"), dx=dev(dx), dr_out=dev(dr), **t,
                                       post=post != "none", eps=0.0)
        backward_close(a, dt, "f32", post != "none", 1.0, 0.0, dx, dr, got)


@pytest.mark.parametrize("dt,d", [(t, d) for t in CLASSES for d in CLASSES[t]])
def test_norm_backward_of_zero_rows_with_little_eps(dt, d):
    """A row of zeros among others: its gradient is dx w / sqrt(eps), and so on to dy."""
    rng = np.random.default_rng(d)
    L, eps = 5, 1e-30
    a = make(rng, L, d, dt, "f32", "weight", "column")
    a["r"][2], a["y"][2], a["y"][4] = 0, 0, 0
    dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), dt)
    t = {k: dev(v) for k, v in a.items()}
    got = B.residual_norm_backward(t.pop("r"), dx=dev(dx), dr_out=dev(dr), **t, eps=eps)
    backward_close(a, dt, "f32", True, 1.0, eps, dx, dr, got)


@pytest.mark.parametrize("gate", [None, "column", "token", "full"])
@pytest.mark.parametrize("dt,d", [(t, d) for t in CLASSES for d in CLASSES[t]])
def test_norm_backward_of_y_not_finite_without_post_norm(dt, d, gate):
    """Without a post norm dy is alpha g dr, whatever y holds; from dr_out alone the
    gate's gradient is that of the formula too."""
    rng = np.random.default_rng(d)
    L = 6
    a = make(rng, L, d, dt, "f32", "none", gate)
    a["y"][1, 3], a["y"][2, 0], a["y"][4, d - 1], a["y"][4, 1] = np.inf, np.nan, -np.inf, -np.inf
    dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), dt)
    t = {k: dev(v) for k, v in a.items()}
    r, w = t.pop("r"), t.pop("weight")
    for given, weight in (((None, dr), None), ((dx, dr), w)):
        got = B.residual_norm_backward(r, dx=dev(given[0]), dr_out=dev(given[1]), **t,
                                       weight=weight, alpha=0.5)
        wide = got.pop("dgate", None)
        with np.errstate(invalid="ignore"):
            backward_close(a, dt, "f32", False, 0.5, 1e-6, *given, got)
        if gate is None:
            continue
        with np.errstate(invalid="ignore"):
            want, mass = OB.residual_norm_backward(
                a["r"], *given, a["y"], a["weight"] if weight is not None else None, None, False,
                a["gate"], 0.5, 1e-6)["dgate"]
        wide = host(wide)
        half = 2.0 ** -8 if wide.dtype == np.uint16 else 2.0 ** -24
        wide = bf16_bits_to_f32(wide) if wide.dtype == np.uint16 else wide
        finite = np.isfinite(want)
        assert not finite.all() and finite.any() and (np.isfinite(wide) == finite).all()
        if given[0] is None or gate != "token":
            np.testing.assert_array_equal(wide[~finite], want[~finite])
        # as backward_close
        tol = (132 + L) * 2.0 ** -23 * mass[finite] + half * 1.001 * np.abs(want[finite]) + 1e-36
        assert (np.abs(wide[finite] - want[finite]) <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 2048, 16384])
def test_norm_of_rows_whose_squares_pass_float32(dt, d):
    """An infinite mean of squares: the norm is 0, with its gradients; the others' stay."""
    rng = np.random.default_rng(d)
    a = make(rng, 3, d, dt, "f32", "weight", None)
    a["r"][1], a["y"][1] = (f32_to_bf16_bits(np.float32(1e25)) if dt == "bf16" else 1e25), -1e25
    t = {k: dev(v) for k, v in a.items()}
    r1, x = B.residual_norm(**t)
    assert torch.equal(r1[1], t["r"][1]) and (x[1] == 0).all() and (x[[0, 2]] != 0).any(dim=1).all()
    dx = dev(arr(rng, (3, d), "f32"))
    g = B.residual_norm_backward(r1, dx=dx, **{k: v for k, v in t.items() if k != "r"})
    rest = B.residual_norm_backward(r1[[0, 2]], dx=dx[[0, 2]], y=t["y"][[0, 2]],
                                    weight=t["weight"], post_weight=t["post_weight"])
    for name in ("dr", "dy"):
        assert (g[name][1] == 0).all() and torch.equal(g[name][[0, 2]], rest[name])
    for name in ("dweight", "dpost_weight"):
        assert torch.isfinite(g[name]).all()


@pytest.mark.parametrize("gate", [None, "token"])
@pytest.mark.parametrize("r,y", [(1e25, 1.0), (1.0, 1e25), (1e14, 1e25), (1e25, 1e14)])
def test_norm_gradients_of_one_norm_past_float32(r, y, gate):
    """Against the oracle with the lost norm's root as 0: the product of y and r passes
    float32's range in the last two."""
    rng = np.random.default_rng(3)
    L, d = 5, 136
    a = make(rng, L, d, "f32", "f32", "weight", gate)
    a["r"][2] *= np.float32(r)
    a["y"][2] *= np.float32(y)
    dx, dr = arr(rng, (L, d), "f32"), arr(rng, (L, d), "f32")
    t = {k: dev(v) for k, v in a.items()}
    got = {k: host(v) for k, v in
           B.residual_norm_backward(t.pop("r"), dx=dev(dx), dr_out=dev(dr), **t).items()}
    b = dict(a)
    if r == 1e25:  # x of that row is 0: dr is dr_out, and so dx may be taken as 0
        dx[2] = 0
    kw = {k: b.get(k) for k in ("y", "post_weight", "gate")}
    want = OB.residual_norm_backward(b["r"], dx, dr, kw["y"], b["weight"], kw["post_weight"], True,
                                     kw["gate"], 1.0, 1e-6)
    for name, g in got.items():
        w, mass = (v.copy() for v in want[name])
        if y == 1e25 and name in ("dy", "dgate"):
            w[2], mass[2] = 0, 0
        if y == 1e25 and name == "dpost_weight":  # without that row's term
            rows = [0, 1, 3, 4]
            part = {k: v[rows] if v is not None and v.shape[0] == L else v for k, v in kw.items()}
            w, mass = OB.residual_norm_backward(b["r"][rows], dx[rows], dr[rows], part["y"],
                                                b["weight"], part["post_weight"], True,
                                                part["gate"], 1.0, 1e-6)[name]
        steps = 100 + (L + 32 if name in ("dweight", "dpost_weight") else 0)
        close(g, w, steps * 2.0 ** -23 * mass + 2.0 ** -24 * 1.001 * np.abs(w) + 1e-36, name)
