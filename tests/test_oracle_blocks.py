"""The oracle of routing, residual norms and 4-bit rows against worked values,
against differences of its own forward, and against brute force."""
import itertools

import numpy as np
import pytest

from oracle import omni_blocks as OB


def test_route_worked_example():
    # group values 0.9 + 0.2, 0.8 + 0.4, 0.7 + 0.6: groups 2 and 1 stay
    s = np.array([0.9, 0.2, 0.8, 0.4, 0.7, 0.6])
    z = np.log(s / (1 - s))[None]
    idx, gate, sc = OB.expert_route(z, 3, fn="sigmoid", groups=3, top_groups=2, group_best=2,
                                    scale=2.0)
    assert idx.tolist() == [[2, 4, 5]]
    np.testing.assert_allclose(sc[0], s, rtol=1e-12)
    np.testing.assert_allclose(gate[0], 2 * np.array([0.8, 0.7, 0.6]) / 2.1, rtol=1e-12)
    # the best member alone: groups 0 and 1; the bias selects, the gates do not see it
    idx, gate, _ = OB.expert_route(z, 2, fn="sigmoid", groups=3, top_groups=2, group_best=1,
                                   renormalize=False)
    assert idx.tolist() == [[0, 2]]
    idx, gate, _ = OB.expert_route(z, 2, bias=[0, 0.75, 0, 0, 0, 0], fn="sigmoid",
                                   renormalize=False)
    assert idx.tolist() == [[1, 0]]
    np.testing.assert_allclose(gate[0], [0.2, 0.9], rtol=1e-12)


def test_route_ties_masks_and_nan():
    z = np.array([[1.0, 1.0, 0.0, 1.0], [-np.inf] * 4, [0.0, np.nan, 2.0, -np.inf]])
    idx, gate, s = OB.expert_route(z, 2)
    assert idx.tolist() == [[0, 1], [0, 1], [2, 0]]
    assert gate[1].tolist() == [0, 0] and np.isnan(gate[2]).all() and s[1].tolist() == [0] * 4
    idx, gate, _ = OB.expert_route(z, 2, fn="sigmoid")
    assert idx.tolist() == [[0, 1], [0, 1], [2, 0]] and np.isfinite(gate[2]).all()
    # scores far below float32's range still share out
    idx, gate, _ = OB.expert_route(np.array([[-400.0, -401.0, -500.0]]), 2, fn="sigmoid")
    np.testing.assert_allclose(gate[0], [1 / (1 + np.exp(-1)), 1 / (1 + np.e)], rtol=1e-12)


@pytest.mark.parametrize("fn,renorm,ds", itertools.product(["softmax", "sigmoid"], [True, False],
                                                           [None, "shared", "full"]))
def test_route_backward_against_differences(fn, renorm, ds):
    rng = np.random.default_rng(3)
    L, E, K, scale = 3, 7, 3, 1.7
    z = rng.standard_normal((L, E))
    idx, _, _ = OB.expert_route(z, K, fn=fn)
    dg = rng.standard_normal((L, K))
    dscore = {None: None, "shared": rng.standard_normal(E), "full": rng.standard_normal((L, E))}[ds]

    def loss(z):
        s = OB.scores(z, fn)
        w = np.take_along_axis(s, idx, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (scale * w * dg).sum() + (0.0 if dscore is None else (s * dscore).sum())
    dz, mass = OB.expert_route_backward(z, idx, dg, fn, renorm, scale, dscore)
    h = 1e-5
    for t, e in itertools.product(range(L), range(E)):
        p, m = z.copy(), z.copy()
        p[t, e] += h
        m[t, e] -= h
        assert abs((loss(p) - loss(m)) / (2 * h) - dz[t, e]) < 1e-8
    assert (mass >= np.abs(dz) - 1e-12).all()


@pytest.mark.parametrize("post,gate,use", itertools.product(
    ["none", "ones", "weight"], [None, "column", "token", "full"], ["both", "dx", "dr"]))
def test_norm_backward_against_differences(post, gate, use):
    rng = np.random.default_rng(5)
    L, d, alpha, eps = 3, 5, 0.6, 1e-3
    a = {"r": rng.standard_normal((L, d)), "y": rng.standard_normal((L, d)),
         "weight": rng.standard_normal(d)}
    if post == "weight":
        a["post_weight"] = rng.standard_normal(d)
    if gate:
        a["gate"] = rng.standard_normal({"column": (d,), "token": (L, 1), "full": (L, d)}[gate])
    dx = rng.standard_normal((L, d)) if use != "dr" else None
    dr = rng.standard_normal((L, d)) if use != "dx" else None

    def fwd(a):
        return OB.residual_norm(a["r"], a["y"], a["weight"], a.get("post_weight"), post != "none",
                                a.get("gate"), alpha, eps)

    def loss(a):
        r1, x, _ = fwd(a)
        return (0.0 if dx is None else (x * dx).sum()) + (0.0 if dr is None else (r1 * dr).sum())
    r1 = fwd(a)[0]
    g = OB.residual_norm_backward(r1, dx, dr, a["y"], a["weight"] if dx is not None else None,
                                  a.get("post_weight"), post != "none", a.get("gate"), alpha, eps)
    names = {"r": "dr", "y": "dy", "gate": "dgate", "post_weight": "dpost_weight",
             "weight": "dweight"}
    for name, arr in a.items():
        if name == "weight" and dx is None:
            continue
        got, mass = g[names[name]]
        assert got.shape == arr.shape
        for i in np.ndindex(arr.shape):
            p, m = dict(a), dict(a)
            p[name], m[name] = arr.copy(), arr.copy()
            p[name][i] += 1e-5
            m[name][i] -= 1e-5
            assert abs((loss(p) - loss(m)) / 2e-5 - got[i]) < 1e-7, (name, i)
        assert (mass >= np.abs(got) - 1e-12).all()


def test_norm_alone_and_zero_row():
    r = np.array([[3.0, 4.0], [0.0, 0.0]])
    _, x, _ = OB.residual_norm(r, eps=0.5)
    np.testing.assert_allclose(x[0], r[0] / np.sqrt(13.0))
    assert x[1].tolist() == [0, 0]


def test_microscale_worked_values():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :12] = [6, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.0, 7]
    x[0, 32] = 2.0 ** -130
    code, byte = OB.microscale_rows(x)
    assert byte.tolist() == [[127, 0]]
    q, scale = OB.pack_rows(code, byte)
    v = OB.unpack_rows(q, scale)
    assert v[0, :12].tolist() == [6, 0, 0.5, 1, 1, 2, 2, 4, 4, -4, 0, 6]
    assert code[0, 10] == 8 and scale.tolist() == [[127, 0, 127, 127]]
    assert v[0, 32] == 0  # 2^-130 is an eighth of the scale 2^-127
    x[0, 40] = np.nan
    code, byte = OB.microscale_rows(x)
    assert byte[0, 1] == 255 and not code[0, 32:].any()


def test_microscale_rounds_to_the_nearest():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((4, 96)) * 2.0 ** rng.integers(-20, 20, (4, 96))).astype(np.float32)
    code, byte = OB.microscale_rows(x)
    v = OB.unpack_rows(*OB.pack_rows(code, byte))
    unit = np.repeat(2.0 ** (byte.astype(float) - 127), 32, axis=1)
    grid = np.concatenate([-OB.E2M1[::-1], OB.E2M1])
    best = np.abs(x[..., None] / unit[..., None] - grid).min(axis=-1)
    np.testing.assert_array_equal(np.abs(x - v) / unit, best)
    top = np.abs(x).reshape(4, 3, 32).max(axis=2)
    s = 2.0 ** (byte.astype(float) - 127)
    assert ((top >= 4 * s) & (top < 8 * s)).all()
