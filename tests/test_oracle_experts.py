"""CPU pins of the expert oracle: its products against scalar loops, its
gradients against differences of the forward, its integers against the
definition of nearest."""
import numpy as np
import pytest

from oracle import omni_experts as OE
from oracle.omni_oracle import silu

OFF = np.array([0, 2, 2, 5, 6], dtype=np.int32)
M, N, K = 7, 3, 4  # one task behind the last expert


def case(seed=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((5, K)).astype(np.float32)
    w = rng.standard_normal((4, N, K)).astype(np.float32)
    return rng, x, w, rng.integers(0, 5, M).astype(np.int32), rng.permutation(M).astype(np.int32)


def expert_of(m):
    return next(e for e in range(4) if OFF[e] <= m < OFF[e + 1])


def test_forward_is_the_sum_it_says():
    rng, x, w, xr, orow = case()
    out0 = rng.standard_normal((M, N))
    got, _ = OE.expert_matmul_f64(x, w, OFF, M, out0, xr, orow)
    want = out0.copy()
    for m in range(6):
        e = expert_of(m)
        for j in range(N):
            want[orow[m], j] = sum(float(x[xr[m], c]) * float(w[e, j, c]) for c in range(K))
    np.testing.assert_allclose(got, want, rtol=1e-14, atol=1e-14)


def test_swiglu_and_scales():
    rng, x, w, xr, _ = case(1)
    w2 = np.concatenate([w, rng.standard_normal((4, N, K)).astype(np.float32)], axis=1)
    xs, ws = rng.random(5), rng.random((4, 2 * N))
    got, _ = OE.expert_matmul_f64(x, w2, OFF, M, np.zeros((M, N)), xr, swiglu=True, x_scale=xs,
                                  w_scale=ws)
    for m in range(6):
        e = expert_of(m)
        z = (w2[e].astype(np.float64) @ x[xr[m]]) * xs[xr[m]] * ws[e]
        np.testing.assert_allclose(got[m], silu(z[:N]) * z[N:], rtol=1e-13)


def test_gradients_against_differences():
    rng, x, w, xr, orow = case(2)
    x, w = x.astype(np.float64), w.astype(np.float64)
    dy = rng.standard_normal((M, N))

    def loss(x, w):
        out, _ = OE.expert_matmul_f64(x, w, OFF, M, np.zeros((M, N)), xr, orow)
        return (out * dy).sum()
    dw, _ = OE.expert_weight_grad_f64(x, dy, OFF, M, xr, orow)
    per_task, _ = OE.expert_matmul_f64(dy, w, OFF, M, np.zeros((M, K)), orow, transpose=True)
    dx = np.zeros_like(x)
    for m in range(6):
        dx[xr[m]] += per_task[m]
    h = 1e-5
    for grad, a in ((dw, w), (dx, x)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = loss(x, w)
            a[i] = keep - h
            down = loss(x, w)
            a[i] = keep
            # the loss is linear in each entry: only rounding, about 1e-15 / h, is left
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-8


def test_combine_against_differences():
    rng = np.random.default_rng(3)
    L, k, n = 3, 2, 4
    o, gate, dy = rng.standard_normal((L * k, n)), rng.random((L, k)), rng.standard_normal((L, n))
    do, dg, _ = OE.expert_combine_backward_f64(o, gate, dy)
    f = lambda: (OE.expert_combine_f64(o, k, gate)[0] * dy).sum()
    h = 1e-5
    for grad, a in ((do, o), (dg, gate)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = f()
            a[i] = keep - h
            down = f()
            a[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-8


def test_rows_out_of_range():
    rng, x, w, xr, orow = case(4)
    xr[1], orow[3] = -1, M
    got, _ = OE.expert_matmul_f64(x, w, OFF, M, np.full((M, N), 9.0), xr, orow)
    assert (got[orow[1]] == 0).all()
    assert (got == 9).all(axis=1).sum() == 2      # the dropped row's place and the idle task's
    dw, _ = OE.expert_weight_grad_f64(x, rng.standard_normal((M, N)), OFF, M, xr, orow)
    assert (dw[1] == 0).all()


@pytest.mark.parametrize("seed", range(3))
def test_quantized_rows_are_nearest(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((4, 32)) * 10.0 ** rng.integers(-20, 20, (4, 1))).astype(np.float32)
    x[1] = 0
    q, s = OE.quantize_rows(x)
    assert s[1] == 0 and (q[1] == 0).all()
    for r in (0, 2, 3):
        assert np.abs(q[r]).max() == 127
        ratio = x[r].astype(np.float64) / np.float64(s[r])
        assert (np.abs(ratio - q[r]) <= 0.5 + 1e-12).all()


def test_ties_go_to_even():
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.4999998]], dtype=np.float32)
    q, s = OE.quantize_rows(x)
    assert s[0] == 1.0
    np.testing.assert_array_equal(q[0], [127, 0, 2, 2, 0, -2, -2, 3])


def test_rows_that_are_not_finite():
    x = np.array([[1, np.nan, 2, np.inf], [1, -np.inf, 2, 3], [1, 0, 0, 2]], dtype=np.float32)
    q, s = OE.quantize_rows(x)
    assert np.isnan(s[0]) and s[1] == np.inf and not q[:2].any()
    np.testing.assert_array_equal(q[2], [64, 0, 0, 127])   # 1 / scale = 63.5000002
