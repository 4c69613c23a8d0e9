"""Every kernel form of the expert operators, with contractions that reach the
pipeline's steady loop, against the float64 oracle (tolerances as in
test_gpu_k_experts.py); sums of the length that training meets by their norm."""
import numpy as np
import pytest
import torch

from oracle import omni_experts as OE
from tests import expert_forms as F
from tests import test_gpu_k_experts as K
from tests.gpu_helpers import dev, host, log

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [c for c in F.PRODUCTS if c[1] != "i8"], ids=F.name)
def test_product_forms(case, monkeypatch):
    form, dt, counts, n, k, transpose, swiglu = case
    assert F.PAD == K.PAD
    monkeypatch.setitem(K.SHAPES, form, (counts, n, k))
    K.check_matmul(form, dt, gather=True, scatter=True, transpose=transpose, swiglu=swiglu)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", [c for c in F.PRODUCTS if c[1] == "i8"], ids=F.name)
def test_quantized_product_forms(case, dt):
    form, _, counts, n, k, _, swiglu = case
    rng = np.random.default_rng(31)
    off = K.offsets(counts)
    M, E, rows = int(off[-1]) + F.PAD, len(counts), n * (2 if swiglu else 1)
    R = M // 2 + 1
    xq = rng.integers(-128, 128, (R, k)).astype(np.int8)
    wq = rng.integers(-128, 128, (E, rows, k)).astype(np.int8)
    xs = (rng.random(R) * 2.0 ** -8).astype(np.float32)
    ws = (rng.random((E, rows)) / k ** 0.5 * 2.0 ** -6).astype(np.float32)
    xr, orow = rng.integers(0, R, M).astype(np.int32), rng.permutation(M).astype(np.int32)
    out0 = K.rand(rng, (M, n), dt)
    log(f"[quantized_expert_matmul] {F.name(case)} out {dt} M={M}")
    want, mass = OE.expert_matmul_f64(xq.astype(np.float32), wq.astype(np.float32), off, M,
                                      K.f32(out0), xr, orow, swiglu=swiglu, x_scale=xs, w_scale=ws)
    out = dev(out0)
    B.quantized_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                              out=out, out_row=dev(orow), swiglu=swiglu)
    got = host(out)
    idle, busy = orow[int(off[-1]):], orow[:int(off[-1])]
    np.testing.assert_array_equal(got[idle], out0[idle])
    K.close(got[busy], want[busy], K.q_tol(mass[busy], want[busy], dt, swiglu), form)


@pytest.mark.parametrize("lists", [True, False])
@pytest.mark.parametrize("case", F.WEIGHT_GRADIENTS, ids=lambda c: F.name(c) + f"-{max(c[3])}")
def test_weight_gradient_forms(case, lists):
    tile, parts, dt, counts, n, k = case
    rng = np.random.default_rng(32)
    off = K.offsets(counts)
    M = int(off[-1]) + F.PAD
    assert (B.lib().omni_expert_weight_grad_workspace(dt == "bf16", M, len(counts), n, k) > 0) \
        == parts
    x, dy = K.rand(rng, (M, k), dt), K.rand(rng, (M, n), dt)
    xr = rng.integers(0, M, M).astype(np.int32) if lists else None
    yr = rng.permutation(M).astype(np.int32) if lists else None
    log(f"[expert_weight_grad] tile {tile} parts {parts} {dt} M={M} n={n} k={k} lists={lists}")
    want, mass = OE.expert_weight_grad_f64(x, dy, off, M, xr, yr)
    dw = torch.full(want.shape, float("nan"), device="cuda")
    B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr), dy_row=dev(yr), dw=dw)
    tol = K.sum_tol(max(counts), mass, want, "f32")
    tol[mass == 0] = 0
    got = host(dw)
    K.close(got, want, tol, "dw")
    # of random signs the roundings of c / 8 additions (of 8 exact products of bf16 each,
    # or of 4 of float32, whose products round too) add up by their squares
    assert relative(got, want) <= norm_bound(max(counts), dt)


def relative(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def norm_bound(c, dt):
    """Relative error of sums of c terms of random sign, kept in float32: a rounding to
    float32 at step i is at most 2^-24 of a partial sum of sqrt(i) terms.  An MFMA adds
    its products (32 steps of bf16, 4 of float32) in groups of 8 at least (4), with a
    rounding each: sum over i = g, 2g, .. c of i, relative to c, is c / (2 g).  float32
    terms are rounded themselves, by 2^-24 at most."""
    return 2.0 ** -24 * (c / 16 + 1 if dt == "bf16" else c / 8 + 2) ** 0.5


@pytest.mark.parametrize("steps", [1000, 3424])
def test_long_float32_sums_of_the_tiles(steps):
    """Products wide enough for the 64 x 64 tiles, whose sums run in blocks of 128 steps:
    the bound of test_gpu_k_experts.py's test_long_float32_sums, whose forward case has
    fewer columns and takes the rows kernel (an eighth of the steps to an accumulator)."""
    bound = 2.0 ** -24 * (64 + steps / 256 + 240 ** 2 / (2 * steps)) ** 0.5
    rng = np.random.default_rng(steps)
    off, M, wide = K.offsets([150, 170, 90, 200]), 610, 840
    x, w = K.rand(rng, (M, steps), "f32"), K.rand(rng, (4, wide, steps), "f32")
    want, _ = OE.expert_matmul_f64(x, w, off, M, np.zeros((M, wide)))
    err = relative(host(B.expert_matmul(dev(x), dev(w), dev(off))), want)
    log(f"  {steps} steps: {err:.2e}, bound {bound:.2e}")
    assert err <= bound


@pytest.mark.parametrize("steps", [1000, 3424])
def test_long_weight_gradient_sums_of_bf16(steps):
    """One expert's tasks in one accumulator (dW of 1024 tiles is not cut into parts):
    the float32 sums of exact products, by their norm over rows of several tiles."""
    rng = np.random.default_rng(steps)
    n = k = 8192
    x, dy = K.rand(rng, (steps, k), "bf16"), K.rand(rng, (steps, n), "bf16")
    assert B.lib().omni_expert_weight_grad_workspace(1, steps, 1, n, k) == 0
    dw = B.expert_weight_grad(dev(x), dev(dy), dev(K.offsets([steps])))
    rows = np.concatenate([np.arange(0, 24), np.arange(250, 262), np.arange(8180, 8192)])
    want, _ = OE.expert_weight_grad_f64(x, np.ascontiguousarray(dy[:, rows]), [0, steps], steps)
    err = relative(host(dw[0, torch.from_numpy(rows).cuda()]), want[0])
    log(f"  {steps} tasks: {err:.2e}, bound {norm_bound(steps, 'bf16'):.2e}")
    assert err <= norm_bound(steps, "bf16")
