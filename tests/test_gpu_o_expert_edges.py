"""Values and rows at the edges of the expert operators' definitions."""
import numpy as np
import pytest
import torch

from oracle import omni_experts as OE
from synth import bf16_bits_to_f32
from tests.gpu_helpers import dev, host, log

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,n,k", [
    ([3, 0, 2], 40, 48),            # few rows
    ([33, 40], 512, 64),            # more rows than few, few tiles
    ([700, 90, 300], 1032, 80)])    # tiles
def test_8_bit_rows_out_of_range_are_zeros_beside_any_scale(counts, n, k, swiglu, dt):
    """As in the float products, a row out of range gives zeros where a weight's scale
    is a NaN or an infinity too."""
    rng = np.random.default_rng(n)
    E, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = n * (2 if swiglu else 1)
    log(f"[quantized_expert_matmul] rows out of range {counts} n={n} k={k} swiglu={swiglu} {dt}")
    xq = rng.integers(-128, 128, (M, k)).astype(np.int8)
    wq = rng.integers(-128, 128, (E, rows, k)).astype(np.int8)
    xs = (rng.random(M) * 2.0 ** -8).astype(np.float32)
    ws = (rng.random((E, rows)) / k ** 0.5 * 2.0 ** -6).astype(np.float32)
    xr = rng.permutation(M).astype(np.int32)
    lost = rng.permutation(M)[:max(2, M // 4)]
    xr[lost] = np.where(np.arange(lost.size) % 2, M, -1)
    out = torch.full((M, n), 7.0, device="cuda",
                     dtype=torch.bfloat16 if dt == "bf16" else torch.float32)
    plain = B.quantized_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                                      out=out.clone(), swiglu=swiglu)
    ws[:, ::3], ws[:, 1::3] = np.nan, np.inf
    B.quantized_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr), out=out,
                              swiglu=swiglu)
    got = host(out.float())
    assert (got[lost] == 0).all()
    kept = np.setdiff1d(np.arange(M), lost)
    # columns with finite scales: as without the others
    cols = np.arange(n) % 3 == 2
    if swiglu:
        cols &= (np.arange(n) + n) % 3 == 2
    np.testing.assert_array_equal(got[kept][:, cols], host(plain.float())[kept][:, cols])
    assert not np.isfinite(got[kept][:, np.arange(n) % 3 == 0]).any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [16, 48, 2064, 16400])
def test_quantized_rows_of_infinities_and_zeros(k, dt):
    """Scales without quotients give q 0 for every value of the row: an infinity of
    either sign, alone, beside zeros, beside the largest number, or all along."""
    big = np.float32(3.3895314e38)   # the largest bf16
    x = np.zeros((7, k), np.float32)
    x[0, k // 2] = -np.inf
    x[1] = np.inf
    x[2, ::2], x[2, 1::2] = -np.inf, big
    x[3, :], x[3, k - 1] = np.nan, np.inf
    x[5] = -big
    x[6] = np.where(np.arange(k) % 3, np.float32(1e-45), 0) if dt == "f32" else 0
    xd = dev(x) if dt == "f32" else dev(x).bfloat16()
    q, s = B.quantize_rows(xd, q=torch.full((7, k), 99, dtype=torch.int8, device="cuda"))
    q, s = host(q), host(s)
    assert (q[[0, 1, 2, 3, 4, 6]] == 0).all() and (q[5] == -127).all()
    assert (s[:3] == np.inf).all() and np.isnan(s[3]) and s[4] == 0 and s[6] == 0
    assert s[5] == np.float32(np.float64(big) / 127)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L,K,n", [(1, 1, 8), (5, 3, 72), (67, 6, 1000), (33, 64, 264)])
def test_combine_backward_without_gates_or_their_gradient(L, K, n, dt):
    """Gates of one (the backward of a sum without gates), and no gradient of the
    gates; through the Python call and the library's own, o missing there."""
    rng = np.random.default_rng(L * 10 + K)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    o = dev(rng.standard_normal((L * K, n)).astype(np.float32)).to(dtype)
    gate = rng.random((L, K)).astype(np.float32)
    dy = rng.standard_normal((L, n)).astype(np.float32)
    log(f"[combine_backward] L={L} K={K} n={n} {dt}")
    ones = np.ones_like(gate)
    want, want_dg, mass = OE.expert_combine_backward_f64(host(o), ones, dy)
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    value = lambda t: host(t.float()).astype(np.float64)
    do, dgate = B.expert_combine_backward(o, None, dev(dy))
    assert (np.abs(value(do) - want) <= half * 1.001 * np.abs(want)).all()
    # a sum of n products in float32, as of any gates
    assert (np.abs(host(dgate) - want_dg) <= (n + 2) * 2.0 ** -23 * mass).all()
    # the same bits as gates that are ones
    do1, dgate1 = B.expert_combine_backward(o, dev(ones), dev(dy))
    assert torch.equal(do, do1) and torch.equal(dgate, dgate1)
    # no gradient of the gates: do as before, o not read
    with_dg, _ = B.expert_combine_backward(o, dev(gate), dev(dy))
    nan = torch.full_like(o, float("nan"))
    for g in (dev(gate), None):
        got, none = B.expert_combine_backward(nan, g, dev(dy), want_dgate=False)
        assert none is None and torch.equal(got, do if g is None else with_dg)
    raw = torch.full_like(o, float("nan"))
    d = dev(dy)
    assert B.lib().omni_expert_combine_backward(
        1 if dt == "bf16" else 0, L, K, n, None, None, d.data_ptr(), raw.data_ptr(), None,
        torch.cuda.current_stream().cuda_stream) == B.OMNI_OK
    torch.cuda.synchronize()
    assert torch.equal(raw, do)


def test_combine_backward_refuses_what_does_not_fit():
    o = torch.zeros((7, 16), device="cuda")
    dy = torch.zeros((2, 16), device="cuda")
    with pytest.raises(ValueError, match="not a multiple"):
        B.expert_combine_backward(o, None, dy)
    with pytest.raises(ValueError, match="not wanted"):
        B.expert_combine_backward(o[:6].contiguous(), None, dy, want_dgate=False,
                                  dgate=torch.zeros((2, 3), device="cuda"))
    with pytest.raises(ValueError, match="expected"):
        B.expert_combine_backward(o, torch.zeros((2, 3), device="cuda"), dy)
    empty = torch.zeros((0, 16), device="cuda")
    do, dgate = B.expert_combine_backward(empty, None, empty)
    assert do.shape == (0, 16) and dgate.shape[0] == 0


@pytest.mark.parametrize("counts,n,k", [([9, 0, 12], 40, 72), ([700, 640], 2056, 328)])
def test_tasks_that_share_an_output_row(counts, n, k):
    """Every element of the row is one of its tasks' results."""
    rng = np.random.default_rng(n)
    E, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = dev(rng.standard_normal((M, k)).astype(np.float32)).bfloat16()
    w = dev((rng.standard_normal((E, n, k)) * k ** -0.5).astype(np.float32)).bfloat16()
    alone = host(B.expert_matmul(x, w, dev(off)).float())
    row = rng.integers(0, M // 2, M).astype(np.int32)
    out0 = rng.standard_normal((M, n)).astype(np.float32)
    out = dev(out0).bfloat16()
    kept = host(out.float())
    B.expert_matmul(x, w, dev(off), out=out, out_row=dev(row))
    got = host(out.float())
    for r in range(M):
        tasks = np.flatnonzero(row == r)
        if tasks.size == 0:
            np.testing.assert_array_equal(got[r], kept[r])
        else:
            assert (alone[tasks] == got[r]).any(axis=0).all()
