"""Products with experts that are matrices, their gradients, the combination
of a token's experts and the 8-bit products, against the float64 oracle.

Tolerances, entry by entry.  A float32 sum of terms with absolute sum S, in
any order of at most c additions, is off by at most c 2^-23 S (each addition,
rounded or cut, by 2^-23 of the partial sum, which S bounds); products of
bf16 numbers are exact in float32, those of float32 numbers off by 2^-24 of
the term (the c + 2 below).  Rounding the result to bf16 adds 2^-8 of it,
to float32 2^-24.  silu(g) u in float32 adds the exponential's error, a few
2^-22 (1 + |g|) relative: 2^-16 covers |g| <= 12.  The 8-bit sum is exact: its
conversion and the two scalings are off by 2^-24 each."""
import numpy as np
import pytest
import torch

from oracle import omni_experts as OE
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from tests.gpu_helpers import dev, host, log

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
gpu = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rand(rng, shape, dt, scale=1.0):
    a = (rng.standard_normal(shape) * scale).astype(np.float32)
    return f32_to_bf16_bits(a) if dt == "bf16" else a


def f32(a):
    return bf16_bits_to_f32(a) if a.dtype == np.uint16 else a


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def close(got, want, tol, what):
    got = f32(got).astype(np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: "
                             f"{got[i]} want {want[i]} tol {tol[i]}")


def sum_tol(c, mass, want, dt):
    return (c + 2) * 2.0 ** -23 * mass + HALF[dt] * np.abs(want) * 1.001 + 1e-38


# name: counts of the experts, n, k
SHAPES = {
    "one_task": ([1], 8, 8),
    "one_row_each": ([1, 0, 1, 1, 0], 72, 136),
    "empty_ends": ([0, 5, 0, 0, 17, 0], 40, 64),
    "all_empty": ([0, 0, 0], 64, 64),
    "tile_edges": ([16, 15, 17, 63, 64, 65, 127, 128, 129, 1], 136, 200),
    "skewed": ([700, 3, 0, 41, 1, 9, 0, 130], 264, 96),
    "many_experts": ([i % 5 for i in range(200)], 48, 72),
    "short_inner": ([33, 2, 90], 152, 8),
    "long_inner": ([3, 9], 24, 2056),
    "wide": ([300, 257], 1032, 40),
    "dense": ([513], 256, 256),
}
PAD = 7  # tasks behind the last expert's


def case(name, dt, seed, gather, scatter, transpose=False, swiglu=False, n=None):
    counts, n0, k = SHAPES[name]
    n = n or n0
    rng = np.random.default_rng(seed)
    off = offsets(counts)
    M = int(off[-1]) + PAD
    R = M // 3 + 2 if gather else M
    inner, width = (n, k) if transpose else (k, n)
    x = rand(rng, (R, inner), dt)
    w = rand(rng, (len(counts), (2 if swiglu else 1) * n, k), dt, 1 / np.sqrt(inner))
    x_row = rng.integers(0, R, M).astype(np.int32) if gather else None
    out_row = rng.permutation(M).astype(np.int32) if scatter else None
    out0 = rand(rng, (M, width), dt)
    return rng, off, M, x, w, x_row, out_row, out0


def check_matmul(name, dt, gather, scatter, transpose=False, swiglu=False, n=None):
    rng, off, M, x, w, xr, orow, out0 = case(name, dt, 11, gather, scatter, transpose, swiglu, n)
    log(f"[expert_matmul] {name} {dt} gather={gather} scatter={scatter} transpose={transpose} "
        f"swiglu={swiglu} M={M} w={w.shape}")
    want, mass = OE.expert_matmul_f64(x, w, off, M, f32(out0), xr, orow, transpose, swiglu)
    out = dev(out0)
    B.expert_matmul(dev(x), dev(w), dev(off), x_row=dev(xr), out=out, out_row=dev(orow),
                    transpose=transpose, swiglu=swiglu)
    got = host(out)
    tol = sum_tol(x.shape[1], mass, want, dt)
    if swiglu:
        tol = tol + 2.0 ** -16 * np.abs(want)
    tol[mass == 0] = 0
    close(got, want, tol, name)
    # rows of no task: untouched, bit for bit
    rows = np.arange(M) if orow is None else orow
    idle = rows[int(off[-1]):]
    np.testing.assert_array_equal(got[idle], out0[idle])


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_expert_matmul(name, dt):
    check_matmul(name, dt, gather=True, scatter=False)
    check_matmul(name, dt, gather=False, scatter=True)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_expert_matmul_transposed(name, dt):
    check_matmul(name, dt, gather=True, scatter=True, transpose=True)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_expert_matmul_swiglu(name, dt):
    check_matmul(name, dt, gather=True, scatter=True, swiglu=True)


# enough tiles for every tile size: counts, outputs, inputs
WIDE = {
    "rows_32": ([64, 65], 512, 520),
    "rows_64": ([129, 200], 256, 264),
    "small": ([510, 3], 2048, 72),
    "mid": ([1020, 5], 4096, 40),
    "wide": ([2041], 4096, 40),
    "big": ([2041, 1800], 4096, 40),
    "big_last_rows": ([5, 3830], 3848, 136),   # a tile with 5 rows, one with 8 columns
}


@gpu
@pytest.mark.parametrize("swiglu", [False, True])
def test_float32_tiles(swiglu, monkeypatch):
    monkeypatch.setitem(SHAPES, "f32_tiles", ([100, 0, 99, 101, 61], 1032 if swiglu else 2056, 72))
    check_matmul("f32_tiles", "f32", gather=True, scatter=True, swiglu=swiglu)


@gpu
@pytest.mark.parametrize("swiglu,transpose", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("name", list(WIDE))
def test_every_tile_size(name, swiglu, transpose, monkeypatch):
    counts, n, k = WIDE[name]
    if transpose:
        n, k = k, n
    monkeypatch.setitem(SHAPES, name, (counts, n // 2 if swiglu else n, k))
    check_matmul(name, "bf16", gather=True, scatter=True, swiglu=swiglu, transpose=transpose)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 33, 255])
def test_expert_matmul_odd_width(dt, n):
    # rows of odd width are not 16-byte aligned
    check_matmul("skewed", dt, gather=True, scatter=False, n=n)
    check_matmul("empty_ends", dt, gather=False, scatter=True, swiglu=True, n=n)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_expert_weight_grad(name, dt):
    counts, n, k = SHAPES[name]
    rng = np.random.default_rng(5)
    off = offsets(counts)
    M = int(off[-1]) + PAD
    x, dy = rand(rng, (M // 2 + 1, k), dt), rand(rng, (M, n), dt)
    xr = rng.integers(0, x.shape[0], M).astype(np.int32)
    yr = rng.permutation(M).astype(np.int32)
    log(f"[expert_weight_grad] {name} {dt} M={M} n={n} k={k}")
    for a, b in ((xr, yr), (None, None), (xr, None)):
        xa = x if a is not None else rand(rng, (M, k), dt)
        want, mass = OE.expert_weight_grad_f64(xa, dy, off, M, a, b)
        dw = torch.full(want.shape, float("nan"), device="cuda")
        B.expert_weight_grad(dev(xa), dev(dy), dev(off), x_row=dev(a), dy_row=dev(b), dw=dw)
        tol = sum_tol(max(counts), mass, want, "f32")
        tol[mass == 0] = 0
        close(host(dw), want, tol, name)


@gpu
@pytest.mark.parametrize("counts,n,k", [
    ([70 + e for e in range(13)], 1032, 760),      # 256 x 256 tiles, short experts
    ([700, 0, 130, 64, 1, 33], 1536, 1280),
    ([9] * 40, 520, 264)])                         # 128 x 128 tiles
def test_expert_weight_grad_large_tiles(counts, n, k):
    rng = np.random.default_rng(16)
    off = offsets(counts)
    M = int(off[-1]) + PAD
    x, dy = rand(rng, (M // 2 + 1, k), "bf16"), rand(rng, (M, n), "bf16")
    xr = rng.integers(0, x.shape[0], M).astype(np.int32)
    yr = rng.permutation(M).astype(np.int32)
    for b in (yr, None):
        want, mass = OE.expert_weight_grad_f64(x, dy, off, M, xr, b)
        dw = torch.full(want.shape, float("nan"), device="cuda")
        B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr), dy_row=dev(b), dw=dw)
        tol = sum_tol(max(counts), mass, want, "f32")
        tol[mass == 0] = 0
        close(host(dw), want, tol, "dw")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,n,k", [
    ([3000], 72, 136),                        # one expert in parts, ragged last part
    ([0, 2500, 0, 1024, 1025, 1, 300, 0], 64, 64),  # parts, one part, none
    ([490 + i * 7 % 90 + (3100 if i % 50 == 1 else 0) for i in range(130)], 24, 16),  # > 64 lanes
    ([5000, 40, 17], 640, 520)])
def test_expert_weight_grad_in_parts(counts, n, k, dt):
    rng = np.random.default_rng(6)
    off = offsets(counts)
    M = int(off[-1]) + PAD
    assert B.lib().omni_expert_weight_grad_workspace(dt == "bf16", M, len(counts), n, k) > 0
    x, dy = rand(rng, (M // 2 + 1, k), dt), rand(rng, (M, n), dt)
    xr = rng.integers(0, x.shape[0], M).astype(np.int32)
    xr[7] = -1
    yr = rng.permutation(M).astype(np.int32)
    want, mass = OE.expert_weight_grad_f64(x, dy, off, M, xr, yr)
    dw = torch.full(want.shape, float("nan"), device="cuda")
    B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr), dy_row=dev(yr), dw=dw)
    tol = sum_tol(max(counts), mass, want, "f32")
    tol[mass == 0] = 0
    close(host(dw), want, tol, "dw in parts")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_out_of_range(dt):
    """x rows out of range count as zeros, output rows out of range are dropped,
    and their tasks add nothing to the weight gradient."""
    rng = np.random.default_rng(8)
    counts, n, k = [40, 0, 77], 72, 64
    off = offsets(counts)
    M = int(off[-1])
    x, w = rand(rng, (50, k), dt), rand(rng, (3, n, k), dt)
    xr = rng.integers(0, 50, M).astype(np.int32)
    xr[[0, 50, 116]] = [-1, 50, 2 ** 31 - 1]
    orow = rng.permutation(M).astype(np.int32)
    orow[[1, 60]] = [M, -5]
    out0 = rand(rng, (M, n), dt)
    want, mass = OE.expert_matmul_f64(x, w, off, M, f32(out0), xr, orow)
    out = dev(out0)
    B.expert_matmul(dev(x), dev(w), dev(off), x_row=dev(xr), out=out, out_row=dev(orow))
    close(host(out), want, sum_tol(k, mass, want, dt) * (mass > 0), "rows")
    dy = rand(rng, (M, n), dt)
    want, mass = OE.expert_weight_grad_f64(x, dy, off, M, xr, orow)
    dw = B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr), dy_row=dev(orow))
    close(host(dw), want, sum_tol(max(counts), mass, want, "f32"), "dw rows")


@gpu
def test_offsets_out_of_order():
    """Offsets outside [0, M] and ends before starts: clamped, nothing outside
    the arrays is touched."""
    rng = np.random.default_rng(9)
    M, n, k = 90, 64, 64
    x, w = rand(rng, (M, k), "bf16"), rand(rng, (4, n, k), "bf16")
    off = np.array([-3, 20, 20, 10, 10 ** 9], dtype=np.int32)  # expert 3: [10, 90)
    out0 = rand(rng, (M, n), "bf16")
    want, mass = OE.expert_matmul_f64(x, w, off, M, f32(out0))
    out = dev(out0)
    B.expert_matmul(dev(x), dev(w), dev(off), out=out)
    got = host(out)
    assert got.shape == (M, n)
    # rows 0 .. 9 are expert 0's alone, rows 20 .. 89 expert 3's alone
    tol = sum_tol(k, mass, want, "bf16")
    close(got[:10], want[:10], tol[:10], "clamped")
    close(got[20:], want[20:], tol[20:], "clamped")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L,K,n", [(1, 1, 8), (1, 8, 2048), (5, 3, 72), (67, 6, 1000),
                                   (300, 2, 128), (33, 64, 264)])
def test_combine(L, K, n, dt):
    rng = np.random.default_rng(L * 100 + K)
    o = rand(rng, (L * K, n), dt)
    gate = rng.random((L, K)).astype(np.float32)
    base = rng.standard_normal((L, n)).astype(np.float32)
    dy = rng.standard_normal((L, n)).astype(np.float32)
    log(f"[combine] L={L} K={K} n={n} {dt}")
    for g in (gate, None):
        for acc in (False, True):
            want, mass = OE.expert_combine_f64(o, K, g, base if acc else None)
            y = dev(base) if acc else torch.full((L, n), float("nan"), device="cuda")
            B.expert_combine(dev(o), K, gate=dev(g), y=y, accumulate=acc)
            close(host(y), want, sum_tol(K, mass, want, "f32"), "combine")
    do, dg, mass = OE.expert_combine_backward_f64(o, gate, dy)
    gdo, gdg = B.expert_combine_backward(dev(o), dev(gate), dev(dy))
    close(host(gdo), do, HALF[dt] * np.abs(do) * 1.001 + 2.0 ** -24 * np.abs(do), "do")
    close(host(gdg), dg, sum_tol(n, mass, dg, "f32"), "dgate")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,k", [(1, 16), (3, 48), (7, 1040), (2, 2064), (2, 4112), (2, 8208),
                                 (2, 16400), (65, 128)])
def test_quantize_rows(R, k, dt):
    rng = np.random.default_rng(R + k)
    x = f32(rand(rng, (R, k), dt))
    x[:, ::7] *= 20
    if R > 2:
        x[1] = 0.0                       # a row of zeros
        x[2, 1:] = 0.0                   # one value alone
    if R > 4:
        x[3] = rng.integers(-254, 255, k) * 0.5 * 2.0 ** -10   # exact halves of the scale: ties
        x[3, 0] = 127 * 2.0 ** -10
        x[3, 1:] = np.clip(x[3, 1:], -126.5 * 2.0 ** -10, 126.5 * 2.0 ** -10)
        x[4] *= np.float32(1e-38)        # near the smallest normal numbers
        x[5] *= np.float32(1e36)        # near the largest
    if dt == "bf16":
        x = f32_to_bf16_bits(x)
    q, s = OE.quantize_rows(x)
    gq, gs = B.quantize_rows(dev(x))
    np.testing.assert_array_equal(host(gs), s)
    np.testing.assert_array_equal(host(gq), q)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", [16, 1040, 2064, 4112, 8208, 16400])
def test_quantize_rows_not_finite(k, dt):
    """A NaN or an infinity anywhere in a row is its scale, q is 0 and a product
    with the row is NaN; the rows beside it are as ever."""
    rng = np.random.default_rng(k)
    x = rng.standard_normal((9, k)).astype(np.float32)
    x[1, 0], x[3, k - 1], x[5, k // 2], x[7, 0], x[7, k - 1] = np.nan, np.inf, -np.inf, np.inf, np.nan
    if dt == "f32":
        x[8, k // 3] = np.array([0xFFFFFFFF], np.uint32).view(np.float32)[0]
        xd = x
    else:
        xd = f32_to_bf16_bits(x)
        xd[1, 0] = xd[7, k - 1] = 0x7FFF
    q, s = OE.quantize_rows(xd)
    assert np.isnan(s[[1, 7]]).all() and np.isinf(s[[3, 5]]).all() and not q[[1, 3, 5, 7]].any()
    gq, gs = B.quantize_rows(dev(xd))
    np.testing.assert_array_equal(host(gs), s)
    np.testing.assert_array_equal(host(gq), q)
    y = B.quantized_matmul(gq, gs, dev(np.ones((8, k), np.int8)), dev(np.ones(8, np.float32)),
                           out_dtype=torch.float32)
    np.testing.assert_array_equal(np.isnan(host(y)).all(axis=1), ~np.isfinite(s))


def q_tol(mass, want, dt, swiglu):
    t = 4 * 2.0 ** -24 * mass + HALF[dt] * np.abs(want) * 1.001 + 1e-38
    return t + 2.0 ** -16 * np.abs(want) if swiglu else t


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,n,k", [(1, 8, 16), (1, 264, 2064), (3, 5, 80), (17, 130, 64),
                                   (130, 136, 144), (257, 520, 96), (64, 1000, 272),
                                   (1030, 2056, 48), (2050, 4096, 16), (4090, 4096, 16)])
def test_quantized_matmul(M, n, k, swiglu, dt):
    rng = np.random.default_rng(M + n + k)
    rows = n * (2 if swiglu else 1)
    xq = rng.integers(-128, 128, (M, k)).astype(np.int8)
    wq = rng.integers(-128, 128, (rows, k)).astype(np.int8)
    xq[0], wq[0] = -128, -128                    # the largest sum
    xs = (rng.random(M) * 2.0 ** -8).astype(np.float32)
    ws = (rng.random(rows) / k ** 0.5 * 2.0 ** -6).astype(np.float32)
    want, mass = OE.expert_matmul_f64(xq.astype(np.float32), wq.astype(np.float32)[None],
                                      [0, M], M, np.zeros((M, n)), swiglu=swiglu, x_scale=xs,
                                      w_scale=ws[None])
    log(f"[quantized_matmul] M={M} n={n} k={k} swiglu={swiglu} {dt}")
    out = B.quantized_matmul(dev(xq), dev(xs), dev(wq), dev(ws), swiglu=swiglu,
                             out_dtype=torch.bfloat16 if dt == "bf16" else torch.float32)
    close(host(out), want, q_tol(mass, want, dt, swiglu), "quantized")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("name", ["one_task", "one_row_each", "empty_ends", "all_empty",
                                  "tile_edges", "many_experts", "skewed", "dense"])
def test_quantized_expert_matmul(name, swiglu, dt):
    counts, n, k = SHAPES[name]
    k = (k + 15) // 16 * 16
    rng = np.random.default_rng(3)
    off = offsets(counts)
    M, E, rows = int(off[-1]) + PAD, len(counts), n * (2 if swiglu else 1)
    R = M // 2 + 1
    xq = rng.integers(-128, 128, (R, k)).astype(np.int8)
    wq = rng.integers(-128, 128, (E, rows, k)).astype(np.int8)
    xs = (rng.random(R) * 2.0 ** -8).astype(np.float32)
    ws = (rng.random((E, rows)) / k ** 0.5 * 2.0 ** -6).astype(np.float32)
    xr = rng.integers(0, R, M).astype(np.int32)
    orow = rng.permutation(M).astype(np.int32)
    out0 = rand(rng, (M, n), dt)
    log(f"[quantized_expert_matmul] {name} swiglu={swiglu} {dt} M={M} n={n} k={k}")
    want, mass = OE.expert_matmul_f64(xq.astype(np.float32), wq.astype(np.float32), off, M,
                                      f32(out0), xr, orow, swiglu=swiglu, x_scale=xs, w_scale=ws)
    out = dev(out0)
    B.quantized_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                              out=out, out_row=dev(orow), swiglu=swiglu)
    got = host(out)
    idle = orow[int(off[-1]):]
    np.testing.assert_array_equal(got[idle], out0[idle])
    busy = orow[:int(off[-1])]
    close(got[busy], want[busy], q_tol(mass[busy], want[busy], dt, swiglu), name)


@gpu
def test_values_of_no_task_do_not_matter():
    """NaN in rows that no task reads, in experts without tasks and behind the
    last task reaches no output."""
    rng = np.random.default_rng(21)
    counts, n, k = [37, 0, 260, 3], 136, 72
    off = offsets(counts)
    M, nan = int(off[-1]) + 40, 0x7FC0
    x, w = rand(rng, (M + 5, k), "bf16"), rand(rng, (4, n, k), "bf16", k ** -0.5)
    dy = rand(rng, (M, n), "bf16")
    xr = rng.permutation(M + 5)[:M].astype(np.int32)
    used = np.zeros(M + 5, bool)
    used[xr[:int(off[-1])]] = True
    x[~used], w[1], dy[int(off[-1]):] = nan, nan, nan
    clean = [np.where(a == nan, 0, a).astype(np.uint16) for a in (x, w, dy)]
    want, mass = OE.expert_matmul_f64(clean[0], clean[1], off, M, np.zeros((M, n)), xr)
    out = torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
    B.expert_matmul(dev(x), dev(w), dev(off), x_row=dev(xr), out=out)
    close(host(out), want, sum_tol(k, mass, want, "bf16") * (mass > 0), "out")
    want, mass = OE.expert_weight_grad_f64(clean[0], clean[2], off, M, xr)
    dw = B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr))
    close(host(dw), want, sum_tol(max(counts), mass, want, "f32"), "dw")
    want, mass = OE.expert_matmul_f64(clean[2], clean[1], off, M, np.zeros((M, k)),
                                      transpose=True)
    dx = torch.zeros((M, k), dtype=torch.bfloat16, device="cuda")
    B.expert_matmul(dev(dy), dev(w), dev(off), out=dx, transpose=True)
    close(host(dx), want, sum_tol(n, mass, want, "bf16") * (mass > 0), "dx")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,n,k", [
    ([300, 0, 5, 61], 72, 136),
    ([9] * 40, 520, 264),
    ([700, 0, 130, 64, 1, 33], 1536, 1280)])
def test_weight_grad_of_tasks_without_a_row(counts, n, k, dt):
    """A task with one row out of range adds nothing, whatever its other row holds."""
    rng = np.random.default_rng(24)
    off = offsets(counts)
    M = int(off[-1])
    x, dy = rand(rng, (M, k), dt), rand(rng, (M, n), dt)
    xr, yr = rng.permutation(M).astype(np.int32), rng.permutation(M).astype(np.int32)
    lost = rng.permutation(M)[:M // 3]
    bad_x, bad_y = lost[::2], lost[1::2]
    nan, inf = (0x7FC0, 0x7F80) if dt == "bf16" else (np.nan, np.inf)
    cx, cy = x.copy(), dy.copy()
    x[xr[bad_y]], dy[yr[bad_x]] = nan, inf
    cx[xr[bad_y]], cy[yr[bad_x]] = 0, 0
    xr[bad_x], yr[bad_y] = -1, M
    want, mass = OE.expert_weight_grad_f64(cx, cy, off, M, xr, yr)
    dw = B.expert_weight_grad(dev(x), dev(dy), dev(off), x_row=dev(xr), dy_row=dev(yr))
    tol = sum_tol(max(counts), mass, want, "f32")
    tol[mass == 0] = 0
    close(host(dw), want, tol, "dw")


@gpu
@pytest.mark.parametrize("steps", [1000, 3424])
def test_long_float32_sums(steps):
    """float32 sums of terms of random sign run in blocks of 128 steps (the last
    up to 240).  A sum's rounding at step i is at most 2^-24 of sqrt(i) terms:
    over a block of b steps b^2 / 2 in squares, over the totals steps^2 / 256; in
    all 64 + steps / 256 + 240^2 / (2 steps), relative to the sum's own steps.
    One accumulator throughout would have steps / 2."""
    bound = 2.0 ** -24 * (64 + steps / 256 + 240 ** 2 / (2 * steps)) ** 0.5
    rng = np.random.default_rng(steps)
    off, M, wide = offsets([150, 170, 90, 200]), 610, 200
    rel = lambda got, want: np.linalg.norm(host(got) - want) / np.linalg.norm(want)
    x, w = rand(rng, (M, steps), "f32"), rand(rng, (4, wide, steps), "f32")
    want, _ = OE.expert_matmul_f64(x, w, off, M, np.zeros((M, wide)))
    assert rel(B.expert_matmul(dev(x), dev(w), dev(off)), want) <= bound
    w = np.ascontiguousarray(w.transpose(0, 2, 1))
    want, _ = OE.expert_matmul_f64(x, w, off, M, np.zeros((M, wide)), transpose=True)
    assert rel(B.expert_matmul(dev(x), dev(w), dev(off), transpose=True), want) <= bound
    x, dy = rand(rng, (steps, 64), "f32"), rand(rng, (steps, 72), "f32")
    want, _ = OE.expert_weight_grad_f64(x, dy, [0, steps], steps)
    assert rel(B.expert_weight_grad(dev(x), dev(dy), dev(offsets([steps]))), want) <= bound


@gpu
def test_thousands_of_experts():
    rng = np.random.default_rng(23)
    counts = rng.integers(0, 3, 3001)
    counts[[0, 700, 3000]] = [0, 400, 90]
    n, k, off = 24, 40, offsets(counts)
    M = int(off[-1])
    x, w, dy = rand(rng, (M, k), "bf16"), rand(rng, (3001, n, k), "bf16"), rand(rng, (M, n), "bf16")
    want, mass = OE.expert_matmul_f64(x, w, off, M, np.zeros((M, n)))
    close(host(B.expert_matmul(dev(x), dev(w), dev(off))), want, sum_tol(k, mass, want, "bf16"),
          "out")
    want, mass = OE.expert_weight_grad_f64(x, dy, off, M)
    close(host(B.expert_weight_grad(dev(x), dev(dy), dev(off))), want,
          sum_tol(400, mass, want, "f32"), "dw")


@gpu
def test_no_tasks():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((3, 32, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert B.expert_matmul(x, w, off).shape == (0, 32)
    dw = torch.full((3, 32, 64), float("nan"), device="cuda")
    B.expert_weight_grad(x, x[:, :32].contiguous(), off, dw=dw)
    assert (dw == 0).all()
    q, s = B.quantize_rows(x)
    assert B.quantized_matmul(q, s, torch.ones((8, 64), dtype=torch.int8, device="cuda"),
                              torch.ones(8, device="cuda")).shape == (0, 8)
    assert B.expert_combine(x, 4).shape == (0, 64)


@gpu
def test_rows_behind_4_gib():
    """Byte offsets of x rows, output rows and experts past 32 bits."""
    rng = np.random.default_rng(22)
    k, n, R = 2048, 2048, (1 << 32) // 4096 + 300
    x = torch.empty((R, k), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((R, n), dtype=torch.bfloat16, device="cuda")
    counts = [40, 33]
    off, M = offsets(counts), 73
    rows = np.concatenate([[0, R - 1], rng.integers((1 << 32) // 4096 - 5, R - 1, M - 2)])
    rows = np.unique(rows)
    rows = np.concatenate([rows, rng.choice(rows, M - rows.size)]).astype(np.int32)
    dst = (R - 1 - rng.permutation(M)).astype(np.int32)
    data = rand(rng, (M, k), "bf16")
    x[torch.from_numpy(rows).long().cuda()] = dev(data)
    data = host(x[torch.from_numpy(rows).long().cuda()].contiguous())  # repeated rows: one value
    w = rand(rng, (2, n, k), "bf16", k ** -0.5)
    want, mass = OE.expert_matmul_f64(data, w, off, M, np.zeros((M, n)))
    B.expert_matmul(x, dev(w), dev(off), x_row=dev(rows), out=out, out_row=dev(dst))
    got = host(out[torch.from_numpy(dst).long().cuda()].contiguous())
    close(got, want, sum_tol(k, mass, want, "bf16"), "far rows")
    want, mass = OE.expert_weight_grad_f64(data, got, off, M)
    dw = B.expert_weight_grad(x, out, dev(off), x_row=dev(rows), dy_row=dev(dst))
    close(host(dw), want, sum_tol(40, mass, want, "f32"), "far dw")
    del x, out, dw
    # experts: the last of 600 weights of 8 MiB
    w = torch.zeros((600, n, k), dtype=torch.bfloat16, device="cuda")
    w[599] = dev(rand(rng, (n, k), "bf16", k ** -0.5))
    off = torch.zeros(601, dtype=torch.int32, device="cuda")
    off[600] = 5
    a = rand(rng, (5, k), "bf16")
    want, mass = OE.expert_matmul_f64(a, host(w[599:].contiguous()), [0, 5], 5, np.zeros((5, n)))
    close(host(B.expert_matmul(dev(a), w, off)), want, sum_tol(k, mass, want, "bf16"), "far w")


@gpu
def test_strides_and_types_are_refused():
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 32, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.expert_matmul(x, w.transpose(1, 2).contiguous().transpose(1, 2), off)
    with pytest.raises(ValueError, match="contiguous"):
        B.expert_matmul(x.t().contiguous().t(), w, off)
    with pytest.raises(TypeError):
        B.expert_matmul(x.half(), w.half(), off)
    with pytest.raises(TypeError, match="w must be"):
        B.expert_matmul(x, w.float(), off)
    with pytest.raises(TypeError, match="offsets"):
        B.expert_matmul(x, w, off.long())
    with pytest.raises(ValueError, match="expected"):
        B.expert_matmul(x, w, off[:2].contiguous())
    with pytest.raises(ValueError, match="expected"):
        B.expert_matmul(x[:, :32].contiguous(), w, off)
    with pytest.raises(ValueError, match="lists 9 tasks"):
        B.expert_matmul(x, w, off, out_row=torch.zeros(9, dtype=torch.int32, device="cuda"))
    with pytest.raises(B.OmniError):
        B.expert_matmul(x, w, off, out=x.new_zeros((4, 32)))   # fewer output rows than tasks
    with pytest.raises(B.OmniError):
        B.quantize_rows(x[:, :24].contiguous())
