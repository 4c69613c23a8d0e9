"""4-bit rows and their products against the oracle.

The rows are exact: codes and scale bytes are compared as they are.  A product of
two elements and their scales is exact in float32, the sum of k of them runs in
steps of 128 with at most k / 128 + 64 additions, each off by 2^-23 of the sum of
the absolute terms at most.  silu(g) u in float32 adds 2^-16 of the value for
|g| <= 12, and the error of either half; bfloat16 results 2^-8 of the value,
float32 ones 2^-24."""
import numpy as np
import pytest
import torch

from oracle import omni_blocks as OB
from oracle import omni_experts as OE
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from tests.gpu_helpers import dev, host

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rows_equal(x):
    q, s = B.microscale_rows(dev(x))
    wq, ws = OB.pack_rows(*OB.microscale_rows(x))
    np.testing.assert_array_equal(host(s), ws)
    np.testing.assert_array_equal(host(q), wq)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,k", [(1, 32), (1, 128), (3, 64), (2, 96), (5, 160), (17, 256),
                                 (4, 704), (2, 1408), (33, 992), (1, 5632)])
def test_rows(R, k, dt):
    rng = np.random.default_rng(R + k)
    x = (rng.standard_normal((R, k)) * 2.0 ** rng.integers(-9, 9, (R, 1))).astype(np.float32)
    x[:, rng.integers(0, k, 2)] *= 30
    rows_equal(f32_to_bf16_bits(x) if dt == "bf16" else x)


def test_rows_borders_zeros_and_what_is_not_finite():
    """Every border between two elements and its neighbours at many scales, the
    smallest and largest numbers, zeros of both signs, NaN and infinities."""
    e = OB.E2M1
    mids = (e[1:] + e[:-1]) / 2
    base = np.concatenate([e, mids, [7.0, 7.999]]).astype(np.float32)
    rows = []
    for p in (-149, -140, -131, -130, -128, -127, -126, -125, -124, -100, -3, 0, 5, 100, 124, 125):
        with np.errstate(over="ignore"):
            v = np.ldexp(base.astype(np.float64), p).astype(np.float32)
        v = v[np.isfinite(v)]
        near = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))])
        near = near[np.isfinite(near)]
        near = np.concatenate([near, -near])
        for i in range(0, len(near), 30):  # each block holds its scale's largest element
            blk = np.zeros(32, np.float32)
            part = near[i:i + 30]
            blk[:len(part)] = part
            top = np.float32(np.ldexp(6.0, p)) if p < 125 else np.float32(v.max())
            blk[31] = top
            rows.append(blk)
    z = np.zeros(32, np.float32)
    rows += [z, -z]
    for bad in (np.nan, np.inf, -np.inf):
        b = np.ones(32, np.float32)
        b[7] = bad
        rows.append(b)
    b = np.ones(32, np.float32)
    b[3], b[4] = np.inf, np.nan
    rows += [b, np.full(32, np.finfo(np.float32).max), np.full(32, 2.0 ** -149, np.float32)]
    while len(rows) % 3:
        rows.append(z)
    x = np.stack(rows).astype(np.float32)
    rows_equal(x)
    rows_equal(x.reshape(-1, 96))
    rows_equal(f32_to_bf16_bits(x))


def test_rows_every_bfloat16():
    """All 65,536 bfloat16 numbers, each in a block of its own scale and of a larger one."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    x = np.zeros((65536 // 16, 32), dtype=np.uint16)
    x[:, :16] = bits.reshape(-1, 16)
    q, s = B.microscale_rows(dev(x))
    v = bf16_bits_to_f32(x).astype(np.float64)
    with np.errstate(invalid="ignore"):
        top = np.abs(v).max(axis=1)
        want = np.where(top > 0, np.maximum(np.frexp(np.where(top > 0, top, 1))[1] - 3, -127), -127)
    finite = np.isfinite(top)
    s = host(s)
    assert (s[~finite, 0] == 255).all() and not host(q)[~finite].any()
    np.testing.assert_array_equal(s[finite, 0], want[finite] + 127)
    got = OB.unpack_rows(host(q)[finite], s[finite])
    unit = 2.0 ** want[finite].astype(float)[:, None]
    a = np.abs(v[finite]) / unit
    dist = np.abs(a[:, :, None] - OB.E2M1).min(axis=2)
    np.testing.assert_array_equal(np.abs(np.abs(got) / unit - a), dist)
    assert (np.signbit(got) == np.signbit(v[finite])).all()


def test_rows_of_many_groups():
    """More rows than one launch wave of workgroups, an odd number of fours of blocks."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5000, 160)).astype(np.float32)
    q, s = B.microscale_rows(dev(x))
    for r in (0, 1, 2047, 2048, 4095, 4999):
        wq, ws = OB.pack_rows(*OB.microscale_rows(x[r:r + 1]))
        np.testing.assert_array_equal(host(q)[r:r + 1], wq)
        np.testing.assert_array_equal(host(s)[r:r + 1], ws)


def packed(rng, shape, spread=3):
    """Random 4-bit rows: every code, scales around one."""
    *lead, k = shape
    q = rng.integers(0, 256, (*lead, k // 2)).astype(np.uint8)
    s = rng.integers(127 - spread, 128 + spread, (*lead, (k + 127) // 128 * 4)).astype(np.uint8)
    return q, s


def values(q, s):
    return OB.unpack_rows(q, s)


def close(got, want, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3],
                           want[bad][:3])


def tol_of(k, mass, want, dt, swiglu):
    t = (k / 128 + 64) * 2.0 ** -23 * mass + HALF[dt] * 1.001 * np.abs(want) + 1e-37
    return t + 2.0 ** -16 * np.abs(want) if swiglu else t


DENSE = [(1, 8, 32), (1, 16, 128), (2, 72, 64), (5, 1, 96), (16, 40, 160), (17, 100, 256),
         (33, 64, 704), (64, 33, 1408), (65, 130, 512), (129, 256, 384), (200, 520, 1056),
         (256, 256, 2048), (300, 264, 640), (513, 136, 224), (1, 3000, 2048), (40, 2048, 5632)]


@pytest.mark.parametrize("M,n,k", DENSE)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_dense(M, n, k, swiglu, dt):
    rng = np.random.default_rng(M + n + k)
    xq, xs = packed(rng, (M, k))
    wq, ws = packed(rng, ((2 if swiglu else 1) * n, k))
    xs, ws = xs - np.uint8(4), ws - np.uint8(4)  # gates within |g| <= 12 or so
    if swiglu:
        ws = ws - np.uint8(3)
    got = B.microscaled_matmul(dev(xq), dev(xs), dev(wq), dev(ws), out_dtype=dt, swiglu=swiglu)
    want, mass = OE.expert_matmul_f64(values(xq, xs), values(wq, ws)[None], np.array([0, M]), M,
                                      np.zeros((M, n)), swiglu=swiglu)
    close(got, want, tol_of(k, mass, want, dt, swiglu), "dense")


EXPERTS = {
    "one_task": ([1], 8, 32),
    "one_row_each": ([1, 0, 1, 1, 0], 72, 160),
    "empty_ends": ([0, 5, 0, 0, 17, 0], 40, 64),
    "all_empty": ([0, 0, 0], 64, 64),
    "tile_edges": ([16, 15, 17, 63, 64, 65, 127, 128, 129, 1], 136, 224),
    "skewed": ([700, 3, 0, 41, 1, 9, 0, 130], 264, 96),
    "many_experts": ([i % 5 for i in range(200)], 48, 96),
    "long_inner": ([33, 2, 90], 152, 3200),
    "wide": ([40, 0, 24], 1408, 704),
    "large": ([300, 520, 0, 256], 512, 1024),
}


@pytest.mark.parametrize("name", EXPERTS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("rows", ["none", "gather", "scatter", "both"])
def test_experts(name, swiglu, rows):
    counts, n, k = EXPERTS[name]
    rng = np.random.default_rng(len(name) + n)
    E, M = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = max(1, M // 2 + 1) if rows in ("gather", "both") else M
    xq, xs = packed(rng, (R, k))
    wq, ws = packed(rng, (E, (2 if swiglu else 1) * n, k))
    xs, ws = xs - np.uint8(4), ws - np.uint8(7 if swiglu else 4)
    xr = rng.integers(0, R, M).astype(np.int32) if rows in ("gather", "both") else None
    Ro = M + 3 if rows in ("scatter", "both") else M
    orow = rng.permutation(Ro)[:M].astype(np.int32) if rows in ("scatter", "both") else None
    for dt in (torch.bfloat16, torch.float32):
        base = np.full((Ro, n), 3.0)
        out = torch.full((Ro, n), 3.0, device="cuda", dtype=dt)
        B.microscaled_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                                    out=out, out_row=dev(orow), swiglu=swiglu)
        want, mass = OE.expert_matmul_f64(values(xq, xs), values(wq, ws), off, M, base, x_row=xr,
                                          out_row=orow, swiglu=swiglu)
        close(out, want, tol_of(k, mass, want, dt, swiglu), (name, rows))


@pytest.mark.parametrize("M", [6, 90, 700])
@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_out_of_range_and_odd_offsets(M, swiglu):
    """Rows out of range give zeros whatever the weights hold (NaN scales among it),
    output rows out of range are dropped, offsets out of order are clamped, tasks
    behind the last offset keep their rows, and NaN scales of rows and weights give
    NaN where they have a part and nowhere else."""
    rng = np.random.default_rng(M)
    E, n, k, R = 4, 264, 416, 50
    off = np.array([0, M // 3, M // 2, M // 2, M - 2], dtype=np.int32)
    xq, xs = packed(rng, (R, k))
    wq, ws = packed(rng, (E, (2 if swiglu else 1) * n, k))
    xs, ws = xs - np.uint8(5), ws - np.uint8(6)
    ws[0, 5, 2] = 255
    xs[7, 12] = 255
    xs[:, 13:], ws[:, :, 13:] = 255, 255  # the rest of the last four: no scales
    xr = rng.integers(0, R, M).astype(np.int32)
    xr[[0, 2, M - 3]] = [-1, R, 2 ** 31 - 1]
    xr[1] = 7
    orow = rng.permutation(M).astype(np.int32)
    orow[[3, 4]] = [-1, M]
    out = torch.full((M, n), 3.0, device="cuda")
    B.microscaled_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                                out=out, out_row=dev(orow), swiglu=swiglu)
    with np.errstate(invalid="ignore"):
        x, w = values(xq, xs), values(wq, ws)
        zero = (xr < 0) | (xr >= R)
        want, mass = OE.expert_matmul_f64(x, w, off, M, np.full((M, n), 3.0), x_row=xr,
                                          out_row=orow, swiglu=swiglu)
    for m in np.nonzero(zero)[0]:
        if off[0] <= m < off[-1] and 0 <= orow[m] < M:
            want[orow[m]], mass[orow[m]] = 0, 0
    mass = np.where(np.isnan(mass), 0, mass)
    close(out, want, tol_of(k, mass, want, torch.float32, swiglu), "odd rows")
    assert np.isnan(want).any()
    # offsets past the tasks, negative and in falling order: nothing outside is touched
    for o in ([-5, M + 9, 2 ** 31 - 1, 0, M], [M, 0, 0, 0, 0], [3, 3, 2, 2, 1]):
        pad = torch.full((M + 2, n), 3.0, device="cuda")
        B.microscaled_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws),
                                    dev(np.array(o, np.int32)), x_row=dev(xr), out=pad[:M],
                                    swiglu=swiglu, out_row=dev(orow))
        assert (pad[M:] == 3).all()


def test_scales_of_the_whole_range():
    """Scales from 2^-127 up, whose products stay among float32's normal numbers."""
    rng = np.random.default_rng(3)
    k, n = 256, 48
    for M in (3, 40, 300):
        xq, xs = packed(rng, (M, k))
        wq, ws = packed(rng, (n, k))
        xs[:] = rng.integers(0, 254, (M, 1))
        ws[:] = (254 - xs[rng.integers(0, M, n), :1].astype(int)).clip(0, 254)
        x, w = values(xq, xs), values(wq, ws)
        got = B.microscaled_matmul(dev(xq), dev(xs), dev(wq), dev(ws), out_dtype=torch.float32)
        want, mass = x @ w.T, np.abs(x) @ np.abs(w).T
        ok = (mass < 2.0 ** 127) & (mass > 2.0 ** -100)
        got = got.double().cpu().numpy()
        tol = (k / 128 + 64) * 2.0 ** -23 * mass
        assert ok.sum() > n and (np.abs(got - want) <= tol)[ok].all()


def test_quantised_product_end_to_end_and_captured():
    rng = np.random.default_rng(9)
    L, E, K, n, k = 75, 6, 2, 200, 352
    x = [rng.standard_normal((L, k)).astype(np.float32) for _ in range(3)]
    w = rng.standard_normal((E * 2 * n, k)).astype(np.float32) / np.float32(np.sqrt(k))
    wq, ws = B.microscale_rows(dev(w))
    wq, ws = wq.view(E, 2 * n, k // 2), ws.view(E, 2 * n, -1)
    counts = rng.multinomial(L * K, np.ones(E) / E)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xr = rng.integers(0, L, L * K).astype(np.int32)
    buf, offd, xrd = dev(x[0]), dev(off), dev(xr)
    q, s = B.microscale_rows(buf)
    out = torch.empty((L * K, n), device="cuda")

    def step(stream=None):
        B.microscale_rows(buf, q=q, scale=s, stream=stream)
        B.microscaled_expert_matmul(q, s, wq, ws, offd, x_row=xrd, out=out, swiglu=True,
                                    stream=stream)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    wv = values(host(wq), host(ws))
    for a in x:
        buf.copy_(dev(a))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        step(other)
        other.synchronize()
        assert torch.equal(got, out)
        av = values(*OB.pack_rows(*OB.microscale_rows(a)))
        want, mass = OE.expert_matmul_f64(av, wv, off, L * K, np.zeros((L * K, n)), x_row=xr,
                                          swiglu=True)
        close(got, want, tol_of(k, mass, want, torch.float32, True), "end to end")
