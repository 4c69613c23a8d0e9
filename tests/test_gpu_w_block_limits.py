"""Routing, residual norms and 4-bit rows where arrays pass 2^31 elements, where results
go over inputs, and with two calls under way at once.

Rows do not depend on the rest of the batch, so what is far down an array is compared
bit for bit with a call on those rows alone; 4-bit products of whole numbers below
2^24 are exact in float32 whatever their order."""
import numpy as np
import pytest
import torch

from synth import f32_to_bf16_bits
from tests.gpu_helpers import dev

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(rng, shape, dt, scale=1.0):
    a = (rng.standard_normal(shape) * scale).astype(np.float32)
    return dev(f32_to_bf16_bits(a)) if dt is BF else dev(a)


def far(L, d, dt, rows):
    """[L, d] of zeros with rows at its end."""
    a = torch.zeros(L, d, dtype=dt, device="cuda")
    a[L - len(rows):] = rows
    return a


def test_route_past_32_bits():
    rng = np.random.default_rng(1)
    L, E, K, n = (1 << 21) + 5, 1024, 9, 5
    z = far(L, E, BF, rand(rng, (n, E), BF, 2.0))
    bias = rand(rng, (E,), F32, 0.01)
    idx, gate, _ = B.expert_route(z, K, bias=bias, scores="sigmoid", groups=8, top_groups=3)
    alone = B.expert_route(z[-n:], K, bias=bias, scores="sigmoid", groups=8, top_groups=3)
    assert torch.equal(idx[-n:], alone[0]) and torch.equal(gate[-n:], alone[1])
    dg = torch.zeros(L, K, device="cuda")
    dg[-n:] = rand(rng, (n, K), F32)
    dz = B.expert_route_backward(z, idx, dg, renormalize=False)
    want = B.expert_route_backward(z[-n:], idx[-n:].contiguous(), dg[-n:].contiguous(),
                                   renormalize=False)
    assert torch.equal(dz[-n:], want) and not (dz[:-n] != 0).any() and (want != 0).any()


@pytest.mark.parametrize("dt,L,d", [(BF, (1 << 20) + 3, 2056), (F32, (1 << 18) + 3, 8196)])
def test_norm_past_32_bits(dt, L, d):
    rng = np.random.default_rng(2)
    n = 3
    ends = [rand(rng, (n, d), dt) for _ in range(2)]
    w = rand(rng, (d,), dt)
    r, y = (far(L, d, dt, v) for v in ends)
    r1, x = B.residual_norm(r, y=y, weight=w, r_out=r, gate=w, post=True)
    a, b = B.residual_norm(ends[0], y=ends[1], weight=w, gate=w, post=True)
    assert r1 is r and torch.equal(a, r[-n:]) and torch.equal(b, x[-n:])
    small = B.residual_norm_backward(a, dx=ends[1], dr_out=b, weight=w)
    got = B.residual_norm_backward(r, dx=y, dr_out=x, weight=w, out={"dr": x})
    assert got["dr"] is x and torch.equal(x[-n:], small["dr"]) and (x[:5] == 0).all()
    # the rows before are zeros: three terms, perhaps in another order
    a, p = a.double(), ends[1].double()
    terms = (p * a * (a.square().mean(1, keepdim=True) + 1e-6).rsqrt()).abs().sum(0)
    diff = (got["dweight"].double() - small["dweight"].double()).abs()
    assert (diff <= 5 * 2.0 ** -24 * terms).all() and (small["dweight"] != 0).any()


def test_microscale_past_32_bits():
    rng = np.random.default_rng(3)
    R, k, n = (1 << 20) + 3, 2080, 3
    x = far(R, k, BF, rand(rng, (n, k), BF))
    q, s = B.microscale_rows(x)
    a, b = B.microscale_rows(x[-n:])
    assert torch.equal(q[-n:], a) and torch.equal(s[-n:], b)
    assert not q[:-n].any() and not s[:4, :k // 32].any()


@pytest.mark.parametrize("M", [3, 700])
@pytest.mark.parametrize("swiglu", [False, True])
def test_microscaled_experts_past_32_bits(M, swiglu):
    """Weights of 4 GiB: all tasks go to the last expert."""
    g = torch.Generator(device="cuda").manual_seed(M)
    E, rows, k = 65, 8192, 16384
    G = k // 32

    def codes(*shape):  # 0.5, 1, 1.5 and their negatives
        lo = torch.randint(1, 4, shape, generator=g, device="cuda", dtype=torch.uint8)
        hi = torch.randint(9, 12, shape, generator=g, device="cuda", dtype=torch.uint8)
        return lo | hi << 4
    wq = torch.zeros(E, rows, k // 2, dtype=torch.uint8, device="cuda")
    ws = torch.full((E, rows, G), 120, dtype=torch.uint8, device="cuda")
    wq[-1] = codes(rows, k // 2)
    xq, xs = codes(M, k // 2), torch.full((M, G), 127, dtype=torch.uint8, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = M
    assert wq.numel() > 1 << 32
    out = B.microscaled_expert_matmul(xq, xs, wq, ws, off, out_dtype=F32, swiglu=swiglu)
    want = B.microscaled_matmul(xq, xs, wq[-1], ws[-1], out_dtype=F32, swiglu=swiglu)
    assert torch.equal(out, want) and (out != 0).any()


@pytest.mark.parametrize("dt,d", [(BF, 200), (BF, 1000), (BF, 2048), (BF, 4104), (BF, 8200),
                                  (F32, 256), (F32, 520), (F32, 4096), (F32, 8192), (F32, 16384)])
def test_norm_results_over_their_inputs(dt, d):
    """r_out over r; dr over dr_out, or over dx, and dy over y; more rows than workgroups."""
    rng = np.random.default_rng(d)
    L = (1 << 20) // d + 600
    r, y, dx, up = (rand(rng, (L, d), dt) for _ in range(4))
    w, pw, gate = (rand(rng, (d,), dt) for _ in range(3))
    kw = dict(weight=w, post_weight=pw, gate=gate, alpha=0.5)
    r1, x = B.residual_norm(r, y=y, **kw)
    r2 = r.clone()
    assert B.residual_norm(r2, y=y, r_out=r2, **kw)[0] is r2 and torch.equal(r1, r2)
    want = B.residual_norm_backward(r1, dx=dx, dr_out=up, y=y, **kw)
    for over in ("dr_out", "dx"):
        t = {"dx": dx.clone(), "dr_out": up.clone(), "y": y.clone()}
        got = B.residual_norm_backward(r1, **t, **kw, out={"dr": t[over], "dy": t["y"]})
        for name in want:
            assert torch.equal(got[name], want[name]), (over, name)


@pytest.mark.parametrize("d,L", [(96, 9000), (16384, 300)])
def test_norm_sums_do_not_depend_on_the_run(d, L):
    rng = np.random.default_rng(d)
    r, dx = rand(rng, (L, d), BF), rand(rng, (L, d), F32)
    w = torch.ones(d, device="cuda", dtype=BF)
    a, b = (B.residual_norm_backward(r, dx=dx, weight=w) for _ in range(2))
    assert torch.equal(a["dweight"], b["dweight"]) and torch.equal(a["dr"], b["dr"])
    # dw: dx r1 a over the rows, a's relative error 40 x 2^-23, L + 32 additions
    terms = dx.double() * r.double() * (r.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
    tol = (40 * 2.0 ** -23 + (L + 32) * 2.0 ** -24) * terms.abs().sum(0)
    assert ((a["dweight"].double() - terms.sum(0)).abs() <= tol).all()


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(5)
    L, d, E = 4000, 1024, 128
    sets = [(rand(rng, (L, d), BF), rand(rng, (L, d), F32), rand(rng, (L, E), F32)) for _ in range(2)]
    w = torch.ones(d, device="cuda", dtype=BF)

    def step(r, dx, z, stream=None):
        n = B.residual_norm_backward(r, dx=dx, weight=w, stream=stream)
        idx, gate, _ = B.expert_route(z, 6, stream=stream)
        return [n["dr"], n["dweight"], idx, gate,
                B.expert_route_backward(z, idx, gate, stream=stream),
                *B.microscale_rows(r, stream=stream)]
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = [step(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for p, q in zip(a, b):
                assert torch.equal(p, q)


def test_route_of_the_most_tokens():
    """2^26 - 4 of them, four to a workgroup: 2^32 - 256 work-items."""
    rng = np.random.default_rng(6)
    L, E, K, n = (1 << 26) - 4, 17, 17, 6
    ends = rand(rng, (n, E), BF, 2.0)
    z = far(L, E, BF, ends)
    idx, gate, _ = B.expert_route(z, K, scores="sigmoid")
    alone = B.expert_route(ends, K, scores="sigmoid")
    assert torch.equal(idx[-n:], alone[0]) and torch.equal(gate[-n:], alone[1])
    # equal logits: the experts in order, an equal share each
    assert (idx[:-n] == torch.arange(K, device="cuda", dtype=torch.int32)).all()
    assert (gate[:-n] == gate[0, 0]).all() and abs(float(gate[0, 0]) - 1 / K) < 1e-6
    dz = B.expert_route_backward(z, idx, gate, scores="sigmoid", renormalize=False)
    want = B.expert_route_backward(ends, alone[0], alone[1], scores="sigmoid", renormalize=False)
    assert torch.equal(dz[-n:], want) and (dz[:-n] == dz[0, 0]).all() and (want != 0).all()
