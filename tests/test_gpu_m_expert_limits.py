"""The largest sizes that the expert operators take, and their neighbours."""
import pytest
import torch

from tests.gpu_helpers import log

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu

SLICE = 1 << 26


def slices(n):
    return [slice(c, min(c + SLICE, n)) for c in range(0, n, SLICE)]


def test_combine_rows_of_2_to_the_31_columns():
    """The widest rows: every column index, and the step past the last, in 32 bits.
    Values are small whole numbers times powers of two, so every result is exact:
    o is zero but for the first and last 5000 columns, where the sum of 10^4 terms
    of at most 4 x 4 fits 24 bits."""
    n = (1 << 31) - 8
    log(f"[combine] 1 row of {n} columns")
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.empty((1, n), device="cuda")
    for s in slices(n):
        dy[0, s] = torch.randint(-4, 5, (s.stop - s.start,), generator=g, device="cuda").float()
    o = torch.zeros((1, n), dtype=torch.bfloat16, device="cuda")
    for s in (slice(0, 5000), slice(n - 5000, n)):
        o[0, s] = torch.randint(-4, 5, (5000,), generator=g, device="cuda").bfloat16()
    gate = torch.tensor([[0.75]], device="cuda")
    y = B.expert_combine(o, 1, gate=gate)
    for s in slices(n):
        assert torch.equal(y[0, s], 0.75 * o[0, s].float())
    del y
    do = torch.full((1, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    do, dgate = B.expert_combine_backward(o, gate, dy, do=do)
    want = sum((dy[0, s].double() * o[0, s].double()).sum().item()
               for s in (slice(0, 5000), slice(n - 5000, n)))
    assert dgate.item() == want
    for s in slices(n):
        assert torch.equal(do[0, s], (0.75 * dy[0, s]).bfloat16())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantize_rows_of_2_to_the_31_columns(dt):
    """Row indices as above.  The quotient of two numbers of 24 bits is not nearer to
    a half than 2^-26 unless it is one, so its value in 64 bits rounds as the exact
    one does."""
    k = (1 << 31) - 16
    log(f"[quantize_rows] 1 row of {k} columns, {dt}")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((1, k), dtype=dt, device="cuda")
    for s in slices(k):
        x[0, s] = (torch.rand(s.stop - s.start, generator=g, device="cuda") - 0.5).to(dt)
    x[0, k - 3] = -1.25                                     # the largest, in the last step
    q = torch.full((1, k), 99, dtype=torch.int8, device="cuda")
    q, scale = B.quantize_rows(x, q=q)
    want = torch.tensor(1.25, dtype=torch.float64, device="cuda").div(127).float()
    assert scale.item() == want.item()
    for s in slices(k):
        assert torch.equal(q[0, s], torch.round(x[0, s].double() / want.double()).to(torch.int8))


def test_combination_of_2_to_the_26_tasks():
    L, K, n = (1 << 23) + 5, 8, 8
    log(f"[combine] {L} tokens, {K} rows of {n}")
    g = torch.Generator(device="cuda").manual_seed(3)
    o = torch.randint(-8, 9, (L * K, n), generator=g, device="cuda").bfloat16()
    gate = torch.randint(0, 5, (L, K), generator=g, device="cuda").float()
    y = B.expert_combine(o, K, gate=gate)              # whole numbers: every sum is exact
    for s in range(0, L, 1 << 20):
        e = min(L, s + (1 << 20))
        want = (o[s * K:e * K].float().view(-1, K, n) * gate[s:e, :, None]).sum(1)
        assert torch.equal(y[s:e], want)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantize_2_to_the_24_rows(dt):
    R, k = (1 << 24) + 5, 16
    log(f"[quantize_rows] {R} rows of {k}, {dt}")
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((R, k), generator=g, device="cuda").to(dt)
    q, scale = B.quantize_rows(x)
    for s in range(0, R, 1 << 22):
        a = x[s:s + (1 << 22)].double()
        want = (a.abs().amax(1) / 127).float()
        assert torch.equal(scale[s:s + (1 << 22)], want)
        assert torch.equal(q[s:s + (1 << 22)],
                           torch.round(a / want.double()[:, None]).clamp(-127, 127).to(torch.int8))


def test_weight_gradient_of_2_to_the_23_experts():
    E, M = (1 << 23) + 5, 40
    log(f"[expert_weight_grad] {E} experts of 8 x 8")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-4, 5, (M, 8), generator=g, device="cuda").bfloat16()
    dy = torch.randint(-4, 5, (M, 8), generator=g, device="cuda").bfloat16()
    expert = torch.tensor([0] * 3 + [70] * 20 + [1 << 22] * 7 + [E - 1] * 10, device="cuda")
    off = torch.searchsorted(expert, torch.arange(E + 1, device="cuda")).int()
    dw = torch.full((E, 8, 8), float("nan"), device="cuda")
    B.expert_weight_grad(x, dy, off, dw=dw)
    want = torch.zeros((E, 8, 8), device="cuda")
    want.index_add_(0, expert, dy.float()[:, :, None] * x.float()[:, None, :])  # exact
    assert torch.equal(dw, want)
