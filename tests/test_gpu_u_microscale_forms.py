"""Every kernel form of the 4-bit products against the float64 oracle (tolerances as
in test_gpu_s_microscale.py): rows gathered, scattered and out of range, tasks behind
the last expert's, workgroups that run several tiles in turn."""
import numpy as np
import pytest
import torch

from oracle import omni_experts as OE
from tests import microscale_forms as F
from tests import test_gpu_s_microscale as S
from tests.gpu_helpers import dev, log

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lists", [False, True])
@pytest.mark.parametrize("case", F.CASES, ids=F.name)
def test_forms(case, lists):
    form, _, counts, n, k, swiglu = case
    rng = np.random.default_rng(n + k)
    E, M = len(counts), sum(counts) + F.PAD
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = M // 2 + 1 if lists else M
    xq, xs = S.packed(rng, (R, k), 2)
    wq, ws = S.packed(rng, (E, (2 if swiglu else 1) * n, k), 2)
    # sums of about one: gates within |g| <= 12
    xs, ws = xs - np.uint8(4), ws - np.uint8(6)
    xs[:, k // 32:], ws[:, :, k // 32:] = 255, 255
    xr = orow = None
    if lists:
        xr, orow = rng.integers(0, R, M).astype(np.int32), rng.permutation(M).astype(np.int32)
        xr[3], orow[4] = -1, -1
    dt = torch.float32 if lists else torch.bfloat16
    log(f"[microscaled_expert_matmul] {F.name(case)} lists={lists} M={M}")
    out = torch.full((M, n), 3.0, device="cuda", dtype=dt)
    B.microscaled_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), x_row=dev(xr),
                                out=out, out_row=dev(orow), swiglu=swiglu)
    want, mass = OE.expert_matmul_f64(S.values(xq, xs), S.values(wq, ws), off, M,
                                      np.full((M, n), 3.0), x_row=xr, out_row=orow, swiglu=swiglu)
    S.close(out, want, S.tol_of(k, mass, want, dt, swiglu), F.name(case))


@pytest.mark.parametrize("n", [2424, 1288])
def test_tiles_in_turn_of_overlapping_offsets(n):
    """Offsets out of order that ask for many more tiles than there can be: the call
    ends, and rows past the tasks stay as they were."""
    rng = np.random.default_rng(n)
    E, M, k = 40, 1500, 416
    xq, xs = S.packed(rng, (M, k), 2)
    wq, ws = S.packed(rng, (E, n, k), 2)
    off = np.where(np.arange(E + 1) % 2 == 1, M, 0).astype(np.int32)
    out = torch.full((M + 3, n), 3.0, device="cuda")
    B.microscaled_expert_matmul(dev(xq), dev(xs), dev(wq), dev(ws), dev(off), out=out[:M])
    torch.cuda.synchronize()
    assert (out[M:] == 3).all()


def test_calls_on_two_streams_at_once():
    """Two products of different sizes at once, each as it is alone."""
    rng = np.random.default_rng(1)
    work = []
    for M, n, k in ((3000, 2424, 448), (900, 1288, 800)):
        x, w = S.packed(rng, (M, k), 2), S.packed(rng, (n, k), 2)
        t = [dev(a) for a in (*x, *w)]
        alone = B.microscaled_matmul(*t)
        work.append((t, alone, torch.empty_like(alone), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for t, _, out, s in work:
            B.microscaled_matmul(*t, out=out, stream=s)
    torch.cuda.synchronize()
    for _, alone, out, _ in work:
        assert torch.equal(alone, out)
