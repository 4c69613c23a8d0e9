"""Routing to experts and its gradient against the float64 oracle.

Tolerances.  The ids are exact: what selects is compared in float64 (or by the
logits).  A score is formed of exponentials of differences of logits, at most D
apart: the difference is off by 2^-24 D, which is that much of the exponential,
the exponential itself by 2^-22; sums of at most E positive terms in at most 24
steps add 24 x 2^-24, the division and the scale 2^-22.  Twice that for a quotient
of two such: (2 D + 32) 2^-23 relative.  A gradient's terms hold at most three such
factors, its sums over K and E terms 64 + 24 steps: (6 D + 160) 2^-23 of the sum of
the absolute terms.  Results below float32's normal numbers: 1e-37.  A rounding to
bfloat16 adds 2^-8 of the value, to float32 2^-24."""
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


def logits(rng, L, E, dt, spread=1.5):
    z = (rng.standard_normal((L, E)) * spread).astype(np.float32)
    return f32_to_bf16_bits(z) if dt == "bf16" else z


def span(z):
    z = OB.widen(z)
    z = z[np.isfinite(z)]
    return float(np.abs(z).max() * 2) if z.size else 0.0


def close(got, want, tol, what):
    got = bf16_bits_to_f32(got) if got.dtype == np.uint16 else got
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], want[bad][:3])


def check(z, K, bias=None, **kw):
    fn = kw.pop("fn", "softmax")
    idx, gate, score = B.expert_route(dev(z), K, bias=dev(bias), scores=fn, want_score=True, **kw)
    wi, wg, ws = OB.expert_route(z, K, bias=bias, fn=fn, **kw)
    np.testing.assert_array_equal(host(idx), wi)
    rel = (2 * span(z) + 32) * 2.0 ** -23
    close(host(gate), wg, rel * np.abs(wg) + 1e-37 * abs(kw.get("scale", 1.0)) + 1e-37, "gate")
    close(host(score), ws, rel * ws + 1e-37, "score")
    return host(idx), host(gate)


SIZES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (5, 7, 3), (17, 60, 6), (33, 64, 64), (64, 65, 4),
         (19, 128, 8), (23, 200, 9), (40, 256, 8), (9, 257, 33), (6, 512, 16), (5, 1000, 64),
         (3, 1024, 1), (130, 96, 2)]


@pytest.mark.parametrize("L,E,K", SIZES)
@pytest.mark.parametrize("fn,biased,renorm", [("softmax", False, True), ("softmax", True, False),
                                              ("sigmoid", False, False), ("sigmoid", True, True)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_sizes(L, E, K, fn, biased, renorm, dt):
    rng = np.random.default_rng(L * 1000 + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    check(logits(rng, L, E, dt), K, bias=bias, fn=fn, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,top,best,K", [
    (8, 8, 3, 2, 3), (8, 8, 8, 1, 8), (16, 4, 1, 2, 4), (60, 5, 2, 1, 7), (64, 8, 4, 2, 8),
    (256, 8, 4, 2, 8), (250, 10, 9, 2, 40), (512, 64, 5, 1, 40), (960, 64, 63, 2, 64),
    (192, 3, 2, 2, 64), (1024, 2, 1, 1, 12)])
@pytest.mark.parametrize("fn,biased", itertools.product(["softmax", "sigmoid"], [False, True]))
def test_route_groups(E, groups, top, best, K, fn, biased):
    rng = np.random.default_rng(E + groups)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    for dt in ("f32", "bf16"):
        check(logits(rng, 37, E, dt), K, bias=bias, fn=fn, groups=groups, top_groups=top,
              group_best=best)


@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8), (1000, 4)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(E, groups, biased):
    """Logits of a few values, zeros of both signs among them, and equal biases."""
    rng = np.random.default_rng(E)
    z = rng.choice(np.array([-1.0, -0.0, 0.0, 0.5], np.float32), (50, E))
    bias = rng.choice(np.array([0.0, 0.25], np.float32), E) if biased else None
    for fn in ("softmax", "sigmoid"):
        for best in (1, 2):
            check(z, 16, bias=bias, fn=fn, groups=groups, top_groups=max(1, groups // 2),
                  group_best=best)
    check(np.zeros((3, E), np.float32), 16, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("E", [64, 256, 1000])
def test_route_scores_next_to_each_other(E):
    """Biased scores that float32 cannot tell apart: their differences are below its
    rounding, and the order is that of float64."""
    rng = np.random.default_rng(E)
    z = (3.0 + rng.integers(0, 4, (40, E)) * 2.0 ** -22).astype(np.float32)
    bias = np.full(E, 0.25, np.float32)
    for fn in ("softmax", "sigmoid"):
        i, _ = check(z, 8, bias=bias, fn=fn)
        j, _ = check(z, 8, fn=fn)
        np.testing.assert_array_equal(i, j)
        check(z, 8, bias=bias, fn=fn, groups=4, top_groups=2, group_best=2)


@pytest.mark.parametrize("E,K,groups,pairs", [
    (40, 4, 1, 3), (64, 8, 4, 6), (128, 16, 1, 10), (256, 8, 8, 8), (256, 8, 1, 120),
    (250, 33, 1, 20), (512, 16, 8, 12), (1000, 60, 4, 40)])
@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
def test_route_pairs_next_to_each_other(E, K, groups, pairs, fn):
    """A few pairs of experts whose biased scores differ by less than float32 tells,
    among the best and about the K-th, in rows that are otherwise well apart."""
    rng = np.random.default_rng(E + K)
    row = logits(rng, 1, E, "f32")[0]
    s = OB.scores(row[None], fn)[0]
    bias = (0.3 * rng.standard_normal(E)).astype(np.float32)
    order = np.argsort(-(s + bias))
    for i in range(pairs):
        a, b = order[2 * i], order[2 * i + 1]
        # the neighbour's bias, a few of its last places to either side
        bias[b] = np.float32(s[a] + np.float64(bias[a]) - s[b])
        for _ in range(rng.integers(0, 3)):
            bias[b] = np.nextafter(bias[b], np.float32(rng.choice([-9, 9])))
    z = np.repeat(row[None], 21, 0)
    z[7:] += np.float32(2.0 ** -9) * rng.standard_normal((14, E)).astype(np.float32)
    z[14:] = logits(rng, 7, E, "f32")
    top = max(1, groups // 2)
    for best in (1, 2):
        check(z, K, bias=bias, fn=fn, groups=groups, top_groups=top, group_best=best)
    check(z, K, bias=bias + np.float32(100.0), fn=fn, groups=groups, top_groups=top)


@pytest.mark.parametrize("fn", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups", [(24, 1), (64, 4), (256, 8), (520, 8)])
def test_route_masks_infinities_and_nan(fn, renorm, E, groups):
    """Masked experts (-infinity and the type's lowest), rows of nothing else, NaN."""
    rng = np.random.default_rng(7)
    z = logits(rng, 12, E, "f32")
    z[1:, : E // 2] = -np.inf
    z[2, :] = -np.inf
    z[3, 3:] = -np.inf
    z[4, :] = np.finfo(np.float32).min
    z[5, 1:] = np.finfo(np.float32).min
    z[6, E // 2 + 1] = np.nan
    z[7, :] = np.nan
    z[8, E // 2 + 2] = np.inf
    z[9, :] = -200.0 - np.arange(E) % 5
    z[10, :] = 120.0 + np.arange(E) % 5
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    low = bias.copy()
    low[E // 2:] = -np.inf
    low[5] = np.nan
    for b in (None, bias, low):
        for K in (1, 8):
            idx, _, _ = B.expert_route(dev(z), K, bias=dev(b), scores=fn, groups=groups,
                                       top_groups=max(1, groups // 2), renormalize=renorm)
            i = host(idx)
            assert ((i >= 0) & (i < E)).all() and all(len(set(r)) == K for r in i.tolist())
            # rows whose oracle ordering is by -infinity alone rank by index, as the kernel's
            check(z, K, bias=b, fn=fn, groups=groups, top_groups=max(1, groups // 2),
                  renormalize=renorm)


@pytest.mark.parametrize("dt,E", [("f32", 256), ("bf16", 60), ("f32", 7)])
def test_route_into_given_arrays_leaves_the_rest(dt, E):
    """Rows behind the last token, and memory beside the outputs, stay as they were."""
    rng = np.random.default_rng(2)
    L, K = 21, 5
    z = logits(rng, L + 3, E, dt)
    idx = torch.full((L + 3, K), -7, dtype=torch.int32, device="cuda")
    gate, score = torch.full((L + 3, K), -7.0, device="cuda"), torch.full((L + 3, E), -7.0,
                                                                          device="cuda")
    dz = torch.full((L + 3, E), -7.0, device="cuda").to(dev(z).dtype)
    zd = dev(z)
    B.expert_route(zd[:L], K, expert_idx=idx[:L], gate=gate[:L], score=score[:L])
    B.expert_route_backward(zd[:L], idx[:L], gate[:L], dlogits=dz[:L])
    for t in (idx, gate, score, dz):
        assert (t[L:] == -7).all() and not (t[:L] == -7).all()
    wi, _, _ = OB.expert_route(z[:L], K)
    np.testing.assert_array_equal(host(idx)[:L], wi)


def test_route_of_no_tokens():
    z = torch.empty((0, 16), device="cuda")
    idx, gate, score = B.expert_route(z, 4, want_score=True)
    assert idx.shape == gate.shape == (0, 4) and score.shape == (0, 16)
    assert B.expert_route_backward(z, idx, gate).shape == (0, 16)


def check_backward(z, idx, dg, fn, renorm, scale, ds, dt):
    dz = B.expert_route_backward(dev(z), dev(idx), dev(dg), scores=fn, renormalize=renorm,
                                 scale=scale, dscore=dev(ds))
    want, mass = OB.expert_route_backward(z, idx, dg, fn, renorm, scale, ds)
    tol = (6 * span(z) + 160) * 2.0 ** -23 * mass + HALF[dt] * 1.001 * np.abs(want) + 1e-37
    close(host(dz), want, tol, "dlogits")


@pytest.mark.parametrize("L,E,K", SIZES)
@pytest.mark.parametrize("fn,renorm,ds", itertools.product(
    ["softmax", "sigmoid"], [True, False], [None, "shared", "full"]))
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_backward(L, E, K, fn, renorm, ds, dt):
    rng = np.random.default_rng(L + E + K)
    z = logits(rng, L, E, dt)
    idx, _, _ = OB.expert_route(z, K, fn=fn)
    dg = rng.standard_normal((L, K)).astype(np.float32)
    shape = {None: None, "shared": (E,), "full": (L, E)}[ds]
    ds = None if shape is None else rng.standard_normal(shape).astype(np.float32)
    check_backward(z, idx.astype(np.int32), dg, fn, renorm, 1.5, ds, dt)


@pytest.mark.parametrize("fn,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("E", [40, 300])
def test_route_backward_ids_twice_and_out_of_range(fn, renorm, E):
    rng = np.random.default_rng(11)
    z = logits(rng, 9, E, "f32")
    z[3, :] = -np.inf
    z[4, 1:] = -np.inf
    z[5, :] = -150.0 + np.arange(E) % 3
    idx = rng.integers(0, E, (9, 6)).astype(np.int32)
    idx[0] = [3, 3, 3, 5, 5, 1]
    idx[1] = [-1, E, 2, 2 ** 31 - 1, -2 ** 31, 4]
    idx[2] = -1
    dg = rng.standard_normal((9, 6)).astype(np.float32)
    for ds in (None, rng.standard_normal(E).astype(np.float32)):
        check_backward(z, idx, dg, fn, renorm, 1.0, ds, "f32")


@pytest.mark.parametrize("fn,renorm", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_route_gradient_against_differences(fn, renorm):
    """The gradient against differences of the gates that the forward itself gives."""
    rng = np.random.default_rng(1)
    L, E, K, h = 4, 24, 3, 2.0 ** -6
    z = logits(rng, L, E, "f32", 0.8)
    idx, _, _ = B.expert_route(dev(z), K, scores=fn, renormalize=renorm)
    dg = rng.standard_normal((L, K)).astype(np.float32)
    dz = host(B.expert_route_backward(dev(z), idx, dev(dg), scores=fn, renormalize=renorm))
    keep = host(idx)

    def loss(z):
        i, g, s = B.expert_route(dev(z), K, scores=fn, renormalize=False, want_score=True)
        w = np.take_along_axis(host(s).astype(np.float64), keep.astype(np.int64), 1)
        return ((w / w.sum(1, keepdims=True) if renorm else w) * dg).sum(1)
    for e in range(E):
        p, m = z.copy(), z.copy()
        p[:, e] += np.float32(h)
        m[:, e] -= np.float32(h)
        diff = (loss(p) - loss(m)) / (p[:, e].astype(np.float64) - m[:, e])
        # h^2 / 6 times a third derivative below 6 |dg|, and float32 scores over 2 h
        tol = (h * h + 2.0 ** -20 / h) * np.abs(dg).sum(1)
        assert (np.abs(diff - dz[:, e]) <= tol).all()


def test_route_captured_and_on_another_stream():
    rng = np.random.default_rng(4)
    z = [logits(rng, 70, 128, "f32") for _ in range(4)]
    dg = rng.standard_normal((70, 6)).astype(np.float32)
    buf, dgd = dev(z[0]), dev(dg)
    idx = torch.empty((70, 6), dtype=torch.int32, device="cuda")
    gate, dz = torch.empty((70, 6), device="cuda"), torch.empty((70, 128), device="cuda")

    def step(stream=None):
        B.expert_route(buf, 6, groups=4, top_groups=2, expert_idx=idx, gate=gate, stream=stream)
        B.expert_route_backward(buf, idx, dgd, dlogits=dz, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for a in z:
        buf.copy_(dev(a))
        g.replay()
        torch.cuda.synchronize()
        got = [host(t).copy() for t in (idx, gate, dz)]
        step()
        for x, t in zip(got, (idx, gate, dz)):
            np.testing.assert_array_equal(x, host(t))
        np.testing.assert_array_equal(got[0], OB.expert_route(a, 6, groups=4, top_groups=2)[0])
