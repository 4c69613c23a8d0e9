"""A block of matrix experts as a model runs it, through the public calls alone: the
norm before it, the routing, the schedule, the experts (bfloat16 with their
gradients, or 4-bit), the combination, the norm after it with its gate and residual;
forward and backward against float64, and the serving form captured for one token.

Tolerances: the operators' own are tested by themselves; here each stage's oracle
takes the arrays that the stage was given, so that one stage's rounding is not
counted as the next one's error."""
import numpy as np
import pytest
import torch

from oracle import omni_blocks as OB
from oracle import omni_experts as OE
from tests.gpu_helpers import dev, host
from tests.test_gpu_r_norm import arr, backward_close, close

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


def block(t, K, four_bit, groups=2):
    """The block's forward; t: r, weights.  Every array a later stage needs."""
    v = {}
    _, v["x"] = B.residual_norm(t["r"], weight=t["w_pre"])
    E = t["w_route"].shape[0]
    v["logits"] = B.expert_matmul(v["x"], t["w_route"][None], t["one"])
    v["idx"], v["gate"], _ = B.expert_route(v["logits"], K, bias=t["bias"], scores="sigmoid",
                                            groups=groups, top_groups=1, scale=1.5)
    s = v["sched"] = B.schedule_tasks(v["idx"], v["gate"], E, 1, grouping="window")
    off = s.group_offsets
    if four_bit:
        q, qs = B.microscale_rows(v["x"])
        v["h"] = B.microscaled_expert_matmul(q, qs, *t["in4"], off, x_row=s.task_token,
                                             swiglu=True)
        hq, hs = B.microscale_rows(v["h"])
        v["o"] = B.microscaled_expert_matmul(hq, hs, *t["out4"], off, out_row=s.task_index)
    else:
        v["h"] = B.expert_matmul(v["x"], t["w_in"], off, x_row=s.task_token, swiglu=True)
        v["o"] = B.expert_matmul(v["h"], t["w_out"], off, out_row=s.task_index)
    v["y"] = B.expert_combine(v["o"], K, gate=v["gate"])
    v["r1"], v["x1"] = B.residual_norm(t["r"], y=v["y"], weight=t["w_next"],
                                       post_weight=t["w_post"], gate=t["layer"], alpha=0.5)
    return v


def weights(rng, L, d, n, E, rows=None):
    a = {"r": arr(rng, (L, d), "bf16", 2.0), "w_pre": arr(rng, (d,), "bf16", 0.1, 1.0),
         "w_route": arr(rng, (E, d), "bf16", 1 / np.sqrt(d)),
         "w_in": arr(rng, (E, 2 * n, d), "bf16", 1 / np.sqrt(d)),
         "w_out": arr(rng, (E, d, n), "bf16", 1 / np.sqrt(n)),
         "w_post": arr(rng, (d,), "bf16", 0.1, 1.0), "layer": arr(rng, (d,), "bf16", 0.1, 0.5),
         "w_next": arr(rng, (d,), "bf16", 0.1, 1.0)}
    t = {k: dev(v) for k, v in a.items()}
    t["bias"] = dev((0.02 * rng.standard_normal(E)).astype(np.float32))
    t["one"] = dev(np.array([0, L], np.int32))
    for name, w in (("in4", t["w_in"]), ("out4", t["w_out"])):
        q, s = B.microscale_rows(w.view(-1, w.shape[2]))
        t[name] = (q.view(E, w.shape[1], -1), s.view(E, w.shape[1], -1))
    return a, t


@pytest.mark.parametrize("L,d,n,E,K", [(1, 64, 96, 8, 2), (37, 256, 160, 16, 4),
                                       (300, 512, 352, 12, 3)])
@pytest.mark.parametrize("four_bit", [False, True])
def test_block_forward(L, d, n, E, K, four_bit):
    rng = np.random.default_rng(L)
    a, t = weights(rng, L, d, n, E)
    v = block(t, K, four_bit)
    h = {k: host(x) for k, x in v.items() if isinstance(x, torch.Tensor)}
    f = lambda x: OB.widen(x)
    _, x, _ = OB.residual_norm(a["r"], w=a["w_pre"])
    close(h["x"], x, 2.0 ** -8 * 1.01 * np.abs(x) + 1e-6, "x")
    idx, gate, _ = OB.expert_route(h["logits"], K, bias=host(t["bias"]), fn="sigmoid", groups=2,
                                   top_groups=1, scale=1.5)
    np.testing.assert_array_equal(h["idx"], idx)
    close(h["gate"], gate, 1e-5 * np.abs(gate), "gate")
    flat = np.argsort(idx.reshape(-1), kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(idx.reshape(-1), minlength=E))])
    if four_bit:
        rows = lambda q: OB.unpack_rows(*OB.pack_rows(*OB.microscale_rows(q)))
        wide = lambda w: OB.unpack_rows(host(w[0]), host(w[1]))
        xr, hr, w_in, w_out = rows(h["x"]), rows(h["h"]), wide(t["in4"]), wide(t["out4"])
    else:
        xr, hr, w_in, w_out = f(h["x"]), f(h["h"]), f(a["w_in"]), f(a["w_out"])
    M = L * K
    want, mass = OE.expert_matmul_f64(xr, w_in, off, M, np.zeros((M, n)), x_row=flat // K,
                                      swiglu=True)
    close(h["h"], want, 2.0 ** -8 * 1.02 * np.abs(want) + 2.0 ** -14 * mass, "h")
    want, mass = OE.expert_matmul_f64(hr, w_out, off, M, np.zeros((M, d)), out_row=flat)
    close(h["o"], want, 2.0 ** -8 * 1.02 * np.abs(want) + 2.0 ** -14 * mass, "o")
    want, mass = OE.expert_combine_f64(h["o"], K, gate=h["gate"])
    close(h["y"], want, 2.0 ** -20 * mass, "y")
    r1, x1, mass = OB.residual_norm(a["r"], h["y"], a["w_next"], a["w_post"], True, a["layer"], 0.5)
    close(h["r1"], r1, 2.0 ** -8 * 1.01 * np.abs(r1) + 2.0 ** -17 * mass, "r1")
    rms = np.sqrt((r1 * r1).mean(1, keepdims=True))
    close(h["x1"], x1, 2.0 ** -8 * 1.01 * np.abs(x1) + 2.0 ** -15 * mass / rms, "x1")


def test_block_backward():
    """The gradients of the residual, of every weight and of the router's logits."""
    rng = np.random.default_rng(5)
    L, d, n, E, K = 61, 256, 96, 8, 2
    a, t = weights(rng, L, d, n, E)
    # the two products without the SwiGLU between them, whose gradient is the caller's
    t["w_in"] = t["w_in"][:, :n].contiguous()
    a["w_in"] = a["w_in"][:, :n]
    _, x = B.residual_norm(t["r"], weight=t["w_pre"])
    logits = B.expert_matmul(x, t["w_route"][None], t["one"])
    idx, gate, score = B.expert_route(logits, K, bias=t["bias"], scores="softmax", want_score=True)
    s = B.schedule_tasks(idx, gate, E, 1, grouping="window")
    off, tok, flat = s.group_offsets, s.task_token, s.task_index
    h = B.expert_matmul(x, t["w_in"], off, x_row=tok)
    o = B.expert_matmul(h, t["w_out"], off, out_row=flat)
    y = B.expert_combine(o, K, gate=gate)
    r1, x1 = B.residual_norm(t["r"], y=y, weight=t["w_next"], post_weight=t["w_post"],
                             gate=t["layer"], alpha=0.5)
    # backward
    dx1, dr1 = dev(arr(rng, (L, d), "bf16")), dev(arr(rng, (L, d), "bf16"))
    balance = dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    g1 = B.residual_norm_backward(r1, dx=dx1, dr_out=dr1, y=y, weight=t["w_next"],
                                  post_weight=t["w_post"], gate=t["layer"], alpha=0.5)
    do, dgate = B.expert_combine_backward(o, gate, g1["dy"])
    dh = B.expert_matmul(do, t["w_out"], off, x_row=flat, transpose=True)
    dw_out = B.expert_weight_grad(h, do, off, dy_row=flat)
    dxt = B.expert_matmul(dh, t["w_in"], off, out_row=flat, transpose=True)
    dw_in = B.expert_weight_grad(x, dh, off, x_row=tok)
    dz = B.expert_route_backward(logits, idx, dgate, scores="softmax", dscore=balance)
    dx = B.expert_combine(dxt, K)
    B.expert_combine(B.expert_matmul(dz, t["w_route"][None], t["one"], transpose=True), 1, y=dx,
                     accumulate=True)
    dw_route = B.expert_weight_grad(x, dz, t["one"])
    g0 = B.residual_norm_backward(t["r"], dx=dx, dr_out=g1["dr"], weight=t["w_pre"])
    # each stage against its oracle
    backward_close({"r": host(r1), "y": host(y), "weight": a["w_next"], "post_weight": a["w_post"],
                    "gate": a["layer"]}, "bf16", "bf16", True, 0.5, 1e-6, host(dx1), host(dr1), g1)
    wdo, wdg, mass = OE.expert_combine_backward_f64(host(o), host(gate), host(g1["dy"]))
    close(host(do), wdo, 2.0 ** -8 * 1.01 * np.abs(wdo) + 1e-30, "do")
    close(host(dgate), wdg, 2.0 ** -16 * mass, "dgate")
    wdz, mass = OB.expert_route_backward(host(logits), host(idx), host(dgate), "softmax", True, 1.0,
                                         host(balance))
    close(host(dz), wdz, 2.0 ** -8 * 1.01 * np.abs(wdz) + 2.0 ** -15 * mass, "dz")
    offs = host(off)
    wdx, mass = OE.expert_combine_f64(host(dxt), K)
    wr = OB.widen(a["w_route"])
    wdx = wdx + (OB.widen(host(dz)) @ wr)
    mass = mass + np.abs(OB.widen(host(dz))) @ np.abs(wr)
    close(host(dx), wdx, 2.0 ** -7 * mass, "dx")
    for got, xx, dyy, rows in ((dw_out, h, do, dict(dy_row=host(flat))),
                               (dw_in, x, dh, dict(x_row=host(tok)))):
        want, mass = OE.expert_weight_grad_f64(host(xx), host(dyy), offs, L * K, **rows)
        close(host(got), want, 2.0 ** -15 * mass + 1e-30, "dw")
    want, mass = OE.expert_weight_grad_f64(host(x), host(dz), np.array([0, L]), L)
    close(host(dw_route), want, 2.0 ** -15 * mass + 1e-30, "dw_route")
    backward_close({"r": a["r"], "weight": a["w_pre"]}, "bf16", "f32", False, 1.0, 1e-6, host(dx),
                   host(g1["dr"]), g0)
    assert set(g0) == {"dr", "dweight"}


def test_block_of_one_token_captured():
    """The 4-bit block for a single token, captured once and replayed for others."""
    rng = np.random.default_rng(8)
    a, t = weights(rng, 1, 256, 160, 16)
    tokens = [dev(arr(rng, (1, 256), "bf16", 2.0)) for _ in range(3)]
    block(t, 4, True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v = block(t, 4, True)
    for x in tokens:
        t["r"].copy_(x)
        g.replay()
        torch.cuda.synchronize()
        got = {k: v[k].clone() for k in ("idx", "gate", "h", "y", "r1", "x1")}
        eager = block(t, 4, True)
        for k in got:
            assert torch.equal(got[k], eager[k]), k
