"""The expert operators in one run, as a layer of matrix experts uses them:
flat router, schedule (id windows of one expert: its group offsets are the
experts' offsets), gate and up halves with SwiGLU, down product scattered back
to token order, gates applied and summed onto the shared branch; the same in
8 bits; the backward pass; all of it captured into graphs, on other streams
and in two streams at once."""
import numpy as np
import pytest
import torch

from oracle import omni_experts as OE
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from tests.gpu_helpers import dev, host, log, rel_err

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu

L, K, E, D, F = 93, 4, 11, 128, 72


def inputs(seed=3):
    rng = np.random.default_rng(seed)

    def bf(shape, scale=1.0):
        return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))
    return {"x": bf((L, D)), "wf": bf((E, D), D ** -0.5), "w_in": bf((E, 2 * F, D), D ** -0.5),
            "w_out": bf((E, D, F), F ** -0.5),
            "dy": rng.standard_normal((L, D)).astype(np.float32),
            "base": rng.standard_normal((L, D)).astype(np.float32)}


def route(t):
    r = B.flat_router_topk(t["x"], t["wf"], K)
    s = B.schedule_tasks(r["expert_idx"], r["gate"], E, 1, grouping="window")
    return r["gate"], s.task_token, s.task_index, s.group_offsets


def forward(t, gate, token, index, off):
    h = B.expert_matmul(t["x"], t["w_in"], off, x_row=token, swiglu=True)
    o = B.expert_matmul(h, t["w_out"], off, out_row=index)
    return h, o, B.expert_combine(o, K, gate=gate, y=t["base"].clone(), accumulate=True)


def host_routing(off, token, index):
    off, token, index = (host(a) for a in (off, token, index))
    assert off[0] == 0 and off[-1] == L * K and (np.diff(off) >= 0).all()
    np.testing.assert_array_equal(index // K, token)
    np.testing.assert_array_equal(np.sort(index), np.arange(L * K))
    return off, token, index


def test_layer_forward():
    inp = inputs()
    t = {k: dev(v) for k, v in inp.items()}
    gate, token, index, off = route(t)
    h, o, y = forward(t, gate, token, index, off)
    o_, tok, idx = host_routing(off, token, index)
    h_ref, _ = OE.expert_matmul_f64(inp["x"], inp["w_in"], o_, L * K, np.zeros((L * K, F)), tok,
                                    swiglu=True)
    assert rel_err(bf16_bits_to_f32(host(h)), h_ref) <= 2.0 ** -7   # one bf16 rounding each
    o_ref, _ = OE.expert_matmul_f64(host(h), inp["w_out"], o_, L * K, np.zeros((L * K, D)),
                                    out_row=idx)
    assert rel_err(bf16_bits_to_f32(host(o)), o_ref) <= 2.0 ** -7
    y_ref, mass = OE.expert_combine_f64(host(o), K, host(gate), inp["base"])
    assert (np.abs(host(y) - y_ref) <= (K + 2) * 2.0 ** -23 * mass).all()


def test_layer_forward_in_8_bits():
    inp = inputs(4)
    t = {k: dev(v) for k, v in inp.items()}
    gate, token, index, off = route(t)
    o_, tok, idx = host_routing(off, token, index)
    wq, ws = B.quantize_rows(t["w_in"].view(-1, D))
    vq, vs = B.quantize_rows(torch.nn.functional.pad(t["w_out"], (0, 8)).view(-1, F + 8))
    xq, xs = B.quantize_rows(t["x"])
    h = B.quantized_expert_matmul(xq, xs, wq.view(E, 2 * F, D), ws.view(E, 2 * F), off,
                                  x_row=token, swiglu=True)
    hq, hs = B.quantize_rows(torch.nn.functional.pad(h, (0, 8)))
    o = B.quantized_expert_matmul(hq, hs, vq.view(E, D, F + 8), vs.view(E, D), off,
                                  out_row=index, out_dtype=torch.float32)
    y = B.expert_combine(o, K, gate=gate)
    f = lambda a: host(a).astype(np.float32)
    h_ref, mass = OE.expert_matmul_f64(f(xq), f(wq).reshape(E, 2 * F, D), o_, L * K,
                                       np.zeros((L * K, F)), tok, swiglu=True, x_scale=host(xs),
                                       w_scale=host(ws).reshape(E, -1))
    assert rel_err(bf16_bits_to_f32(host(h)), h_ref) <= 2.0 ** -7
    o_ref, _ = OE.expert_matmul_f64(f(hq), f(vq).reshape(E, D, F + 8), o_, L * K,
                                    np.zeros((L * K, D)), out_row=idx, x_scale=host(hs),
                                    w_scale=host(vs).reshape(E, -1))
    assert rel_err(host(o), o_ref) <= 2.0 ** -21
    y_ref, mass = OE.expert_combine_f64(host(o), K, host(gate))
    assert (np.abs(host(y) - y_ref) <= (K + 2) * 2.0 ** -23 * mass).all()
    # 8 bits against bf16: an error of half a step, 1 / 254 of the row's largest
    # value, at each of four roundings, of sums of random sign
    full = forward(t, gate, token, index, off)[2] - t["base"]
    assert rel_err(host(y), host(full)) <= 0.06


def backward(t, gate, token, index, off, gu, h, o):
    """Gradients of sum(y dy); the activation's own derivative in torch."""
    do, dgate = B.expert_combine_backward(o, gate, t["dy"])
    dh = B.expert_matmul(do, t["w_out"], off, x_row=index, transpose=True)
    dw_out = B.expert_weight_grad(h, do, off, dy_row=index)
    g, u = gu.float().chunk(2, 1)
    sg = torch.sigmoid(g)
    dgu = torch.cat([dh.float() * u * sg * (1 + g * (1 - sg)), dh.float() * g * sg],
                    1).bfloat16()
    dx_task = B.expert_matmul(dgu, t["w_in"], off, out_row=index, transpose=True)
    dw_in = B.expert_weight_grad(t["x"], dgu, off, x_row=token)
    return dgate, dw_out, dw_in, B.expert_combine(dx_task, K)


def training_state(t, gate, token, index, off):
    gu = B.expert_matmul(t["x"], t["w_in"], off, x_row=token)
    g, u = gu.float().chunk(2, 1)
    h = (g * torch.sigmoid(g) * u).bfloat16()
    return gu, h, B.expert_matmul(h, t["w_out"], off, out_row=index)


def test_layer_backward_against_autograd():
    inp = inputs(5)
    t = {k: dev(v) for k, v in inp.items()}
    gate, token, index, off = route(t)
    got = backward(t, gate, token, index, off, *training_state(t, gate, token, index, off))
    # the same layer in float64 on the host, differentiated by torch
    d = {k: torch.from_numpy(bf16_bits_to_f32(v) if v.dtype == np.uint16 else v).double()
         for k, v in inp.items()}
    x, w_in, w_out, g = (a.requires_grad_() for a in (d["x"], d["w_in"], d["w_out"],
                                                      gate.cpu().double()))
    o_, tok, idx = host_routing(off, token, index)
    y = torch.zeros(L, D, dtype=torch.float64)
    for e in range(E):
        for m in range(o_[e], o_[e + 1]):
            z = w_in[e] @ x[tok[m]]
            h = torch.nn.functional.silu(z[:F]) * z[F:]
            y = y.index_add(0, torch.tensor([tok[m]]),
                            (g.view(-1)[idx[m]] * (w_out[e] @ h)).unsqueeze(0))
    (y * d["dy"]).sum().backward()
    # every gradient passes at most four bf16 roundings of its factors
    for name, a, want in zip(("dgate", "dw_out", "dw_in", "dx"), got,
                             (g.grad, w_out.grad, w_in.grad, x.grad)):
        err = rel_err(host(a), want.numpy())
        log(f"  {name}: {err:.2e}")
        assert err <= 4 * 2.0 ** -8, name


def everything(t, parts):
    gate, token, index, off = route(t)
    out = list(forward(t, gate, token, index, off))
    out += backward(t, gate, token, index, off, *training_state(t, gate, token, index, off))
    q, s = B.quantize_rows(t["x"])
    out.append(B.quantized_matmul(q, s, parts["wq"], parts["ws"]))
    out.append(B.expert_weight_grad(parts["x"], parts["dy"], parts["off"]))  # in parts: workspace
    return out


def big_parts(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 3000, 3000, 4100], dtype=torch.int32, device="cuda")
    assert B.lib().omni_expert_weight_grad_workspace(1, 4100, 3, 64, 72) > 0
    return {"x": r(4100, 72), "dy": r(4100, 64), "off": off,
            "wq": torch.randint(-127, 128, (40, D), generator=g, device="cuda",
                                dtype=torch.int8),
            "ws": torch.rand(40, generator=g, device="cuda")}


def same(a, b):
    for u, v in zip(a, b):
        assert u.dtype == v.dtype and u.shape == v.shape
        assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8))


def test_graph_replays_match_eager():
    t = {k: dev(v) for k, v in inputs(6).items()}
    parts = big_parts(1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            everything(t, parts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = everything(t, parts)
    for rep in range(4):
        fresh = {k: dev(v) for k, v in inputs(10 + rep).items()}
        for k in t:
            t[k].copy_(fresh[k])
        for o in out:
            o.zero_()
        g.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        want = everything(t, parts)       # eager work between the replays
        torch.cuda.synchronize()
        same(got, want)
        log(f"  replay {rep} bit-identical")


def test_other_streams_and_two_at_once():
    ts = [{k: dev(v) for k, v in inputs(20 + i).items()} for i in range(2)]
    parts = [big_parts(2), big_parts(3)]
    want = [everything(t, p) for t, p in zip(ts, parts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(5):
        got = [None, None]
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = everything(ts[i], parts[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a, b)
    # the stream argument, from another current stream; fresh outputs and workspaces
    p = parts[0]
    ref = B.expert_weight_grad(p["x"], p["dy"], p["off"])
    torch.cuda.synchronize()
    for rep in range(5):
        junk = torch.empty(1 << 22, device="cuda").normal_()   # keeps the current stream busy
        del junk
        dw = B.expert_weight_grad(p["x"], p["dy"], p["off"], stream=streams[rep % 2])
        streams[rep % 2].synchronize()
        same([dw], [ref])


def test_same_inputs_same_bits():
    t = {k: dev(v) for k, v in inputs(7).items()}
    parts = big_parts(4)
    want = everything(t, parts)
    for _ in range(5):
        same(everything(t, parts), want)
