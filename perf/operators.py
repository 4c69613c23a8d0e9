"""Operators over experts that are matrices, and products in 8-bit integers:
the cases they are measured on, their plain form and their definition in 64
bits.

  matmul     out[o(m)] = x[r(m)] W[e]^T over tasks sorted by expert, ragged
             experts, optionally with the SwiGLU of a gate and an up half
  backward   its input and weight gradients
  combine    y[t] = sum_k g[t, k] o[t K + k], and its backward
  int8       rows made 8-bit with one float32 scale each, then their product
             with 8-bit weights that have a scale for each output channel;
             dense or grouped by expert
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
#
# Keys: L tokens, K experts per token, E experts, active of them that get
# tokens (the rest are empty), zipf the skew of the routing, pad rows behind
# the last task, n outputs, k inputs (of every expert), dt the type.

def listed():
    return [
        # one token of a decoding stream through its experts' gate and up halves
        dict(name="up_token", op="matmul", L=1, K=8, E=64, active=64, zipf=0.0, pad=0,
             n=704, k=2048, dt="bf16", swiglu=True, gather=True, scatter=False),
        # a decoding batch, about 32 rows an expert
        dict(name="up_decode", op="matmul", L=256, K=8, E=64, active=64, zipf=0.5, pad=0,
             n=704, k=2048, dt="bf16", swiglu=True, gather=True, scatter=False),
        # a training batch under skewed routing, gate and up kept for the backward pass
        dict(name="up_train", op="matmul", L=8192, K=8, E=64, active=61, zipf=0.7, pad=0,
             n=1408, k=2048, dt="bf16", swiglu=False, gather=True, scatter=False),
        # float32 experts of a small model, rows scattered back to token order
        dict(name="down_small_f32", op="matmul", L=509, K=8, E=32, active=30, zipf=0.7, pad=5,
             n=128, k=344, dt="f32", swiglu=False, gather=False, scatter=True),
        # gradients of the training batch's product
        dict(name="backward_train", op="backward", L=8192, K=8, E=64, active=61, zipf=0.7, pad=0,
             n=1408, k=2048, dt="bf16"),
        # gradients of a small float32 batch with odd row counts
        dict(name="backward_small_f32", op="backward", L=509, K=8, E=32, active=30, zipf=0.7,
             pad=3, n=344, k=128, dt="f32"),
        # the experts' rows of a training batch summed with their gates
        dict(name="combine_train", op="combine", L=8192, K=8, n=2048, dt="bf16", gates=True),
        # its backward for a smaller, odd batch
        dict(name="combine_backward", op="combine_backward", L=2047, K=6, n=1024, dt="bf16"),
        # one token through an 8-bit dense MLP's gate and up halves
        dict(name="int8_token", op="int8", L=1, K=1, E=0, active=0, zipf=0.0, pad=0, n=5632,
             k=2048, dt="bf16", swiglu=True),
        # a prompt through an 8-bit dense projection
        dict(name="int8_prompt", op="int8", L=8192, K=1, E=0, active=0, zipf=0.0, pad=0,
             n=5632, k=2048, dt="bf16", swiglu=False),
        # a decoding batch through 8-bit experts
        dict(name="int8_experts", op="int8", L=256, K=8, E=64, active=64, zipf=0.5, pad=0,
             n=1408, k=2048, dt="bf16", swiglu=False),
        # an odd prompt through narrower 8-bit experts' gate and up halves
        dict(name="int8_experts_prompt", op="int8", L=2039, K=6, E=32, active=29, zipf=0.9,
             pad=0, n=704, k=1408, dt="bf16", swiglu=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, unit):
    return unit * _between(rng, max(1, lo // unit), hi // unit)


_MOST = 4.0e11  # operations of a drawn product, about those of the largest listed one


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "backward", "backward", "int8", "int8",
                     "combine", "combine_backward"])
    if op in ("combine", "combine_backward"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        K = rng.choice([1, 2, 3, 4, 6, 8])
        n = _width(rng, 64, 4096, 8 if dt == "bf16" else 4)
        L = min(_between(rng, 1, 16384), max(1, 8192 * 8 * 2048 * 2 // (K * n * _SIZE[dt])))
        c = dict(op=op, L=L, K=K, n=n, dt=dt)
        if op == "combine":
            c.update(gates=rng.random() < 0.7)
        return c
    if op == "int8":
        grouped = rng.random() < 0.5
        E = _between(rng, 2, 128) if grouped else 0
        K = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= max(1, E)]) if grouped else 1
        L = _between(rng, 1, 8192)
        n, k = _width(rng, 64, 5632, 8), _width(rng, 128, 5632, 16)
        while max(1, E) * n * k > 1 << 28:
            n = max(64, n // 16 * 8)
        L = max(1, min(L, int(_MOST / (4 * K * n * k))))
        return dict(op=op, L=L, K=K, E=E, active=max(K, E - rng.randint(0, E // 4)) if E else 0,
                    zipf=round(rng.uniform(0, 1.1), 2), pad=0, n=n, k=k,
                    dt=rng.choice(["bf16", "bf16", "f32"]), swiglu=rng.random() < 0.4)
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    u = 8 if dt == "bf16" else 4
    E = _between(rng, 1, 128)
    K = rng.choice([k for k in (1, 2, 3, 4, 6, 8) if k <= E])
    n, k = _width(rng, 64, 4096, u), _width(rng, 64, 4096, u)
    while E * n * k > 1 << 27:
        n, k = max(64, n // (2 * u) * u), max(64, k // (2 * u) * u)
    most = _MOST if dt == "bf16" else _MOST / 8
    L = max(1, min(_between(rng, 1, 16384), int(most / (4 * K * n * k))))
    c = dict(op=op, L=L, K=K, E=E, active=max(K, E - rng.randint(0, E // 4)),
             zipf=round(rng.uniform(0, 1.1), 2), pad=rng.choice([0, 0, 1, 7, 130]), n=n, k=k,
             dt=dt)
    if op == "matmul":
        gather = rng.random() < 0.5
        c.update(swiglu=rng.random() < 0.3, gather=gather,
                 scatter=(not gather) and rng.random() < 0.7)
    return c


# ------------------------------------------------------------------ inputs


def _routing(case, g):
    """Tasks of L tokens sorted by expert: (token, flat index) of each task,
    the experts' offsets, on the GPU and on the host."""
    L, K, E, A = case["L"], case["K"], case["E"], case["active"]
    dev = "cuda"
    order = torch.randperm(E, generator=g, device=dev)[:A]
    logw = -case["zipf"] * torch.log(torch.arange(1, A + 1, device=dev, dtype=torch.float32))
    u = torch.rand((L, A), generator=g, device=dev).clamp_(1e-20, 1 - 1e-7)
    pick = (logw - torch.log(-torch.log(u))).topk(K, dim=1).indices
    eid = order[pick].reshape(-1)
    flat = torch.argsort(eid, stable=True)
    counts = torch.bincount(eid, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = counts.cumsum(0)
    pad = torch.zeros(case["pad"], dtype=torch.int64, device=dev)
    return {"token": torch.cat([flat // K, pad]).int(),
            "flat": torch.cat([flat, L * K + torch.arange(case["pad"], device=dev)]).int(),
            "off": off.int(), "offsets": off.tolist()}


def _normal(shape, g, scale, dt):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    return (t * scale).to(dt)


def _quantized_weights(shape, g):
    """8-bit weights of a Gaussian matrix with a scale for each channel."""
    w = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    top = w.abs().amax(-1, keepdim=True)
    q = torch.round(w * (127.0 / top)).clamp_(-127, 127).to(torch.int8)
    return q, (top.squeeze(-1) / 127.0 / math.sqrt(shape[-1])).contiguous()


def _activations(L, k, g, dt):
    """Rows of unit spread with a few outlying columns, as 8-bit paths meet them."""
    t = torch.empty((L, k), dtype=torch.float32, device="cuda").normal_(generator=g)
    t *= 1 + 15 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    return t.to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op, L, dt = case["op"], case["L"], _DT[case["dt"]]
    if op == "matmul":
        s.update(_routing(case, g))
        M = L * case["K"] + case["pad"]
        s["w"] = _normal((case["E"], (2 if case["swiglu"] else 1) * case["n"], case["k"]), g,
                         1 / math.sqrt(case["k"]), dt)
        s["x"] = _normal((L if case["gather"] else M, case["k"]), g, 1.0, dt)
        s["out"] = torch.zeros((M, case["n"]), dtype=dt, device="cuda")
    elif op == "backward":
        s.update(_routing(case, g))
        M = L * case["K"] + case["pad"]
        s["w"] = _normal((case["E"], case["n"], case["k"]), g, 1 / math.sqrt(case["k"]), dt)
        s["x"] = _normal((L, case["k"]), g, 1.0, dt)
        s["dy"] = _normal((M, case["n"]), g, 0.01, dt)
        s["dx"] = torch.zeros((M, case["k"]), dtype=dt, device="cuda")
        s["dw"] = torch.empty((case["E"], case["n"], case["k"]), device="cuda")
    elif op in ("combine", "combine_backward"):
        K, n = case["K"], case["n"]
        s["o"] = _normal((L * K, n), g, 1.0, dt)
        s["gate"] = torch.softmax(torch.randn((L, K), generator=g, device="cuda"), 1)
        if op == "combine":
            s["y"] = torch.empty((L, n), device="cuda")
        else:
            s["dy"] = _normal((L, n), g, 1.0, torch.float32)
            s["do"], s["dgate"] = torch.empty_like(s["o"]), torch.empty_like(s["gate"])
    else:
        E, k = case["E"], case["k"]
        rows = (2 if case["swiglu"] else 1) * case["n"]
        s["x"] = _activations(L, k, g, dt)
        s["wq"], s["ws"] = _quantized_weights((E, rows, k) if E else (rows, k), g)
        if E:
            s.update(_routing(case, g))
        s["q"] = torch.empty((L, k), dtype=torch.int8, device="cuda")
        s["s"] = torch.empty(L, device="cuda")
        s["out"] = torch.empty((L * case["K"], case["n"]), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from cartesian_routed_atomic_amd import binding as B

    case = s["case"]
    op = case["op"]
    if op == "matmul":
        return B.expert_matmul(s["x"], s["w"], s["off"],
                               x_row=s["token"] if case["gather"] else None,
                               out_row=s["flat"] if case["scatter"] else None, out=s["out"],
                               swiglu=case["swiglu"])
    if op == "backward":
        dx = B.expert_matmul(s["dy"], s["w"], s["off"], x_row=s["flat"], out=s["dx"],
                             out_row=s["flat"], transpose=True)
        dw = B.expert_weight_grad(s["x"], s["dy"], s["off"], x_row=s["token"], dy_row=s["flat"],
                                  dw=s["dw"])
        return dx, dw
    if op == "combine":
        return B.expert_combine(s["o"], case["K"], gate=s["gate"] if case["gates"] else None,
                                y=s["y"])
    if op == "combine_backward":
        return B.expert_combine_backward(s["o"], s["gate"], s["dy"], do=s["do"],
                                         dgate=s["dgate"])
    q, sx = B.quantize_rows(s["x"], q=s["q"], scale=s["s"])
    if case["E"]:
        return B.quantized_expert_matmul(q, sx, s["wq"], s["ws"], s["off"], x_row=s["token"],
                                         out=s["out"], swiglu=case["swiglu"])
    return B.quantized_matmul(q, sx, s["wq"], s["ws"], out=s["out"], swiglu=case["swiglu"])


def _swiglu(z):
    g, u = z.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _quantize(x):
    """Scale and integers of every row; the quotient in 64 bits, since values
    next to a border of two integers need it."""
    top = x.abs().amax(1).double()
    scale = (top / 127).float()
    ratio = x.double() / scale.double().clamp(min=1e-300)[:, None]
    return torch.round(ratio).clamp(-127, 127), scale


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "matmul":
        off, out = s["offsets"], s["out"]
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            xe = s["x"][s["token"][lo:hi]] if case["gather"] else s["x"][lo:hi]
            z = xe.float() @ s["w"][e].float().t()
            z = (_swiglu(z) if case["swiglu"] else z).to(out.dtype)
            if case["scatter"]:
                out[s["flat"][lo:hi]] = z
            else:
                out[lo:hi] = z
        return out
    if op == "backward":
        off, dx, dw = s["offsets"], s["dx"], s["dw"]
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            rows = s["flat"][lo:hi]
            dy = s["dy"][rows].float()
            dx[rows] = (dy @ s["w"][e].float()).to(dx.dtype)
            dw[e] = dy.t() @ s["x"][s["token"][lo:hi]].float()
        return dx, dw
    if op == "combine":
        o = s["o"].float().view(case["L"], case["K"], case["n"])
        if case["gates"]:
            o = o * s["gate"][:, :, None]
        return o.sum(1)
    if op == "combine_backward":
        o = s["o"].float().view(case["L"], case["K"], case["n"])
        do = s["gate"][:, :, None] * s["dy"][:, None, :]
        return (do.to(s["o"].dtype).view(-1, case["n"]), (o * s["dy"][:, None, :]).sum(2))
    q, sx = _quantize(s["x"])
    # the integers' sums pass 24 bits: 64-bit products
    if not case["E"]:
        z = (q @ s["wq"].double().t()).float() * sx[:, None] * s["ws"]
        return (_swiglu(z) if case["swiglu"] else z).to(s["out"].dtype)
    off, out = s["offsets"], s["out"]
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        t = s["token"][lo:hi]
        z = (q[t] @ s["wq"][e].double().t()).float() * sx[t][:, None] * s["ws"][e]
        out[lo:hi] = (_swiglu(z) if case["swiglu"] else z).to(out.dtype)
    return out


# ------------------------------------------------------------------ definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op in ("combine", "combine_backward"):
        L, K, n = case["L"], case["K"], case["n"]
        if op == "combine":
            y = torch.zeros((L, n), dtype=f64, device="cuda")
            for j in range(K):
                row = s["o"][j::K].to(f64)
                y = y + (row * s["gate"][:, j:j + 1].to(f64) if case["gates"] else row)
            return y
        do = torch.empty((L * K, n), dtype=f64, device="cuda")
        dg = torch.empty((L, K), dtype=f64, device="cuda")
        for j in range(K):
            do[j::K] = s["dy"].to(f64) * s["gate"][:, j:j + 1].to(f64)
            dg[:, j] = torch.linalg.vecdot(s["dy"].to(f64), s["o"][j::K].to(f64))
        return do, dg

    def silu_pair(z):
        half = z.shape[1] // 2
        return z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]

    if op == "int8":
        # the scale is a float32 number by definition, the integers follow from it
        x = s["x"].to(f64)
        scale = torch.maximum(x.amax(1), -x.amin(1)).div(127.0).to(torch.float32).to(f64)
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        q = (x / safe.unsqueeze(1)).round()
        q = torch.where(q > 127, 127.0, torch.where(q < -127, -127.0, q))
        rows = q * scale.unsqueeze(1)
        weights = s["wq"] if case["E"] else s["wq"].unsqueeze(0)
        scales = s["ws"] if case["E"] else s["ws"].unsqueeze(0)
    if op == "backward":
        dx = torch.zeros(s["dx"].shape, dtype=f64, device="cuda")
        dw = torch.zeros(s["dw"].shape, dtype=f64, device="cuda")
    else:
        out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    E = case["E"] or 1
    if case["E"]:
        ends = s["off"].to(torch.int64)
        place = torch.arange(int(ends[-1]), device="cuda")
        expert = torch.searchsorted(ends[1:], place, right=True)
    else:
        expert = torch.zeros(case["L"], dtype=torch.int64, device="cuda")
    for e in range(E):
        m = torch.nonzero(expert == e).squeeze(1)
        if m.numel() == 0:
            continue
        if op == "backward":
            to, tok = s["flat"][m].long(), s["token"][m].long()
            dy = s["dy"].index_select(0, to).to(f64)
            dx.index_copy_(0, to, torch.mm(dy, s["w"][e].to(f64)))
            dw[e] = torch.mm(dy.t().contiguous(), s["x"].index_select(0, tok).to(f64))
        elif op == "int8":
            src = rows.index_select(0, s["token"][m].long()) if case["E"] else rows
            w = weights[e].to(f64) * scales[e].to(f64).unsqueeze(1)
            z = torch.mm(src, w.t().contiguous())
            out.index_copy_(0, m, silu_pair(z) if case["swiglu"] else z)
        else:
            src = s["x"].index_select(0, s["token"][m].long() if case["gather"] else m)
            z = torch.mm(src.to(f64), s["w"][e].to(f64).t().contiguous())
            to = s["flat"][m].long() if case["scatter"] else m
            out.index_copy_(0, to, silu_pair(z) if case["swiglu"] else z)
    return (dx, dw) if op == "backward" else out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, L, sz = case["op"], case["L"], _SIZE[case["dt"]]
    K, n = case["K"], case["n"]
    M = L * K
    if op == "combine":
        return {"bytes": M * n * sz + L * n * 4 + (4 * M if case["gates"] else 0),
                "flops": 2 * M * n}
    if op == "combine_backward":
        return {"bytes": 2 * M * n * sz + L * n * 4 + 8 * M, "flops": 3 * M * n}
    k, E = case["k"], case["E"]
    used = min(case["active"], M) if E else 1
    index = 4 * (M + E + 1) if E else 0
    if op == "backward":
        return {"bytes": used * n * k * sz + L * k * sz + M * n * sz + M * k * sz
                + E * n * k * 4 + 2 * index, "flops": 4 * M * n * k}
    rows = (2 if case["swiglu"] else 1) * n
    flops = 2 * M * rows * k
    if op == "int8":
        return {"bytes": used * rows * (k + 4) + L * k * sz + M * n * sz + index,
                "flops": flops}
    read = L if case["gather"] else M
    return {"bytes": used * rows * k * sz + read * k * sz + M * n * sz + index, "flops": flops}
