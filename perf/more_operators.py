"""What a block of matrix experts has around its products: the cases these
operators are measured on, their plain form and their definition in 64 bits.

  route           a token's experts and gates from its logits: softmax or
                  sigmoid scores, a balance bias, groups, top-K, renormalised
  route_backward  the gradient of the logits
  norm            r1 = r + alpha g n(y), x = n(r1): the norm after a block with
                  its gate and residual scale, fused with the norm before the next
  norm_backward   its gradients
  mx              rows made 4-bit floating point with a scale for each 32
                  elements, then their product with weights of that form;
                  dense or grouped by expert
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
#
# Keys: L tokens, E experts, K experts per token, dt the type.  route: fn the
# scores, groups, top groups that stay, best members that make a group's value,
# bias, renorm, scale.  norm: y the type of the block's output ("" without one),
# post whether it is normed, gate "", "column", "token" or "full", dx the type of
# x's gradient.  mx: n outputs, k inputs, out the type of the product.

def listed():
    return [
        # one token of a decoding stream, its logits bfloat16: softmax over 64 experts, 8 kept
        dict(name="route_token", op="route", L=1, E=64, K=8, fn="softmax", groups=1, top=1,
             best=1, bias=False, renorm=True, scale=1.0, dt="bf16", scores=False),
        # a training batch: sigmoid scores with a balance bias, 4 of 8 groups, scores kept
        # for a balance loss
        dict(name="route_train", op="route", L=16384, E=256, K=8, fn="sigmoid", groups=8, top=4,
             best=2, bias=True, renorm=True, scale=2.5, dt="f32", scores=True),
        # gradients of the training batch, a balance loss's share among them
        dict(name="route_backward_train", op="route_backward", L=16384, E=256, K=8, fn="sigmoid",
             renorm=True, scale=2.5, dt="f32", dscore="column"),
        # gradients of a small odd softmax batch without renormalisation
        dict(name="route_backward_small", op="route_backward", L=509, E=60, K=6, fn="softmax",
             renorm=False, scale=1.0, dt="bf16", dscore="full"),
        # the norm before a block for one token of a decoding stream
        dict(name="norm_token", op="norm", L=1, d=2048, dt="bf16", y="bf16", post=False, gate=""),
        # a training batch: the experts' float32 sum normed, scaled by column, added, normed
        dict(name="norm_train", op="norm", L=8192, d=2048, dt="bf16", y="f32", post=True,
             gate="column"),
        # its gradients; the next block's input gradient comes as float32 sums
        dict(name="norm_backward_train", op="norm_backward", L=8192, d=2048, dt="bf16", y="f32",
             post=True, gate="column", dx="f32"),
        # gradients of a small odd float32 batch with a gate for each token
        dict(name="norm_backward_small", op="norm_backward", L=509, d=1000, dt="f32", y="f32",
             post=True, gate="token", dx="f32"),
        # one token through a 4-bit dense MLP's gate and up halves
        dict(name="mx_token", op="mx", L=1, K=1, E=0, active=0, zipf=0.0, n=5632, k=2048,
             dt="bf16", out="bf16", swiglu=True),
        # a prompt through a 4-bit dense projection
        dict(name="mx_prompt", op="mx", L=8192, K=1, E=0, active=0, zipf=0.0, n=5632, k=2048,
             dt="bf16", out="bf16", swiglu=False),
        # a decoding batch through 4-bit experts' gate and up halves
        dict(name="mx_experts", op="mx", L=256, K=8, E=64, active=64, zipf=0.5, n=704, k=2048,
             dt="bf16", out="bf16", swiglu=True),
        # an odd prompt through the experts' down halves, rows of five and a half 128s
        dict(name="mx_experts_prompt", op="mx", L=2039, K=6, E=32, active=29, zipf=0.9, n=1408,
             k=704, dt="bf16", out="bf16", swiglu=False),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, unit):
    return unit * _between(rng, max(1, lo // unit), hi // unit)


_MOST = 1.9e11  # operations of a drawn product, about those of the largest listed one


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "norm", "norm_backward", "mx", "mx"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        E = groups * _between(rng, 8 if groups == 1 else 4, 512 // groups)
        top = rng.randint(1, groups)
        K = min(_between(rng, 1, 32), top * E // groups)
        L = max(1, min(_between(rng, 1, 16384), 16384 * 256 // E, 16384 * 256 // (32 * K)))
        c = dict(op=op, L=L, E=E, K=K, fn=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5, 16.0]),
                 dt=rng.choice(["f32", "f32", "bf16"]))
        if op == "route":
            c.update(groups=groups, top=top, best=rng.choice([1, 2]), bias=rng.random() < 0.5,
                     scores=rng.random() < 0.3)
        else:
            c.update(dscore=rng.choice(["", "", "column", "full"]))
        return c
    if op in ("norm", "norm_backward"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        d = _width(rng, 64, 8192, 8 if dt == "bf16" else 4)
        y = rng.choice(["", "f32", "f32", dt])
        c = dict(op=op, d=d, dt=dt, y=y, post=bool(y) and rng.random() < 0.6,
                 gate=rng.choice(["", "column", "token", "full"]) if y else "")
        most = 8192 * 2048 * 2 // d // _SIZE[dt]
        if op == "norm_backward":
            c["dx"] = rng.choice(["f32", dt])
        c["L"] = max(1, min(_between(rng, 1, 16384), most))
        return c
    grouped = rng.random() < 0.5
    E = _between(rng, 2, 128) if grouped else 0
    K = rng.choice([k for k in (1, 2, 4, 6, 8) if k <= max(1, E)]) if grouped else 1
    L = _between(rng, 1, 8192)
    n, k = _width(rng, 64, 5632, 8), _width(rng, 64, 5632, 32)
    while max(1, E) * n * k > 1 << 27:
        n = max(64, n // 16 * 8)
    L = max(1, min(L, int(_MOST / (4 * K * n * k))))
    return dict(op=op, L=L, K=K, E=E, active=max(K, E - rng.randint(0, E // 4)) if E else 0,
                zipf=round(rng.uniform(0, 1.1), 2), n=n, k=k, dt=rng.choice(["bf16", "bf16", "f32"]),
                out=rng.choice(["bf16", "bf16", "f32"]), swiglu=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs


def _normal(shape, g, scale, dt):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    return (t * scale).to(dt)


def _routing(case, g):
    """Tasks of L tokens sorted by expert: the token of each, the experts' offsets."""
    L, K, E, A = case["L"], case["K"], case["E"], case["active"]
    order = torch.randperm(E, generator=g, device="cuda")[:A]
    logw = -case["zipf"] * torch.log(torch.arange(1, A + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((L, A), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    pick = (logw - torch.log(-torch.log(u))).topk(K, dim=1).indices
    eid = order[pick].reshape(-1)
    flat = torch.argsort(eid, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.bincount(eid, minlength=E).cumsum(0)
    return {"token": (flat // K).int(), "off": off.int(), "offsets": off.tolist()}


def _logits(case, g):
    """Logits of a trained router: experts of unlike popularity, spread per token."""
    z = _normal((case["L"], case["E"]), g, 1.2, torch.float32)
    z += _normal((1, case["E"]), g, 0.5, torch.float32)
    return z.to(_DT[case["dt"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op, L, dt = case["op"], case["L"], _DT[case["dt"]]
    f32, dev = torch.float32, "cuda"
    if op == "route":
        E, K = case["E"], case["K"]
        s["z"] = _logits(case, g)
        s["bias"] = _normal((E,), g, 0.05, f32) if case["bias"] else None
        s["idx"] = torch.empty((L, K), dtype=torch.int32, device=dev)
        s["gate"] = torch.empty((L, K), device=dev)
        s["score"] = torch.empty((L, E), device=dev) if case["scores"] else None
    elif op == "route_backward":
        E, K = case["E"], case["K"]
        s["z"] = _logits(case, g)
        s["idx"] = s["z"].float().topk(K, dim=1).indices.int()
        s["dgate"] = _normal((L, K), g, 0.1, f32)
        s["ds"] = {"": None, "column": (E,), "full": (L, E)}[case["dscore"]]
        if s["ds"] is not None:
            s["ds"] = _normal(s["ds"], g, 0.05, f32)
        s["dz"] = torch.empty_like(s["z"])
    elif op in ("norm", "norm_backward"):
        d = case["d"]
        r = _normal((L, d), g, 3.0, f32)
        r *= 1 + 20 * (torch.rand(d, generator=g, device=dev) < 0.005)  # outlying columns
        s["r"] = r.to(dt)
        s["w"] = (1 + _normal((d,), g, 0.2, f32)).to(dt)
        s["y"] = _normal((L, d), g, 0.5, _DT[case["y"]]) if case["y"] else None
        s["pw"] = (1 + _normal((d,), g, 0.2, f32)).to(dt) if case["post"] else None
        shape = {"": None, "column": (d,), "token": (L, 1), "full": (L, d)}[case["gate"]]
        s["g"] = None if shape is None else torch.rand(shape, generator=g, device=dev).to(dt)
        s["alpha"] = 0.7
        if op == "norm":
            s["r1"] = torch.empty_like(s["r"]) if case["y"] else None
            s["x"] = torch.empty_like(s["r"])
        else:
            s["dx"] = _normal((L, d), g, 0.1, _DT[case["dx"]])
            s["dr1"] = _normal((L, d), g, 0.1, dt)
            out = {"dr": torch.empty_like(s["r"]), "dweight": torch.empty(d, device=dev)}
            if s["y"] is not None:
                out["dy"] = torch.empty_like(s["y"])
            if s["pw"] is not None:
                out["dpost_weight"] = torch.empty(d, device=dev)
            if s["g"] is not None:
                out["dgate"] = torch.empty(shape, dtype=dt if case["gate"] == "full" else f32,
                                           device=dev)
            s["out"] = out
    else:
        E, n, k = case["E"], case["n"], case["k"]
        rows = (2 if case["swiglu"] else 1) * n
        x = _normal((L, k), g, 1.0, f32)
        x *= 1 + 15 * (torch.rand(k, generator=g, device=dev) < 0.01)
        s["x"] = x.to(dt)
        s["wq"], s["ws"] = _packed(_normal((max(1, E) * rows, k), g, 1 / math.sqrt(k), f32))
        groups = s["ws"].shape[1]
        if E:
            s["wq"], s["ws"] = s["wq"].view(E, rows, k // 2), s["ws"].view(E, rows, groups)
            s.update(_routing(case, g))
        s["q"] = torch.empty((L, k // 2), dtype=torch.uint8, device=dev)
        s["s"] = torch.empty((L, groups), dtype=torch.uint8, device=dev)
        s["out"] = torch.empty((L * case["K"], n), dtype=_DT[case["out"]], device=dev)
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from cartesian_routed_atomic_amd import binding as B

    case = s["case"]
    op = case["op"]
    if op == "route":
        idx, gate, score = B.expert_route(
            s["z"], case["K"], bias=s["bias"], scores=case["fn"], groups=case["groups"],
            top_groups=case["top"], group_best=case["best"], renormalize=case["renorm"],
            scale=case["scale"], expert_idx=s["idx"], gate=s["gate"], score=s["score"])
        return (idx, gate) if score is None else (idx, gate, score)
    if op == "route_backward":
        return B.expert_route_backward(s["z"], s["idx"], s["dgate"], scores=case["fn"],
                                       renormalize=case["renorm"], scale=case["scale"],
                                       dscore=s["ds"], dlogits=s["dz"])
    if op == "norm":
        r1, x = B.residual_norm(s["r"], y=s["y"], weight=s["w"], post_weight=s["pw"], gate=s["g"],
                                alpha=s["alpha"], r_out=s["r1"], x=s["x"])
        return x if s["y"] is None else (r1, x)
    if op == "norm_backward":
        return B.residual_norm_backward(s["r"], dx=s["dx"], dr_out=s["dr1"], y=s["y"],
                                        weight=s["w"], post_weight=s["pw"], gate=s["g"],
                                        alpha=s["alpha"], out=s["out"])
    q, sx = B.microscale_rows(s["x"], q=s["q"], scale=s["s"])
    if case["E"]:
        return B.microscaled_expert_matmul(q, sx, s["wq"], s["ws"], s["off"], x_row=s["token"],
                                           out=s["out"], swiglu=case["swiglu"])
    return B.microscaled_matmul(q, sx, s["wq"], s["ws"], out=s["out"], swiglu=case["swiglu"])


def _order(v):
    """Indices by (value descending, index ascending)."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices


def _plain_route(s, case):
    L, E, K, G = case["L"], case["E"], case["K"], case["groups"]
    # 64 bits: values next to a border decide which experts a token gets
    z = s["z"].double()
    if case["fn"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    biased = s["bias"] is not None
    value = score + s["bias"].double() if biased else z
    if G > 1:
        members = (value if biased or case["best"] == 1 else score).view(L, G, E // G)
        top = torch.sort(members, dim=2, descending=True).values[:, :, :case["best"]].sum(2)
        stay = _order(top)[:, :case["top"]]
        keep = torch.zeros((L, G), dtype=torch.bool, device=z.device)
        keep[torch.arange(L, device=z.device)[:, None], stay] = True
        out = ~keep.repeat_interleave(E // G, dim=1)
        value = torch.where(out, torch.full_like(value, -math.inf), value)
    idx = _order(value)[:, :K]
    w = score[torch.arange(L, device=z.device)[:, None], idx]
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    gate = (case["scale"] * w).float()
    return (idx.int(), gate, score.float()) if case["scores"] else (idx.int(), gate)


def _plain_route_backward(s, case):
    z, idx = s["z"].float(), s["idx"].long()
    if case["fn"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    up = case["scale"] * s["dgate"]
    if case["renorm"]:
        w = score.gather(1, idx)
        total = w.sum(1, keepdim=True)
        up = (up - (w * up).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(z) if s["ds"] is None else s["ds"].expand(z.shape).clone()
    ds = ds.scatter_add(1, idx, up)
    if case["fn"] == "softmax":
        dz = score * (ds - (score * ds).sum(1, keepdim=True))
    else:
        dz = score * (1 - score) * ds
    return dz.to(s["z"].dtype)


_EPS = 1e-6


def _rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)


def _plain_norm(s, case):
    r, w = s["r"].float(), s["w"].float()
    if s["y"] is not None:
        n = s["y"].float()
        if s["pw"] is not None:
            n = n * _rms(n) * s["pw"].float()
        if s["g"] is not None:
            n = n * s["g"].float()
        r = r + s["alpha"] * n
    x = (r * _rms(r) * w).to(s["r"].dtype)
    return x if s["y"] is None else (r.to(s["r"].dtype), x)


def _plain_norm_backward(s, case):
    d = case["d"]
    r, w, dx = s["r"].float(), s["w"].float(), s["dx"].float()
    a, p = _rms(r), dx * w
    dr = s["dr1"].float() + a * p - r * (a ** 3 * (p * r).sum(1, keepdim=True) / d)
    out = {"dr": dr.to(s["r"].dtype), "dweight": (dx * r * a).sum(0)}
    if s["y"] is None:
        return out
    y, e = s["y"].float(), s["alpha"] * dr
    n = y
    if s["pw"] is not None:
        b = _rms(y)
        n = y * b * s["pw"].float()
    if s["g"] is not None:
        dg = e * n
        out["dgate"] = {"column": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
                        "full": lambda: dg.to(s["g"].dtype)}[case["gate"]]()
        e = e * s["g"].float()
    if s["pw"] is not None:
        out["dpost_weight"] = (e * y * b).sum(0)
        q = e * s["pw"].float()
        e = b * q - y * (b ** 3 * (q * y).sum(1, keepdim=True) / d)
    out["dy"] = e.to(s["y"].dtype)
    return out


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _microscale(x):
    """Elements (signed values of 4 bits) and the blocks' power-of-two scales."""
    R, k = x.shape
    b = x.float().view(R, k // 32, 32)
    top = b.abs().amax(2, keepdim=True)
    power = torch.clamp(torch.frexp(top).exponent - 3, min=-127)  # floor(log2 top) - 2
    power = torch.where(top > 0, power, torch.full_like(power, -127))
    v = torch.ldexp(b.double(), -power)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    return torch.where(v < 0, -q, q).float(), power.squeeze(2)


def _packed(x):
    """Rows in the 4-bit form: two elements a byte, the earlier one low, and a
    byte 127 + log2(scale) for each block of 32, four blocks at a time."""
    q, power = _microscale(x)
    q = q.view(x.shape)
    table = torch.tensor(_VALUES, device=x.device)
    code = (torch.searchsorted(table, q.abs()) + 8 * (q < 0)).to(torch.uint8)
    blocks = power.shape[1]
    scale = torch.full((x.shape[0], (blocks + 3) // 4 * 4), 127, dtype=torch.uint8,
                       device=x.device)
    scale[:, :blocks] = (power + 127).to(torch.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, scale


def _unpacked(q, scale, k):
    """The float32 numbers that rows [.., k / 2] of bytes and their scales stand for."""
    table = torch.tensor([*_VALUES, *(-v for v in _VALUES)], device=q.device)
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], dim=-1)
    power = scale[..., :k // 32].int() - 127
    return torch.ldexp(v.view(*q.shape[:-1], k // 32, 32),
                       power.unsqueeze(-1)).view(*q.shape[:-1], k)


def _swiglu(z):
    g, u = z.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _plain_mx(s, case):
    k, out = case["k"], s["out"]
    q, power = _microscale(s["x"])
    x = torch.ldexp(q, power.unsqueeze(2)).view(s["x"].shape)
    if not case["E"]:
        z = x @ _unpacked(s["wq"], s["ws"], k).t()
        return (_swiglu(z) if case["swiglu"] else z).to(out.dtype)
    off = s["offsets"]
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        z = x[s["token"][lo:hi]] @ _unpacked(s["wq"][e], s["ws"][e], k).t()
        out[lo:hi] = (_swiglu(z) if case["swiglu"] else z).to(out.dtype)
    return out


def _run_plain(s):
    case = s["case"]
    return {"route": _plain_route, "route_backward": _plain_route_backward, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward, "mx": _plain_mx}[case["op"]](s, case)


# ------------------------------------------------------------------ definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "norm": _exact_norm,
            "norm_backward": _exact_norm_backward, "mx": _exact_mx}[case["op"]](s, case)


def _scores64(z, fn):
    z = z.to(torch.float64)
    return torch.softmax(z, 1) if fn == "softmax" else torch.sigmoid(z)


def _exact_route(s, case):
    L, E, G = case["L"], case["E"], case["groups"]
    z, score = s["z"].to(torch.float64), _scores64(s["z"], case["fn"])
    c = z if s["bias"] is None else score + s["bias"].to(torch.float64)
    place = torch.arange(E, device=z.device)
    left = torch.ones((L, E), dtype=torch.bool, device=z.device)
    if G > 1:
        m = (score if s["bias"] is None and case["best"] == 2 else c).unflatten(1, (G, E // G))
        first, at = m.max(2)
        value = first
        if case["best"] == 2:
            rest = m.scatter(2, at.unsqueeze(2), -math.inf)
            value = first + rest.amax(2)
        # a group stays if fewer than `top` groups come before it
        mine, other = value.unsqueeze(2), value.unsqueeze(1)
        g = torch.arange(G, device=z.device)
        ahead = (other > mine) | ((other == mine) & (g[None, :] < g[:, None]))
        left = (ahead.sum(2) < case["top"]).unsqueeze(2).expand(L, G, E // G).reshape(L, E)
    idx, w = [], []
    for _ in range(case["K"]):
        best = torch.where(left, c, -math.inf).amax(1, keepdim=True)
        hit = left & (c == best)
        i = torch.where(hit, place, E).amin(1, keepdim=True)
        left = left & (place != i)
        idx.append(i)
        w.append(score.gather(1, i))
    idx, w = torch.cat(idx, 1), torch.cat(w, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    res = (idx.to(torch.int32), w * case["scale"])
    return (*res, score) if case["scores"] else res


def _exact_route_backward(s, case):
    idx, f64 = s["idx"].long(), torch.float64
    score, rows = _scores64(s["z"], case["fn"]), torch.arange(case["L"], device="cuda")
    # d gate_j / d z_e, one gate at a time
    total = score.gather(1, idx).sum(1)
    ds = torch.zeros_like(score) if s["ds"] is None else s["ds"].to(f64) + torch.zeros_like(score)
    up = s["dgate"].to(f64) * case["scale"]
    for j in range(case["K"]):
        sj, ej = score[rows, idx[:, j]], idx[:, j]
        if not case["renorm"]:
            ds[rows, ej] += up[:, j]
            continue
        ds[rows, ej] += up[:, j] / total
        for i in range(case["K"]):
            ds[rows, idx[:, i]] -= up[:, j] * sj / total ** 2
    if case["fn"] == "sigmoid":
        return ds * torch.sigmoid(s["z"].to(f64)) * torch.sigmoid(-s["z"].to(f64))
    return score * ds - score * torch.linalg.vecdot(score, ds).unsqueeze(1)


def _exact_norm(s, case):
    f64, d = torch.float64, case["d"]
    r = s["r"].to(f64)
    if s["y"] is not None:
        add = s["y"].to(f64)
        if s["pw"] is not None:
            add = add / torch.sqrt(torch.linalg.vecdot(add, add) / d + _EPS).unsqueeze(1)
            add = add * s["pw"].to(f64)
        if s["g"] is not None:
            add = add * s["g"].to(f64)
        r = r + add * s["alpha"]
    x = r / torch.sqrt(torch.linalg.vecdot(r, r) / d + _EPS).unsqueeze(1) * s["w"].to(f64)
    return x if s["y"] is None else (r, x)


def _exact_norm_backward(s, case):
    f64, d = torch.float64, case["d"]

    def norm_back(v, weight, grad):
        """Gradients of v / sqrt(mean v^2 + eps) * weight."""
        size = torch.sqrt(torch.linalg.vecdot(v, v) / d + _EPS).unsqueeze(1)
        unit = v / size
        inner = grad * weight
        along = torch.linalg.vecdot(inner, unit).unsqueeze(1) / d
        return (inner - unit * along) / size, torch.linalg.vecdot(grad, unit, dim=0), unit

    r, w, dx = s["r"].to(f64), s["w"].to(f64), s["dx"].to(f64)
    back, dw, _ = norm_back(r, w, dx)
    dr = back + s["dr1"].to(f64)
    out = {"dr": dr, "dweight": dw}
    if s["y"] is None:
        return out
    y = s["y"].to(f64)
    g = torch.ones((1, 1), dtype=f64, device="cuda") if s["g"] is None else s["g"].to(f64)
    up = dr * g * s["alpha"]
    if s["pw"] is None:
        n, out["dy"] = y, up
    else:
        out["dy"], out["dpost_weight"], unit = norm_back(y, s["pw"].to(f64), up)
        n = unit * s["pw"].to(f64)
    if s["g"] is not None:
        dg = dr * n * s["alpha"]
        out["dgate"] = {"column": dg.sum(0), "token": dg.sum(1, keepdim=True),
                        "full": dg}[case["gate"]]
    # the order that the calls give their results in
    return {k: out[k] for k in ("dr", "dweight", "dgate", "dpost_weight", "dy") if k in out}


def _exact_mx(s, case):
    f64, k, E = torch.float64, case["k"], case["E"]
    b = s["x"].to(f64).unflatten(1, (k // 32, 32))
    top = b.abs().amax(2)
    power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # log2 may round across a whole number: the power is the largest not above top
    power = torch.where(torch.exp2(power) > top, power - 1, power)
    power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)
    unit = torch.exp2(torch.where(top > 0, power - 2, -127.0).clamp(min=-127.0)).unsqueeze(2)
    a, q = (b / unit).abs(), torch.zeros_like(b)
    # borders between neighbours; on a border the neighbour of even code wins
    for border, above, even in ((0.25, 0.5, 0), (0.75, 1.0, 1), (1.25, 1.5, 0), (1.75, 2.0, 1),
                                (2.5, 3.0, 0), (3.5, 4.0, 1), (5.0, 6.0, 0)):
        q = torch.where(a >= border if even else a > border, above, q)
    x = (torch.sign(b) * q * unit).flatten(1)

    def weights(q, scale):
        lo, hi = (q % 16).to(f64), torch.div(q, 16, rounding_mode="floor").to(f64)
        code = torch.stack([lo, hi], -1).flatten(-2)
        sign = 1 - 2 * (code >= 8).to(f64)
        code = code % 8
        e, m = torch.floor(code / 2), code % 2
        v = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
        unit = torch.exp2(scale[..., :k // 32].to(f64) - 127)
        return v * unit.repeat_interleave(32, dim=-1)

    def product(rows, w):
        z = torch.mm(rows, w.t().contiguous())
        if not case["swiglu"]:
            return z
        half = z.shape[1] // 2
        return z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]

    if not E:
        return product(x, weights(s["wq"], s["ws"]))
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    ends = s["off"].to(torch.int64)
    expert = torch.searchsorted(ends[1:], torch.arange(out.shape[0], device="cuda"), right=True)
    for e in range(E):
        m = torch.nonzero(expert == e).squeeze(1)
        if m.numel():
            rows = x.index_select(0, s["token"][m].long())
            out.index_copy_(0, m, product(rows, weights(s["wq"][e], s["ws"][e])))
    return out


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, L, sz = case["op"], case["L"], _SIZE[case["dt"]]
    if op == "route":
        E, K = case["E"], case["K"]
        return {"bytes": L * E * sz + 8 * L * K + (4 * L * E if case["scores"] else 0)
                + (4 * E if case["bias"] else 0), "flops": L * (10 * E + 8 * K)}
    if op == "route_backward":
        E, K = case["E"], case["K"]
        # the renormalised gates alone need only the selected logits
        dense = case["dscore"] or (case["fn"] == "softmax" and not case["renorm"])
        up = {"": 0, "column": 4 * E, "full": 4 * L * E}[case["dscore"]]
        return {"bytes": L * (E if dense else K) * sz + L * E * sz + 8 * L * K + up,
                "flops": L * (10 * E + 8 * K)}
    if op in ("norm", "norm_backward"):
        d, ysz = case["d"], _SIZE[case["y"]] if case["y"] else 0
        g = {"": 0, "column": d, "token": L, "full": L * d}[case["gate"]]
        small = d * sz * (2 if case["post"] else 1) + g * sz
        if op == "norm":
            return {"bytes": L * d * (2 * sz + (sz + ysz if ysz else 0)) + small,
                    "flops": L * d * (10 if case["post"] else 6)}
        grads = 4 * d * (2 if case["post"] else 1) + g * (sz if case["gate"] == "full" else 4)
        return {"bytes": L * d * (3 * sz + _SIZE[case["dx"]] + 2 * ysz) + small + grads,
                "flops": L * d * (22 if case["post"] else 12)}
    K, E, n, k = case["K"], case["E"], case["n"], case["k"]
    M, rows = L * K, (2 if case["swiglu"] else 1) * n
    used, packed = min(case["active"], M) if E else 1, k // 2 + k // 32
    return {"bytes": used * rows * packed + L * k * sz + M * n * _SIZE[case["out"]]
            + (4 * (M + E + 1) if E else 0), "flops": 2 * M * rows * k}
