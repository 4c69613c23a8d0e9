"""CPU oracle for what stands around the experts that are matrices: routing, the
norms before and after the block, and 4-bit microscaled rows.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or
execute this module.  It shares no code with the GPU library: float64 numpy, a
token or a block at a time.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.omni_oracle import widen

# ------------------------------------------------------------------ routing


def scores(z, fn):
    """Scores [L, E] in float64.  softmax: a row with a NaN or +infinity is NaN, a
    row of -infinity alone 0; sigmoid: one by one."""
    z = widen(z).astype(np.float64)
    s = np.zeros_like(z)
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(z.shape[0]):
            if fn == "sigmoid":
                s[t] = 1.0 / (1.0 + np.exp(-z[t]))
                continue
            top = z[t].max()
            if np.isnan(top) or top == np.inf:
                s[t] = np.nan
            elif top > -np.inf:
                e = np.exp(z[t] - top)
                s[t] = e / e.sum()
    return s


def _rank(values, count, allowed):
    """The `count` best of the allowed indices by (value desc, index asc)."""
    key = [(-v if v == v else math.inf, i) for i, v in enumerate(values) if allowed[i]]
    return [i for _, i in sorted(key)[:count]]


def _shared(z, fn):
    """Scores of some logits over their sum, formed without losing small ones."""
    if fn == "softmax":
        a = np.array(z, dtype=np.float64)
    else:  # log of the sigmoid
        a = np.array([min(v, 0.0) - math.log1p(math.exp(-abs(v))) if v == v else v for v in z])
    if np.isnan(a).any():
        return np.full(len(z), np.nan)
    top = a.max() if len(z) else -math.inf
    if top == -math.inf:
        return np.zeros(len(z))
    e = np.exp(a - top)
    return e / e.sum()


def expert_route(z, K, bias=None, fn="softmax", groups=1, top_groups=None, group_best=2,
                 renormalize=True, scale=1.0):
    """(expert_idx [L, K], gate [L, K] float64, scores [L, E] float64)."""
    z = widen(z).astype(np.float64)
    L, E = z.shape
    top = groups if top_groups is None else top_groups
    size = E // groups
    s = scores(z, fn)
    idx, gate = np.zeros((L, K), dtype=np.int64), np.zeros((L, K))
    for t in range(L):
        c = z[t] if bias is None else s[t] + np.asarray(bias, np.float64)
        allowed = np.ones(E, dtype=bool)
        if top < groups:
            m = s[t] if bias is None and group_best == 2 else c
            m = np.where(np.isnan(m), -np.inf, m)
            value = [sum(sorted(m[g * size:(g + 1) * size], reverse=True)[:group_best])
                     for g in range(groups)]
            for g in set(range(groups)) - set(_rank(value, top, [True] * groups)):
                allowed[g * size:(g + 1) * size] = False
        idx[t] = _rank(c, K, allowed)
        if renormalize:
            w = _shared(z[t, idx[t]], fn)
            if fn == "softmax" and np.isnan(s[t]).any():
                w[:] = np.nan
        else:
            w = s[t, idx[t]]
        gate[t] = scale * w
    return idx, gate, s


def expert_route_backward(z, idx, dgate, fn="softmax", renormalize=True, scale=1.0, dscore=None):
    """(dlogits [L, E] float64, mass): mass is the sum of the absolute values of what
    each entry is formed of."""
    z = widen(z).astype(np.float64)
    L, E = z.shape
    s = scores(z, fn)
    dz, mass = np.zeros((L, E)), np.zeros((L, E))
    for t in range(L):
        ks = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E]
        ids = [int(idx[t, k]) for k in ks]
        a = [scale * float(dgate[t, k]) for k in ks]
        u = np.zeros(E)
        size = np.zeros(E)
        if dscore is not None:
            u += np.asarray(dscore, np.float64)[t if np.ndim(dscore) == 2 else slice(None)]
            size += np.abs(u)
        if renormalize:
            w = _shared(z[t, ids], fn) if ids else []
            m = sum(wk * ak for wk, ak in zip(w, a))
            for e, wk, ak in zip(ids, w, a):
                f = 1.0 if fn == "softmax" else 1.0 / (1.0 + math.exp(min(z[t, e], 700.0)))
                dz[t, e] += wk * f * (ak - m)
                mass[t, e] += wk * f * (abs(ak) + sum(x * abs(y) for x, y in zip(w, a)))
        else:
            for e, ak in zip(ids, a):
                u[e] += ak
                size[e] += abs(ak)
        if dscore is None and renormalize:
            continue
        if fn == "softmax":
            dz[t] += s[t] * (u - np.dot(s[t], u))
            mass[t] += s[t] * (size + np.dot(s[t], size))
        else:
            with np.errstate(over="ignore"):
                f = s[t] / (1.0 + np.exp(z[t]))
            dz[t] += f * u
            mass[t] += f * size
    return dz, mass


# ------------------------------------------------------------------ norms


def _inv_rms(v, eps):
    with np.errstate(divide="ignore"):
        return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _wide(a):
    return None if a is None else widen(a).astype(np.float64)


def residual_norm(r, y=None, w=None, post_w=None, post=False, gate=None, alpha=1.0, eps=1e-6):
    """(r_out, x, mass of r_out) in float64; gate broadcasts against [L, d]."""
    r, y, w, post_w, gate = (_wide(a) for a in (r, y, w, post_w, gate))
    mass = np.abs(r)
    if y is not None:
        n = y
        if post or post_w is not None:
            n = y * _inv_rms(y, eps) * (1.0 if post_w is None else post_w)
        n = alpha * n * (1.0 if gate is None else gate)
        mass = mass + np.abs(n)
        r = r + n
    with np.errstate(invalid="ignore"):
        return r, r * _inv_rms(r, eps) * (1.0 if w is None else w), mass


def residual_norm_backward(r1, dx=None, dr_out=None, y=None, w=None, post_w=None, post=False,
                           gate=None, alpha=1.0, eps=1e-6):
    """dict name -> (gradient in float64, mass); mass as in expert_route_backward."""
    post = post or post_w is not None
    r1, dx, dr_out, y, w, post_w, gate = (_wide(a) for a in (r1, dx, dr_out, y, w, post_w, gate))
    dr, size = np.zeros_like(r1), np.zeros_like(r1)
    res = {}
    if dr_out is not None:
        dr, size = dr + dr_out, size + np.abs(dr_out)
    if dx is not None:
        a = _inv_rms(r1, eps)
        p = dx * (1.0 if w is None else w)
        dr = dr + a * p - r1 * a ** 3 * (p * r1).mean(axis=1, keepdims=True)
        size = size + a * np.abs(p) + np.abs(r1) * a ** 3 * np.abs(p * r1).mean(axis=1,
                                                                               keepdims=True)
        res["dweight"] = ((dx * r1 * a).sum(axis=0), np.abs(dx * r1 * a).sum(axis=0))
    res["dr"] = (dr, size)
    if y is None:
        return res
    g = np.ones((1, 1)) if gate is None else gate
    b = _inv_rms(y, eps) if post else np.ones((y.shape[0], 1))
    pw = 1.0 if post_w is None else post_w
    n = y * b * pw
    dn, dn_size = alpha * g * dr, abs(alpha) * np.abs(g) * size
    dg, dg_size = alpha * dr * n, abs(alpha) * size * np.abs(n)
    if gate is not None:
        axis = {(True, False): 0, (False, True): 1}.get((gate.ndim == 1, gate.ndim == 2 and
                                                         gate.shape[1] == 1 and y.shape[1] > 1))
        res["dgate"] = (dg, dg_size) if axis is None else \
            (dg.sum(axis=axis, keepdims=axis == 1), dg_size.sum(axis=axis, keepdims=axis == 1))
    if not post:
        res["dy"] = (dn, dn_size)
        return res
    res["dpost_weight"] = ((dn * y * b).sum(axis=0), (dn_size * np.abs(y) * b).sum(axis=0))
    q, q_size = dn * pw, dn_size * np.abs(pw)
    res["dy"] = (b * q - y * b ** 3 * (q * y).mean(axis=1, keepdims=True),
                 b * q_size + np.abs(y) * b ** 3 * (q_size * np.abs(y)).mean(axis=1, keepdims=True))
    return res


# ------------------------------------------------------------------ 4-bit rows

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def microscale_rows(x):
    """(codes [R, k] 0..15, scale bytes [R, blocks]) of rows x, block by block."""
    x = np.asarray(widen(x), dtype=np.float32)
    R, k = x.shape
    code = np.zeros((R, k), dtype=np.uint8)
    byte = np.zeros((R, k // 32), dtype=np.uint8)
    for r in range(R):
        for b in range(k // 32):
            v = x[r, 32 * b:32 * b + 32].astype(np.float64)
            top = np.abs(v).max()
            if not np.isfinite(top):
                byte[r, b] = 255
                continue
            power = -127 if top == 0 else max(math.frexp(top)[1] - 3, -127)
            byte[r, b] = power + 127
            a = np.abs(v) / 2.0 ** power
            # the nearest value; between two the one of even code
            dist = np.abs(a[:, None] - E2M1[None, :])
            near = dist == dist.min(axis=1, keepdims=True)
            for i in range(32):
                c = np.nonzero(near[i])[0]
                pick = c[0] if len(c) == 1 or c[0] % 2 == 0 else c[1]
                code[r, 32 * b + i] = pick | (8 if np.signbit(v[i]) else 0)
    return code, byte


def pack_rows(code, byte):
    """(q [R, k / 2], scale [R, 4 ceil(k / 128)]) as the library lays them out."""
    q = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    scale = np.full((byte.shape[0], (byte.shape[1] + 3) // 4 * 4), 127, dtype=np.uint8)
    scale[:, :byte.shape[1]] = byte
    return q, scale


def unpack_rows(q, scale):
    """float64 values of packed rows [.., k / 2]; blocks of scale 255 are NaN."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], 2 * q.shape[-1])
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = scale[..., :v.shape[-1] // 32].astype(np.float64)
    s = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return v * np.repeat(s, 32, axis=-1)
