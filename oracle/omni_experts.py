"""CPU oracle for the experts that are matrices and for the 8-bit products.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or
execute this module.  It shares no code with the GPU library: plain loops
over tasks' experts in float64 (numpy), no tiles, no masks.

Tasks m = 0 .. M-1 belong to expert e for off[e] <= m < off[e+1]; a task
reads row x_row[m] of x and writes row out_row[m] (row m where there is no
list).  An x row out of range counts as zeros, an output row out of range is
dropped, output rows of no task keep what they held.
"""
from __future__ import annotations

import numpy as np

from oracle.omni_oracle import silu, widen


def _segments(off, M):
    """(expert, first, end) of every expert with tasks, offsets clamped."""
    for e in range(len(off) - 1):
        lo = min(max(int(off[e]), 0), M)
        hi = min(max(int(off[e + 1]), lo), M)
        if hi > lo:
            yield e, lo, hi


def _rows(a, rows, lo, hi):
    """Rows a[rows[lo:hi]] in float64, zeros for rows out of range."""
    idx = np.arange(lo, hi) if rows is None else np.asarray(rows[lo:hi], dtype=np.int64)
    ok = (idx >= 0) & (idx < a.shape[0])
    out = np.zeros((hi - lo, a.shape[1]))
    out[ok] = a[idx[ok]]
    return out, ok


def expert_matmul_f64(x, w, off, M, out, x_row=None, out_row=None, transpose=False,
                      swiglu=False, x_scale=None, w_scale=None):
    """Writes the product into out (float64, a copy is returned) and returns
    (out, mass): mass[m, j] = sum_c |x||w| of every written entry (the scale
    of the rounding of its sum; for swiglu a bound of both halves' effect)."""
    x, w = widen(x), widen(w)
    out = np.array(out, dtype=np.float64)
    mass = np.zeros_like(out)
    for e, lo, hi in _segments(off, M):
        a, _ = _rows(x, x_row, lo, hi)
        b = w[e] if transpose else w[e].T
        z, s = a @ b, np.abs(a) @ np.abs(b)
        if w_scale is not None:
            rs, _ = _rows(np.asarray(x_scale, np.float64)[:, None], x_row, lo, hi)
            sc = rs * np.asarray(w_scale[e], np.float64)[None, :]
            z, s = z * sc, np.abs(z * sc)
        if swiglu:
            n = z.shape[1] // 2
            g, u = z[:, :n], z[:, n:]
            # |silu'| <= 1.1, |silu(g)| <= |g|
            s = 1.1 * s[:, :n] * np.abs(u) + np.abs(silu(g)) * s[:, n:]
            z = silu(g) * u
        dst = np.arange(lo, hi) if out_row is None else np.asarray(out_row[lo:hi], np.int64)
        keep = (dst >= 0) & (dst < out.shape[0])
        out[dst[keep]] = z[keep]
        mass[dst[keep]] = s[keep]
    return out, mass


def expert_weight_grad_f64(x, dy, off, M, x_row=None, dy_row=None):
    """(dw [E, n, k], mass) with mass = sum |dy||x| of every entry."""
    x, dy = widen(x), widen(dy)
    E = len(off) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mass = np.zeros_like(dw)
    for e, lo, hi in _segments(off, M):
        a, ok_a = _rows(dy, dy_row, lo, hi)
        b, ok_b = _rows(x, x_row, lo, hi)
        ok = (ok_a & ok_b)[:, None]
        a, b = np.where(ok, a, 0.0), np.where(ok, b, 0.0)
        dw[e] = a.T @ b
        mass[e] = np.abs(a).T @ np.abs(b)
    return dw, mass


def expert_combine_f64(o, K, gate=None, base=None):
    """(y [L, n], mass): y[t] (+)= sum_k gate[t, k] o[t K + k]."""
    o = widen(o)
    L = o.shape[0] // K
    y = np.zeros((L, o.shape[1])) if base is None else np.array(base, dtype=np.float64)
    mass = np.abs(y)
    for t in range(L):
        for k in range(K):
            g = 1.0 if gate is None else float(gate[t, k])
            y[t] += g * o[t * K + k]
            mass[t] += abs(g) * np.abs(o[t * K + k])
    return y, mass


def expert_combine_backward_f64(o, gate, dy):
    """(do [L*K, n], dgate [L, K], mass of dgate)."""
    o, dy = widen(o), np.asarray(dy, np.float64)
    L, K = gate.shape
    do = np.zeros((L * K, dy.shape[1]))
    dg, mass = np.zeros((L, K)), np.zeros((L, K))
    for t in range(L):
        for k in range(K):
            do[t * K + k] = float(gate[t, k]) * dy[t]
            dg[t, k] = np.dot(dy[t], o[t * K + k])
            mass[t, k] = np.dot(np.abs(dy[t]), np.abs(o[t * K + k]))
    return do, dg, mass


def quantize_rows(x):
    """(q int8, scale float32): scale = max|row| / 127 rounded to float32, q the
    integer nearest to the exact quotient, ties to even, decided with whole
    numbers: both operands are float32, so 2^k multiples of integers.  A row with
    a NaN or an infinity has that as its scale and q 0."""
    x = np.asarray(widen(x), dtype=np.float32)
    scale = (np.abs(x).max(axis=1).astype(np.float64) / 127.0).astype(np.float32)
    q = np.zeros(x.shape, dtype=np.int8)
    for r in range(x.shape[0]):
        s = float(scale[r])
        if s == 0.0 or not np.isfinite(s):
            continue
        for c in range(x.shape[1]):
            xn, xd = float(x[r, c]).as_integer_ratio()
            sn, sd = s.as_integer_ratio()
            num, den = abs(xn) * sd, xd * sn          # |x| / s = num / den
            v, rest = divmod(num, den)
            if 2 * rest > den or (2 * rest == den and v % 2 == 1):
                v += 1
            q[r, c] = int(np.sign(xn)) * min(v, 127)
    return q, scale
