"""Thin Python binding of libomni.so (ctypes).

Argument marshalling only: every step of the layer runs in the library's
HIP kernels.  PyTorch supplies device memory and the current stream.  If the
library is missing the import fails; there is no other execution path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("OMNI_LIB", os.path.join(_HERE, "libomni.so"))

OMNI_OK, OMNI_ERR_INVALID_ARG, OMNI_ERR_WORKSPACE, OMNI_ERR_UNSUPPORTED, OMNI_ERR_HIP = range(5)
OMNI_F32, OMNI_BF16 = 0, 1
EXEC_MODES = {"auto": 0, "expert": 1, "token": 2, "grouped": 3}  # omni_exec_mode
GROUPINGS = {"active": 0, "window": 1}             # omni_grouping
ABI_VERSION = 14

# Every symbol the header declares (checked by the CPU test suite).
EXPORTS = (
    "omni_abi_version", "omni_status_string", "omni_router_logits_workspace",
    "omni_router_logits",
    "omni_product_topk_workspace", "omni_product_topk", "omni_schedule_max_groups",
    "omni_schedule_workspace", "omni_schedule_tasks", "omni_atomic_forward_mode",
    "omni_atomic_forward_workspace", "omni_atomic_forward", "omni_routed_backward_workspace",
    "omni_routed_backward", "omni_shared_mlp_workspace", "omni_shared_mlp",
    "omni_atomic_forward_glu", "omni_flat_router_workspace", "omni_flat_router_topk",
    "omni_product_topk_static",
    "omni_expert_matmul", "omni_expert_weight_grad_workspace", "omni_expert_weight_grad",
    "omni_expert_combine",
    "omni_expert_combine_backward", "omni_quantize_rows", "omni_quantized_matmul",
    "omni_quantized_expert_matmul",
)


class OmniError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed: {msg} (status {code})")
        self.code = code


class ScheduleStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("counts", "active", "group_offsets", "task_token", "task_expert",
                 "task_gate", "task_index", "flat_expert", "flat_gate")]


_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "omni_abi_version": (_i, []),
    "omni_status_string": (ctypes.c_char_p, [_i]),
    "omni_router_logits_workspace": (_sz, [_i, _i, _i, _i, _i]),
    "omni_router_logits": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                _vp]),
    "omni_product_topk_workspace": (_sz, [_i, _i, _i, _i, _i]),
    "omni_product_topk": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _vp, _sz, _vp]),
    "omni_product_topk_static": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp]),
    "omni_schedule_max_groups": (_i, [_i, _i, _i, _i, _i]),
    "omni_schedule_workspace": (_sz, [_i, _i, _i, _i, _i]),
    "omni_schedule_tasks": (_i, [_i, _i, _i, _i, _i, _vp, _vp, ctypes.POINTER(ScheduleStruct),
                                 _vp, _sz, _vp]),
    "omni_atomic_forward_mode": (_i, [_i, _i, _i, _i, _i, _i]),
    "omni_atomic_forward_workspace": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "omni_atomic_forward": (_i, [_i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                                 ctypes.POINTER(ScheduleStruct), _vp, _i, _i, _vp, _sz, _vp]),
    "omni_routed_backward_workspace": (_sz, [_i, _i, _i, _i, _i, _i]),
    "omni_routed_backward": (_i, [_i, _i, _i, _i, _i, _i] + [_vp] * 19 + [_sz, _vp]),
    "omni_shared_mlp_workspace": (_sz, [_i, _i, _i, _i]),
    "omni_flat_router_workspace": (_sz, [_i, _i, _i]),
    "omni_flat_router_topk": (_i, [_i, _i, _i, _i, _i] + [_vp] * 8 + [_sz, _vp]),
    "omni_atomic_forward_glu": (_i, [_i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(ScheduleStruct), _vp, _i, _vp, _sz, _vp]),
    "omni_expert_matmul": (_i, [_i] * 7 + [_vp] * 4 + [_i, _i] + [_vp] * 3),
    "omni_expert_weight_grad_workspace": (_sz, [_i] * 5),
    "omni_expert_weight_grad": (_i, [_i] * 7 + [_vp] * 7 + [_sz, _vp]),
    "omni_expert_combine": (_i, [_i] * 4 + [_vp] * 3 + [_i, _vp]),
    "omni_expert_combine_backward": (_i, [_i] * 4 + [_vp] * 6),
    "omni_quantize_rows": (_i, [_i] * 3 + [_vp] * 4),
    "omni_quantized_matmul": (_i, [_i] * 4 + [_vp] * 4 + [_i, _vp, _vp]),
    "omni_quantized_expert_matmul": (_i, [_i] * 7 + [_vp] * 6 + [_i] + [_vp] * 3),
    "omni_shared_mlp": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
}

_lib = None


def lib():
    """Load libomni.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} not found: build it with "
                              f"`python -m cartesian_routed_atomic_amd.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        if h.omni_abi_version() != ABI_VERSION:
            raise ImportError(f"{LIB_PATH} has ABI {h.omni_abi_version()}, this binding "
                              f"expects {ABI_VERSION}: rebuild the library")
        _lib = h
    return _lib


def _check(fn, code):
    if code != OMNI_OK:
        msg = lib().omni_status_string(code).decode()
        raise OmniError(fn, code, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return OMNI_BF16
    if t.dtype == torch.float32:
        return OMNI_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _req(t, name, dtype=None, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(given, nbytes, like, stream=None):
    """The caller's workspace if it holds nbytes, else a fresh one (None where none is
    needed); the kernels take its address, so it has to be memory of like's device."""
    if given is not None:
        dev = given.get_device()
        if dev < 0:
            raise ValueError("workspace must be a device tensor")
        if dev != like.get_device():
            raise ValueError(f"workspace is on {given.device}, not on {like.device}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if given.numel() * given.element_size() >= nbytes:
            return given
    return _empty((nbytes,), torch.uint8, like, stream) if nbytes else given


# ------------------------------------------------------------------ calls


def router_logits(x, wr_t, wc_t, row_bias=None, col_bias=None, row_logits=None,
                  col_logits=None, workspace=None, stream=None):
    """omni_router_logits: returns (row_logits [L,Nr], col_logits [L,Nc]) float32."""
    L, d = x.shape
    Nr, Nc = wr_t.shape[0], wc_t.shape[0]
    _req(x, "x")
    _req(wr_t, "wr_t", x.dtype, (Nr, d))
    _req(wc_t, "wc_t", x.dtype, (Nc, d))
    for b, n, nm in ((row_bias, Nr, "row_bias"), (col_bias, Nc, "col_bias")):
        if b is not None:
            _req(b, nm, torch.float32, (n,))
    if row_logits is None:
        row_logits = torch.empty((L, Nr), dtype=torch.float32, device=x.device)
    if col_logits is None:
        col_logits = torch.empty((L, Nc), dtype=torch.float32, device=x.device)
    _req(row_logits, "row_logits", torch.float32, (L, Nr))
    _req(col_logits, "col_logits", torch.float32, (L, Nc))
    nws = lib().omni_router_logits_workspace(_dtype_code(x), L, d, Nr, Nc)
    ws = _workspace(workspace, nws, x, stream)
    _check("omni_router_logits", lib().omni_router_logits(
        _dtype_code(x), L, d, Nr, Nc, _ptr(x), _ptr(wr_t), _ptr(wc_t), _ptr(row_bias),
        _ptr(col_bias), _ptr(row_logits), _ptr(col_logits), _ptr(ws) if nws else None, nws,
        _stream(stream)))
    return row_logits, col_logits


def product_topk(row_logits, col_logits, kprime, K, want_sel=True, want_logp=True, out=None,
                 stream=None):
    """omni_product_topk: returns dict expert_idx, score, gate, row_logp, col_logp,
    row_sel, col_sel (the last four None unless asked for)."""
    L, Nr = row_logits.shape
    Nc = col_logits.shape[1]
    _req(row_logits, "row_logits", torch.float32)
    _req(col_logits, "col_logits", torch.float32, (L, Nc))
    dev = row_logits.device
    o = dict(out or {})

    def get(name, shape, dtype):
        t = o.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        _req(t, name, dtype, shape)
        return t
    idx = get("expert_idx", (L, K), torch.int32)
    score = get("score", (L, K), torch.float32)
    gate = get("gate", (L, K), torch.float32)
    rlp = get("row_logp", (L, Nr), torch.float32) if want_logp else None
    clp = get("col_logp", (L, Nc), torch.float32) if want_logp else None
    rsel = get("row_sel", (L, kprime), torch.int32) if want_sel else None
    csel = get("col_sel", (L, kprime), torch.int32) if want_sel else None
    nws = lib().omni_product_topk_workspace(L, Nr, Nc, kprime, K)
    ws = _workspace(o.get("workspace"), nws, row_logits, stream)
    _check("omni_product_topk", lib().omni_product_topk(
        L, Nr, Nc, kprime, K, _ptr(row_logits), _ptr(col_logits), _ptr(idx), _ptr(score),
        _ptr(gate), _ptr(rlp), _ptr(clp), _ptr(rsel), _ptr(csel), _ptr(ws),
        nws if ws is not None else 0, _stream(stream)))
    return {"expert_idx": idx, "score": score, "gate": gate, "row_logp": rlp, "col_logp": clp,
            "row_sel": rsel, "col_sel": csel, "workspace": ws}


@dataclass
class Schedule:
    L: int
    K: int
    N: int
    B: int
    grouping: str
    counts: torch.Tensor
    active: torch.Tensor
    group_offsets: torch.Tensor
    task_token: torch.Tensor
    task_expert: torch.Tensor
    task_gate: torch.Tensor
    task_index: torch.Tensor | None
    workspace: torch.Tensor | None
    # the selection the tasks were built from, in flatten order (set by
    # schedule_tasks; the token-centric executor reads the token lists from
    # it; None makes that executor invert the sorted order instead)
    flat_expert: torch.Tensor | None = None
    flat_gate: torch.Tensor | None = None

    def struct(self):
        return ScheduleStruct(*(None if t is None else t.data_ptr() for t in (
            self.counts, self.active, self.group_offsets, self.task_token, self.task_expert,
            self.task_gate, self.task_index, self.flat_expert, self.flat_gate)))


def _grouping(grouping):
    if grouping not in GROUPINGS:
        raise ValueError(f"grouping must be one of {sorted(GROUPINGS)}, got {grouping!r}")
    return GROUPINGS[grouping]


def max_groups(L, K, N, B, grouping="active"):
    return lib().omni_schedule_max_groups(L, K, N, B, _grouping(grouping))


def alloc_schedule(L, K, N, B, device, with_index=True, grouping="active"):
    """Device buffers for a schedule of L*K tasks (and its workspace).
    grouping: "active" (B active experts per group) or "window" (id windows)."""
    M = L * K
    G = max_groups(L, K, N, B, grouping)
    nws = lib().omni_schedule_workspace(L, K, N, B, _grouping(grouping))
    i32 = dict(dtype=torch.int32, device=device)
    return Schedule(L, K, N, B, grouping,
                    counts=torch.zeros(2, **i32),
                    active=torch.empty(max(1, min(N, M)), **i32),
                    group_offsets=torch.empty(G + 1, **i32),
                    task_token=torch.empty(max(1, M), **i32),
                    task_expert=torch.empty(max(1, M), **i32),
                    task_gate=torch.empty(max(1, M), dtype=torch.float32, device=device),
                    task_index=torch.empty(max(1, M), **i32) if with_index else None,
                    workspace=torch.empty(max(1, nws), dtype=torch.uint8, device=device))


def schedule_tasks(expert_idx, gate, N, B, sched=None, stream=None, grouping="active"):
    """omni_schedule_tasks: returns a Schedule of device tensors."""
    L, K = expert_idx.shape
    _req(expert_idx, "expert_idx", torch.int32)
    _req(gate, "gate", torch.float32, (L, K))
    if sched is None:
        sched = alloc_schedule(L, K, N, B, expert_idx.device, grouping=grouping)
    elif sched.grouping != grouping:
        raise ValueError(f"schedule buffers were sized for grouping {sched.grouping!r}")
    st = sched.struct()
    ws = _workspace(sched.workspace, 0, expert_idx)
    _check("omni_schedule_tasks", lib().omni_schedule_tasks(
        L, K, N, B, _grouping(grouping), _ptr(expert_idx), _ptr(gate), ctypes.byref(st), _ptr(ws),
        ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))
    sched.flat_expert, sched.flat_gate = expert_idx, gate
    return sched


def _same_shape_schedule(sched, L, N):
    # the kernels index x, W, V with the schedule's token and expert ids
    if sched.L != L or sched.N != N:
        raise ValueError(f"the schedule was built for L={sched.L}, N={sched.N}; "
                         f"x and the expert matrices give L={L}, N={N}")
    if sched.task_index is None:
        raise ValueError("the schedule must carry task_index")


def _exec_mode(mode):
    if mode not in EXEC_MODES:
        raise ValueError(f"mode must be one of {sorted(EXEC_MODES)}, got {mode!r}")
    return EXEC_MODES[mode]


def atomic_forward_mode(dtype, L, d, N, K, B):
    """omni_atomic_forward_mode: the form mode="auto" runs ("expert" / "token" / "grouped")."""
    code = torch.bfloat16 if dtype == torch.bfloat16 else torch.float32
    m = lib().omni_atomic_forward_mode(OMNI_BF16 if code == torch.bfloat16 else OMNI_F32,
                                       L, d, N, K, B)
    if m == 0:
        raise ValueError("invalid shape for omni_atomic_forward_mode")
    return {1: "expert", 2: "token", 3: "grouped"}[m]


def atomic_forward(x, w, v, sched, y=None, accumulate=False, workspace=None, stream=None,
                   mode="auto"):
    """omni_atomic_forward: returns y [L, d] float32 (y += routed if accumulate).
    mode: "auto", "expert" (expert-centric), "token" (token-centric) or "grouped"
    (per token tile, the most shared experts as two MFMA products and the rest
    per task; bf16 only)."""
    L, d = x.shape
    N = w.shape[0]
    _req(x, "x")
    _req(w, "w", x.dtype, (N, d))
    _req(v, "v", x.dtype, (N, d))
    _same_shape_schedule(sched, L, N)
    code = _exec_mode(mode)
    if y is None:
        y = torch.empty((L, d), dtype=torch.float32, device=x.device)
    _req(y, "y", torch.float32, (L, d))
    st = sched.struct()
    nws = lib().omni_atomic_forward_workspace(_dtype_code(x), L, d, N, sched.K, sched.B, code)
    ws = _workspace(workspace, nws, x, stream)
    _check("omni_atomic_forward", lib().omni_atomic_forward(
        _dtype_code(x), L, d, N, sched.K, sched.B, _ptr(x), _ptr(w), _ptr(v),
        ctypes.byref(st), _ptr(y), int(bool(accumulate)), code, _ptr(ws),
        nws if ws is not None else 0, _stream(stream)))
    return y


def atomic_forward_glu(x, w, u, v, sched, y=None, accumulate=False, workspace=None,
                       stream=None):
    """omni_atomic_forward_glu (SwiGLU-gated experts): returns y [L, d] float32,
    y_t = sum_k g silu(x_t . W[e]) (x_t . U[e]) V[e] (y += that if accumulate)."""
    L, d = x.shape
    N = w.shape[0]
    _req(x, "x")
    for name, t in (("w", w), ("u", u), ("v", v)):
        _req(t, name, x.dtype, (N, d))
    _same_shape_schedule(sched, L, N)
    if y is None:
        y = torch.empty((L, d), dtype=torch.float32, device=x.device)
    _req(y, "y", torch.float32, (L, d))
    st = sched.struct()
    nws = lib().omni_atomic_forward_workspace(_dtype_code(x), L, d, N, sched.K, sched.B,
                                              EXEC_MODES["token"])
    ws = _workspace(workspace, nws, x, stream)
    _check("omni_atomic_forward_glu", lib().omni_atomic_forward_glu(
        _dtype_code(x), L, d, N, sched.K, sched.B, _ptr(x), _ptr(w), _ptr(u), _ptr(v),
        ctypes.byref(st), _ptr(y), int(bool(accumulate)), _ptr(ws),
        nws if ws is not None else 0, _stream(stream)))
    return y


def flat_router_topk(x, wf, K, bias=None, want_logp=False, out=None, workspace=None,
                     stream=None):
    """omni_flat_router_topk (the d x N router baseline): returns dict expert_idx,
    score, gate [L, K] and logp [L, N] (None unless want_logp), workspace."""
    L, d = x.shape
    N = wf.shape[0]
    _req(x, "x")
    _req(wf, "wf", x.dtype, (N, d))
    if bias is not None:
        _req(bias, "bias", torch.float32, (N,))
    o = dict(out or {})
    dev = x.device
    r = {"expert_idx": o.get("expert_idx"), "score": o.get("score"), "gate": o.get("gate")}
    for name, dt in (("expert_idx", torch.int32), ("score", torch.float32),
                     ("gate", torch.float32)):
        if r[name] is None:
            r[name] = torch.empty((L, K), dtype=dt, device=dev)
        _req(r[name], name, dt, (L, K))
    r["logp"] = torch.empty((L, N), dtype=torch.float32, device=dev) if want_logp else None
    code = _dtype_code(x)
    nws = lib().omni_flat_router_workspace(code, L, N)
    ws = _workspace(workspace, max(1, nws), x, stream)
    _check("omni_flat_router_topk", lib().omni_flat_router_topk(
        code, L, d, N, K, _ptr(x), _ptr(wf), _ptr(bias), _ptr(r["expert_idx"]),
        _ptr(r["score"]), _ptr(r["gate"]), _ptr(r["logp"]), _ptr(ws), nws, _stream(stream)))
    r["workspace"] = ws
    return r


def forward(x, wr_t, wc_t, w, v, kprime, K, B, row_bias=None, col_bias=None, stream=None,
            mode="auto"):
    """The four calls back to back on one stream; returns every intermediate."""
    zr, zc = router_logits(x, wr_t, wc_t, row_bias, col_bias, stream=stream)
    sel = product_topk(zr, zc, kprime, K, stream=stream)
    N = wr_t.shape[0] * wc_t.shape[0]
    sched = schedule_tasks(sel["expert_idx"], sel["gate"], N, B, stream=stream)
    y = atomic_forward(x, w, v, sched, stream=stream, mode=mode)
    return {"row_logits": zr, "col_logits": zc, **sel, "schedule": sched, "y": y}


def shared_mlp(x, w_gate, w_up, w_down, y=None, accumulate=False, workspace=None, stream=None):
    """omni_shared_mlp: y [L, d] float32 = (or +=, if accumulate) the shared dense
    MLP branch Wd (silu(Wg x) * (Wu x)); w_gate, w_up [d_ff, d], w_down [d, d_ff]."""
    L, d = x.shape
    d_ff = w_gate.shape[0]
    _req(x, "x")
    _req(w_gate, "w_gate", x.dtype, (d_ff, d))
    _req(w_up, "w_up", x.dtype, (d_ff, d))
    _req(w_down, "w_down", x.dtype, (d, d_ff))
    if y is None:
        y = torch.empty((L, d), dtype=torch.float32, device=x.device)
    _req(y, "y", torch.float32, (L, d))
    code = _dtype_code(x)
    nws = lib().omni_shared_mlp_workspace(code, L, d, d_ff)
    ws = _workspace(workspace, max(1, nws), x, stream)
    _check("omni_shared_mlp", lib().omni_shared_mlp(
        code, L, d, d_ff, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(y),
        int(bool(accumulate)), _ptr(ws), nws, _stream(stream)))
    return y


def layer_forward(x, wr_t, wc_t, w, v, w_gate, w_up, w_down, kprime, K, B, row_bias=None,
                  col_bias=None, stream=None, mode="auto"):
    """The whole OmniMoE layer on one stream: the shared dense MLP writes y, then
    the routed branch (router, product top-K, schedule) runs and its executor
    adds the routed output onto y.  Returns every intermediate of the routed
    branch and y."""
    y = shared_mlp(x, w_gate, w_up, w_down, stream=stream)
    zr, zc = router_logits(x, wr_t, wc_t, row_bias, col_bias, stream=stream)
    sel = product_topk(zr, zc, kprime, K, stream=stream)
    N = wr_t.shape[0] * wc_t.shape[0]
    sched = schedule_tasks(sel["expert_idx"], sel["gate"], N, B, stream=stream)
    atomic_forward(x, w, v, sched, y=y, accumulate=True, stream=stream, mode=mode)
    return {"row_logits": zr, "col_logits": zc, **sel, "schedule": sched, "y": y}


def routed_backward(x, wr_t, wc_t, w, v, expert_idx, gate, dy, out=None, workspace=None,
                    stream=None):
    """omni_routed_backward: gradients of the routed layer for upstream dy [L, d] float32.

    Returns dict dx [L, d], dwr [Nr, d], dwc [Nc, d], drb [Nr], dcb [Nc],
    counts [2], active [min(N, L*K)], dw, dv [min(N, L*K), d] (row r is the
    gradient of expert active[r], r < counts[0]), dgate [L, K]; all float32
    except counts / active (int32)."""
    L, d = x.shape
    Nr, Nc = wr_t.shape[0], wc_t.shape[0]
    N = Nr * Nc
    K = expert_idx.shape[1]
    _req(x, "x")
    for name, t in (("wr_t", wr_t), ("wc_t", wc_t)):
        _req(t, name, x.dtype)
    _req(w, "w", x.dtype, (N, d))
    _req(v, "v", x.dtype, (N, d))
    _req(expert_idx, "expert_idx", torch.int32, (L, K))
    _req(gate, "gate", torch.float32, (L, K))
    _req(dy, "dy", torch.float32, (L, d))
    dev = x.device
    o = dict(out or {})
    na = max(1, min(N, L * K))

    def get(name, shape, dtype):
        t = o.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        _req(t, name, dtype, shape)
        return t
    r = {"dx": get("dx", (L, d), torch.float32), "dwr": get("dwr", (Nr, d), torch.float32),
         "dwc": get("dwc", (Nc, d), torch.float32), "drb": get("drb", (Nr,), torch.float32),
         "dcb": get("dcb", (Nc,), torch.float32), "counts": get("counts", (2,), torch.int32),
         "active": get("active", (na,), torch.int32),
         "dw": get("dw", (na, d), torch.float32), "dv": get("dv", (na, d), torch.float32),
         "dgate": get("dgate", (L, K), torch.float32)}
    code = _dtype_code(x)
    nws = lib().omni_routed_backward_workspace(code, L, d, Nr, Nc, K)
    ws = _workspace(workspace, max(1, nws), x, stream)
    _check("omni_routed_backward", lib().omni_routed_backward(
        code, L, d, Nr, Nc, K, _ptr(x), _ptr(wr_t), _ptr(wc_t), _ptr(w), _ptr(v),
        _ptr(expert_idx), _ptr(gate), _ptr(dy), _ptr(r["dx"]), _ptr(r["dwr"]), _ptr(r["dwc"]),
        _ptr(r["drb"]), _ptr(r["dcb"]), _ptr(r["counts"]), _ptr(r["active"]), _ptr(r["dw"]),
        _ptr(r["dv"]), _ptr(r["dgate"]), _ptr(ws), nws, _stream(stream)))
    r["workspace"] = ws
    return r


# The calls below are short enough that the host's part counts: pointers go to
# ctypes as plain integers, tensors are checked in one pass (the reason is
# looked for only once something is wrong) and the current stream is read
# without building a stream object (torch.cuda.current_stream takes 2.8 us of
# a 13 us call).


def _tensors(dev, *specs):
    """Check (tensor, name, dtype, shape) of arguments on device index dev."""
    for t, name, dtype, shape in specs:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            continue
        _req(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")


def _device_of(t, name):
    """Device index of the argument that the others have to be with."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _call(fn, dev, stream, *args):
    """Call the library on device dev, on `stream` or that device's current one."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the tensors of cuda:{dev}")
    else:
        raw = stream.cuda_stream
    f = getattr(_lib or lib(), fn)
    if torch._C._cuda_getDevice() == dev:
        code = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = f(*args, raw)
    if code:
        _check(fn, code)


def _sizes_fit(bits):
    """bits: the sizes or-ed together.  The library's are 32-bit; ctypes cuts longer ones off."""
    if bits >> 31:
        raise ValueError("sizes of 2^31 or more are not taken")


def _empty(shape, dtype, like, stream):
    """A fresh tensor, of the memory pool of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape


def _experts(w, swiglu, name):
    """E, n, k of the experts' weights."""
    if w.dim() != 3 or (swiglu and w.shape[1] % 2):
        raise ValueError(f"{name} must be [E, n, k] ([E, 2n, k] with swiglu)")
    E, rows, k = w.shape
    return E, rows // 2 if swiglu else rows, k


def _tasks(dev, rows, x_row, other, other_name):
    """The number of tasks: the row lists' length, else the rows there are."""
    M = rows
    if other is not None:
        M = other.numel()
        _tensors(dev, (other, other_name, torch.int32, (M,)))
    if x_row is not None:
        if other is None:
            M = x_row.numel()
        _tensors(dev, (x_row, "x_row", torch.int32, (M,)))
    elif rows < M:
        raise ValueError(f"{other_name} lists {M} tasks, x has {rows} rows")
    return M


def expert_matmul(x, w, offsets, x_row=None, out=None, out_row=None, transpose=False,
                  swiglu=False, stream=None):
    """omni_expert_matmul: out [., n] = x[x_row] W[e]^T over tasks sorted by expert
    (w [E, n, k], offsets [E + 1] int32), or, with transpose, x[x_row] W[e]
    (the input gradient; x [., n], out [., k]).  swiglu: w [E, 2n, k], out [., n]
    = silu(gate half) * up half.  x_row / out_row: int32 row lists or None.
    A fresh out has a row per task (unwritten where no expert has the task)."""
    E, n, k = _experts(w, swiglu, "w")
    R, inner = _matrix(x, "x")
    dev, dt, width = _device_of(x, "x"), x.dtype, k if transpose else n
    M = _tasks(dev, R, x_row, out_row, "out_row")
    if out is None:
        out = _empty((M, width), dt, x, stream)
    Ro = out.shape[0]
    _tensors(dev, (x, "x", dt, (R, n if transpose else k)), (w, "w", dt, w.shape),
             (offsets, "offsets", torch.int32, (E + 1,)), (out, "out", dt, (Ro, width)))
    _sizes_fit(M | E | n | k | R | Ro)
    _call("omni_expert_matmul", dev, stream, _dtype_code(x), M, E, n, k, R, Ro, x.data_ptr(),
          _addr(x_row), w.data_ptr(), offsets.data_ptr(), 1 if transpose else 0,
          1 if swiglu else 0, out.data_ptr(), _addr(out_row))
    return out


def expert_weight_grad(x, dy, offsets, x_row=None, dy_row=None, dw=None, workspace=None,
                       stream=None):
    """omni_expert_weight_grad: dw [E, n, k] float32, dw[e] = sum over expert e's tasks
    of dy[dy_row]^T x[x_row] (x [., k], dy [., n]; zero for experts without tasks)."""
    (R, k), (Ry, n) = _matrix(x, "x"), _matrix(dy, "dy")
    E, dev, dt = offsets.numel() - 1, _device_of(x, "x"), x.dtype
    M = _tasks(dev, R, x_row, dy_row, "dy_row")
    if dy_row is None and Ry < M:
        raise ValueError(f"{M} tasks, dy has {Ry} rows")
    if dw is None:
        dw = _empty((E, n, k), torch.float32, x, stream)
    _tensors(dev, (x, "x", dt, (R, k)), (dy, "dy", dt, (Ry, n)),
             (offsets, "offsets", torch.int32, (E + 1,)), (dw, "dw", torch.float32, (E, n, k)))
    code = _dtype_code(x)
    _sizes_fit(M | E | n | k | R | Ry)
    nws = lib().omni_expert_weight_grad_workspace(code, M, E, n, k)
    ws = _workspace(workspace, nws, x, stream)
    _call("omni_expert_weight_grad", dev, stream, code, M, E, n, k, R, Ry, x.data_ptr(),
          _addr(x_row), dy.data_ptr(), _addr(dy_row), offsets.data_ptr(), dw.data_ptr(),
          _addr(ws) if nws else None, nws)
    return dw


def expert_combine(o, K, gate=None, y=None, accumulate=False, stream=None):
    """omni_expert_combine: y [L, n] float32 = (or +=) sum_k gate[t, k] o[t K + k]
    for o [L*K, n] in flatten order; gate [L, K] float32, None for ones."""
    rows, n = _matrix(o, "o")
    if K < 1 or rows % K:
        raise ValueError(f"o has {rows} rows, not a multiple of K={K}")
    L, dev = rows // K, _device_of(o, "o")
    if y is None:
        if accumulate:
            raise ValueError("accumulate needs y")
        y = _empty((L, n), torch.float32, o, stream)
    _tensors(dev, (o, "o", o.dtype, (rows, n)), (y, "y", torch.float32, (L, n)))
    if gate is not None:
        _tensors(dev, (gate, "gate", torch.float32, (L, K)))
    _sizes_fit(L | K | n)
    _call("omni_expert_combine", dev, stream, _dtype_code(o), L, K, n, o.data_ptr(), _addr(gate),
          y.data_ptr(), 1 if accumulate else 0)
    return y


def expert_combine_backward(o, gate, dy, do=None, dgate=None, want_dgate=True, stream=None):
    """omni_expert_combine_backward: returns (do [L*K, n] of o's type, dgate [L, K]
    float32) for dy [L, n] float32.  gate None: gates of one, K from the rows of o;
    want_dgate False: dgate is None and o's values are not read."""
    (rows, width), (L, n), dev = _matrix(o, "o"), _matrix(dy, "dy"), _device_of(o, "o")
    f32 = torch.float32
    if gate is not None:
        K = _matrix(gate, "gate")[1]
    else:
        K = rows // L if L else 1
        if K < 1 or rows != L * K:
            raise ValueError(f"o has {rows} rows, not a multiple of dy's {L}")
    if do is None:
        do = _empty((rows, width), o.dtype, o, stream)
    if not want_dgate:
        if dgate is not None:
            raise ValueError("dgate is not wanted but given")
    elif dgate is None:
        dgate = _empty((L, K), f32, o, stream)
    _tensors(dev, (o, "o", o.dtype, (L * K, n)), (dy, "dy", f32, (L, n)),
             (do, "do", o.dtype, (L * K, n)))
    if gate is not None:
        _tensors(dev, (gate, "gate", f32, (L, K)))
    if dgate is not None:
        _tensors(dev, (dgate, "dgate", f32, (L, K)))
    _sizes_fit(L | K | n)
    _call("omni_expert_combine_backward", dev, stream, _dtype_code(o), L, K, n, o.data_ptr(),
          _addr(gate), dy.data_ptr(), do.data_ptr(), _addr(dgate))
    return do, dgate


def quantize_rows(x, q=None, scale=None, stream=None):
    """omni_quantize_rows: (q [R, k] int8, scale [R] float32), scale = max|row| / 127,
    q = row / scale to the nearest integer.  Tokens' activations, or weights by
    output channel (view [E, n, k] experts as [E*n, k])."""
    (R, k), dev = _matrix(x, "x"), _device_of(x, "x")
    if q is None:
        q = _empty((R, k), torch.int8, x, stream)
    if scale is None:
        scale = _empty(R, torch.float32, x, stream)
    _tensors(dev, (x, "x", x.dtype, (R, k)), (q, "q", torch.int8, (R, k)),
             (scale, "scale", torch.float32, (R,)))
    _sizes_fit(R | k)
    _call("omni_quantize_rows", dev, stream, _dtype_code(x), R, k, x.data_ptr(), q.data_ptr(),
          scale.data_ptr())
    return q, scale


def quantized_matmul(xq, x_scale, wq, w_scale, out=None, out_dtype=torch.bfloat16, swiglu=False,
                     stream=None):
    """omni_quantized_matmul: out [M, n] = (xq wq^T) * x_scale[m] * w_scale[j] for int8
    xq [M, k], wq [n, k] (swiglu: [2n, k], out = silu(gate half) * up half)."""
    (M, k), rows, dev = _matrix(xq, "xq"), _matrix(wq, "wq")[0], _device_of(xq, "xq")
    if swiglu and rows % 2:
        raise ValueError("swiglu needs an even number of weight rows")
    n = rows // 2 if swiglu else rows
    if out is None:
        out = _empty((M, n), out_dtype, xq, stream)
    i8, f32 = torch.int8, torch.float32
    _tensors(dev, (xq, "xq", i8, (M, k)), (wq, "wq", i8, (rows, k)),
             (x_scale, "x_scale", f32, (M,)), (w_scale, "w_scale", f32, (rows,)),
             (out, "out", out.dtype, (M, n)))
    _sizes_fit(M | n | k)
    _call("omni_quantized_matmul", dev, stream, _dtype_code(out), M, n, k, xq.data_ptr(),
          x_scale.data_ptr(), wq.data_ptr(), w_scale.data_ptr(), 1 if swiglu else 0,
          out.data_ptr())
    return out


def quantized_expert_matmul(xq, x_scale, wq, w_scale, offsets, x_row=None, out=None,
                            out_row=None, out_dtype=torch.bfloat16, swiglu=False, stream=None):
    """omni_quantized_expert_matmul: expert_matmul over int8 rows xq [., k] with
    x_scale [.] and experts wq [E, n, k] with w_scale [E, n]."""
    E, n, k = _experts(wq, swiglu, "wq")
    R, dev = _matrix(xq, "xq")[0], _device_of(xq, "xq")
    M = _tasks(dev, R, x_row, out_row, "out_row")
    if out is None:
        out = _empty((M, n), out_dtype, xq, stream)
    i8, f32, Ro = torch.int8, torch.float32, out.shape[0]
    _tensors(dev, (xq, "xq", i8, (R, k)), (wq, "wq", i8, wq.shape),
             (x_scale, "x_scale", f32, (R,)), (w_scale, "w_scale", f32, wq.shape[:2]),
             (offsets, "offsets", torch.int32, (E + 1,)), (out, "out", out.dtype, (Ro, n)))
    _sizes_fit(M | E | n | k | R | Ro)
    _call("omni_quantized_expert_matmul", dev, stream, _dtype_code(out), M, E, n, k, R, Ro,
          xq.data_ptr(), x_scale.data_ptr(), _addr(x_row), wq.data_ptr(), w_scale.data_ptr(),
          offsets.data_ptr(), 1 if swiglu else 0, out.data_ptr(), _addr(out_row))
    return out
