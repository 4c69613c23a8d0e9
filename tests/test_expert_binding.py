"""What the Python calls hand to the library, without a GPU: device checks and
the library's calls are replaced, so host tensors get as far as the library."""
import pytest
import torch

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")


class Reached(Exception):
    """The library would have been called."""


@pytest.fixture
def host_calls(monkeypatch):
    """Calls of the library raise Reached(name, arguments); tensors count as device 0's,
    except for what _workspace looks at."""
    def reach(fn, dev, stream, *args):
        raise Reached(fn, args)

    def check(fn, code):
        raise Reached(fn, code)
    monkeypatch.setattr(B, "_call", reach)
    monkeypatch.setattr(B, "_check", check)
    monkeypatch.setattr(B, "_device_of", lambda t, name: 0)
    monkeypatch.setattr(B, "_tensors", lambda dev, *specs: None)
    monkeypatch.setattr(B, "_req", lambda *a, **k: None)
    monkeypatch.setattr(B, "_stream", lambda stream=None: None)
    real = B.lib()

    class NoKernels:
        """Workspace sizes are the library's, everything else does nothing."""

        def __getattr__(self, name):
            f = getattr(real, name)
            return f if name.endswith(("_workspace", "_mode")) else lambda *a: 0
    monkeypatch.setattr(B, "lib", lambda: NoKernels())
    return B


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def sched(L, K, N):
    return B.Schedule(L, K, N, 16, "active", *(i32(1) for _ in range(7)), None)


# every call that takes a workspace, at a size that needs one
CALLS = {
    "router_logits": lambda ws: B.router_logits(bf(256, 2048), bf(1024, 2048), bf(1024, 2048),
                                                workspace=ws),
    "product_topk": lambda ws: B.product_topk(torch.zeros(8, 64), torch.zeros(8, 64), 8, 8,
                                              out={"workspace": ws}),
    "atomic_forward": lambda ws: B.atomic_forward(bf(8, 128), bf(64, 128), bf(64, 128),
                                                  sched(8, 4, 64), workspace=ws),
    "atomic_forward_glu": lambda ws: B.atomic_forward_glu(
        bf(8, 128), bf(64, 128), bf(64, 128), bf(64, 128), sched(8, 4, 64), workspace=ws),
    "flat_router_topk": lambda ws: B.flat_router_topk(bf(8, 128), bf(64, 128), 4, workspace=ws),
    "shared_mlp": lambda ws: B.shared_mlp(bf(8, 128), bf(64, 128), bf(64, 128), bf(128, 64),
                                          workspace=ws),
    "routed_backward": lambda ws: B.routed_backward(
        bf(8, 128), bf(8, 128), bf(8, 128), bf(64, 128), bf(64, 128), i32(8, 4),
        torch.zeros(8, 4), torch.zeros(8, 128), workspace=ws),
    "expert_weight_grad": lambda ws: B.expert_weight_grad(bf(8192, 64), bf(8192, 64), i32(2),
                                                          workspace=ws),
}
ENOUGH = 1 << 26


@pytest.mark.parametrize("name", list(CALLS))
def test_workspace_of_the_host_is_refused(host_calls, name):
    with pytest.raises(ValueError, match="workspace must be a device tensor"):
        CALLS[name](torch.zeros(ENOUGH, dtype=torch.uint8))


class Elsewhere:
    """A tensor as if it were on cuda:0 or another device, with its strides and type."""

    def __init__(self, t, index=0):
        self.t, self.index, self.device = t, index, f"cuda:{index}"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_workspace_of_another_device_or_with_strides_is_refused():
    like = Elsewhere(torch.zeros(4))
    big = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        B._workspace(Elsewhere(big, 1), 256, like)
    # one byte of memory with the shape of many
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        B._workspace(Elsewhere(big[:1].expand(4096)), 256, like)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        B._workspace(Elsewhere(big[::2]), 256, like)
    with pytest.raises(ValueError, match="workspace must be a device tensor"):
        B._workspace(big, 0, like)          # also where none is needed
    ws = Elsewhere(big)
    assert B._workspace(ws, 4096, like) is ws
    # bytes count, not elements
    ws = Elsewhere(torch.zeros(64))
    assert B._workspace(ws, 256, like) is ws
    assert B._workspace(None, 0, like) is None


STREAM_CALLS = {
    "router_logits": lambda s: B.router_logits(bf(256, 2048), bf(1024, 2048), bf(1024, 2048),
                                               stream=s),
    "product_topk": lambda s: B.product_topk(torch.zeros(8, 64), torch.zeros(8, 64), 8, 8,
                                             stream=s),
    "atomic_forward": lambda s: B.atomic_forward(bf(8, 128), bf(64, 128), bf(64, 128),
                                                 sched(8, 4, 64), stream=s),
    "atomic_forward_glu": lambda s: B.atomic_forward_glu(
        bf(8, 128), bf(64, 128), bf(64, 128), bf(64, 128), sched(8, 4, 64), stream=s),
    "flat_router_topk": lambda s: B.flat_router_topk(bf(8, 128), bf(64, 128), 4, stream=s),
    "shared_mlp": lambda s: B.shared_mlp(bf(8, 128), bf(64, 128), bf(64, 128), bf(128, 64),
                                         stream=s),
    "routed_backward": lambda s: B.routed_backward(
        bf(8, 128), bf(8, 128), bf(8, 128), bf(64, 128), bf(64, 128), i32(8, 4),
        torch.zeros(8, 4), torch.zeros(8, 128), stream=s),
    "expert_weight_grad": lambda s: B.expert_weight_grad(
        bf(8192, 64), bf(8192, 64), i32(2), dw=torch.zeros(1, 64, 64), stream=s),
}


@pytest.mark.parametrize("name", list(STREAM_CALLS))
def test_a_fresh_workspace_belongs_to_the_stream_of_the_call(host_calls, monkeypatch, name):
    """Freed when the call returns, it may be reused at once by its own stream only."""
    streams = []

    def empty(shape, dtype, like, stream):
        streams.append(stream)
        return torch.empty(shape, dtype=dtype)
    monkeypatch.setattr(B, "_empty", empty)
    mine = object()
    try:
        STREAM_CALLS[name](mine)
    except Reached:
        pass
    assert streams == [mine]


def meta(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


BF, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
FAR = (1 << 32) + 5     # 5 in the library's 32-bit sizes
FAR_CALLS = {
    "rows to quantise": lambda: B.quantize_rows(meta((FAR, 16), BF), q=1, scale=1),
    "columns to quantise": lambda: B.quantize_rows(meta((1, FAR + 11), BF), q=1, scale=1),
    "rows of x": lambda: B.expert_matmul(meta((FAR, 8), BF), meta((2, 8, 8), BF), meta((3,), I32),
                                         x_row=meta((4,), I32)),
    "tasks": lambda: B.expert_matmul(meta((4, 8), BF), meta((2, 8, 8), BF), meta((3,), I32),
                                     x_row=meta((FAR,), I32), out=meta((4, 8), BF)),
    "output rows": lambda: B.expert_matmul(meta((4, 8), BF), meta((2, 8, 8), BF), meta((3,), I32),
                                           out=meta((FAR, 8), BF)),
    "experts": lambda: B.expert_matmul(meta((4, 8), BF), meta((FAR, 8, 8), BF),
                                       meta((FAR + 1,), I32)),
    "outputs": lambda: B.expert_matmul(meta((4, 8), BF), meta((1, FAR, 8), BF), meta((2,), I32)),
    "rows of dy": lambda: B.expert_weight_grad(meta((4, 8), BF), meta((FAR, 8), BF),
                                               meta((3,), I32), dw=meta((2, 8, 8), F32)),
    "experts of dw": lambda: B.expert_weight_grad(meta((4, 8), BF), meta((4, 8), BF),
                                                  meta((FAR + 1,), I32),
                                                  dw=meta((FAR, 8, 8), F32)),
    "rows to combine": lambda: B.expert_combine(meta((FAR, 8), BF), 1, y=meta((FAR, 8), F32)),
    "rows of dout": lambda: B.expert_combine_backward(meta((FAR, 8), BF), None,
                                                      meta((FAR, 8), F32), do=1, dgate=1),
    "8-bit rows": lambda: B.quantized_matmul(meta((FAR, 16), I8), None, meta((8, 16), I8), None,
                                             out=meta((FAR, 8), BF)),
    "8-bit weights": lambda: B.quantized_matmul(meta((4, 16), I8), None, meta((FAR, 16), I8), None,
                                                out=meta((4, FAR), BF)),
    "8-bit output rows": lambda: B.quantized_expert_matmul(
        meta((4, 16), I8), None, meta((2, 8, 16), I8), None, meta((3,), I32),
        out=meta((FAR, 8), BF)),
}


@pytest.mark.parametrize("name", list(FAR_CALLS))
def test_sizes_past_32_bits_are_refused(host_calls, name):
    """The library's sizes are 32-bit: one past them would reach it as another one."""
    with pytest.raises(ValueError, match="2\\^31"):
        FAR_CALLS[name]()
