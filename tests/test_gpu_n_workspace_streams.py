"""A call on another stream than the current one, with a workspace of its own:
memory that the current stream takes right after the call is not that workspace."""
import pytest
import torch

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


def test_workspace_outlives_a_call_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x, wg, wu, wd = r(512, 256), r(512, 256), r(512, 256), r(256, 512)
    a, wr, wc = r(256, 2048), r(1024, 2048), r(1024, 2048)
    want = [B.shared_mlp(x, wg, wu, wd), *B.router_logits(a, wr, wc)]
    torch.cuda.synchronize()
    sizes = [B.lib().omni_shared_mlp_workspace(1, 512, 256, 512),
             B.lib().omni_router_logits_workspace(1, 256, 2048, 1024, 1024)]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)       # the calls below wait behind this
        got = [B.shared_mlp(x, wg, wu, wd, stream=side),
               *B.router_logits(a, wr, wc, stream=side)]
        for n in sizes:
            torch.full((n // 4,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
