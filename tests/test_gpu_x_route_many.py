"""The routing tests with each batch repeated until the tokens are many, which other
kernels take; every repeat has to come out alike."""
import pytest

from tests import test_gpu_q_route as Q
from tests.test_gpu_q_route import (  # noqa: F401
    test_route_backward, test_route_backward_ids_twice_and_out_of_range, test_route_groups,
    test_route_masks_infinities_and_nan, test_route_pairs_next_to_each_other,
    test_route_scores_next_to_each_other, test_route_sizes, test_route_ties_go_to_the_lower_index)

pytest.importorskip("cartesian_routed_atomic_amd.binding")
pytestmark = pytest.mark.gpu


class Many:
    """The binding's calls on repeated batches; what they return, of the first."""

    def __init__(self, calls):
        self.calls = calls

    def times(self, L, E):
        if not 64 < E <= 512:
            pytest.skip("one kernel for all numbers of tokens")
        return 16 * E // L + 2

    def first(self, t, n, L):
        if t is None:
            return None
        v = t.view(n, L, -1)
        assert ((v == v[:1]) | ((v != v) & (v[:1] != v[:1]))).all()
        return t[:L]

    def expert_route(self, logits, K, **kw):
        L, E = logits.shape
        n = self.times(L, E)
        out = self.calls.expert_route(logits.repeat(n, 1), K, **kw)
        return tuple(self.first(t, n, L) for t in out)

    def expert_route_backward(self, logits, expert_idx, dgate, dscore=None, **kw):
        L, E = logits.shape
        n = self.times(L, E)
        if dscore is not None and dscore.dim() == 2:
            dscore = dscore.repeat(n, 1)
        return self.first(self.calls.expert_route_backward(
            logits.repeat(n, 1), expert_idx.repeat(n, 1), dgate.repeat(n, 1), dscore=dscore,
            **kw), n, L)


@pytest.fixture(autouse=True)
def many(monkeypatch):
    monkeypatch.setattr(Q, "B", Many(Q.B))


@pytest.mark.parametrize("E,groups,top,best", [(300, 6, 3, 2), (512, 8, 4, 2), (500, 10, 2, 1),
                                               (264, 12, 11, 2)])
@pytest.mark.parametrize("fn,biased", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_route_groups_of_many_experts(E, groups, top, best, fn, biased):
    rng = Q.np.random.default_rng(E)
    bias = (0.1 * rng.standard_normal(E)).astype(Q.np.float32) if biased else None
    for dt in ("f32", "bf16"):
        Q.check(Q.logits(rng, 61, E, dt), 16, bias=bias, fn=fn, groups=groups, top_groups=top,
                group_best=best)
