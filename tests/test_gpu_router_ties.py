"""Rows of equal fp32 logits without a bias: which of them are picked, and in which order."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle.routing import Rule, route_by  # noqa: E402

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"


@pytest.mark.parametrize("T", [1, 30, 6200])
@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (384, 16), (1024, 32)])
def test_rows_of_equal_logits_without_a_bias(T, E, k):
    """fp32 logits of few different values: each pick is one of many equal ones, its place the expert's number's."""
    x = np.random.default_rng(E).integers(0, 3, (T, E)).astype(np.float32)
    x[::3] = 1.5
    logits = torch.tensor(x, device=DEV)
    for rule in (Rule(), Rule("sigmoid", None, 4, 2)):
        idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
        r = Router(E, k, score=rule.score, groups=rule.groups, top_groups=rule.top_groups)
        want = route_by(rule, x, k)[0]
        for _ in range(20):
            idx.fill_(-1)
            r.route(logits, idx, w)
            assert np.array_equal(idx.cpu().numpy(), want)
