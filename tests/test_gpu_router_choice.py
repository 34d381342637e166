"""The choice of experts where fp64 scores cannot tell values apart: equal
biases, whose order is that of the logits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle.routing import Rule, route_by  # noqa: E402

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"
LOGITS = {"high": (28.0, 60.0), "far": (60.0, 3000.0), "low": (-60.0, -28.0), "both": (-300.0, 300.0), "near": (-2.0, 2.0)}


def spread(T, E, lo, hi, seed):
    return np.random.default_rng(seed).uniform(lo, hi, (T, E)).astype(np.float32)


def picks(E, k, x, bias, score, groups, top_groups):
    logits = torch.tensor(x, device=DEV)
    idx, w = torch.empty(len(x), k, dtype=torch.int32, device=DEV), torch.empty(len(x), k, device=DEV)
    Router(E, k, score=score, bias=torch.tensor(bias, dtype=torch.float32, device=DEV), groups=groups, top_groups=top_groups,
           renormalise=False).route(logits, idx, w)
    return idx.cpu().numpy()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("where", LOGITS)
@pytest.mark.parametrize("bias", [0.0, 0.25, -1e9])
@pytest.mark.parametrize("T,E,k,groups", [(1, 256, 8, 1), (50, 256, 8, 8), (7, 60, 4, 4), (5, 1024, 32, 1), (6200, 64, 8, 2), (6200, 256, 8, 1)])
def test_equal_biases_leave_the_order_of_the_logits(score, where, bias, T, E, k, groups):
    """The same bias for all (0: a learned one at its start) changes no choice, whatever it swallows of the scores."""
    x = spread(T, E, *LOGITS[where], seed=E + T)
    want, _ = route_by(Rule(score, None, groups, max(1, groups // 2)), x, k)  # by the logits alone
    assert np.array_equal(picks(E, k, x, np.full(E, bias), score, groups, max(1, groups // 2)), want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("where", LOGITS)
@pytest.mark.parametrize("T", [9, 6200])
def test_two_biases(score, where, T):
    """Experts of the higher bias first (the scores are below 1), each half by its logits."""
    E, k = 64, 8
    x = spread(T, E, *LOGITS[where], seed=T)
    bias = np.zeros(E)
    bias[5::13] = 2.0  # five of them
    want = np.array([np.lexsort((-row, -bias))[:k] for row in x])
    assert np.array_equal(picks(E, k, x, bias, score, 1, 1), want)


@pytest.mark.parametrize("T", [40, 6200])
def test_values_without_a_number_go_by_the_expert(T):
    """A bias of -inf leaves nothing to compare; one that is NaN counts as that."""
    E, k = 64, 8
    x = spread(T, E, -3.0, 3.0, seed=4)
    bias = np.full(E, -np.inf)
    bias[[60, 20, 33]] = 0.0, 4.0, 2.0
    bias[1] = np.nan
    want = np.tile(np.array([20, 33, 60, 0, 1, 2, 3, 4]), (T, 1))
    assert np.array_equal(picks(E, k, x, bias, "sigmoid", 1, 1), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(512, 8, 1), (512, 16, 8), (384, 9, 3), (1024, 32, 1), (1024, 8, 16)])
def test_close_values_with_many_a_lane(score, E, k, groups):
    """A bias that all but cancels the scores, at 16 and 32 values a lane: the choice is one between values that are equal in
    fp32, for all experts and for every seventh."""
    rng = np.random.default_rng(E)
    x = rng.standard_normal((1, E)).astype(np.float32)
    l = x.astype(np.float64)
    s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l) / np.exp(l).sum()
    all_of_them = (0.75 - s[0]).astype(np.float32).astype(np.float64)
    for bias in (all_of_them, np.where(np.arange(E) % 7 == 0, all_of_them, 0.0)):
        want, _ = route_by(Rule(score, bias, groups, max(1, groups // 2)), x, k)
        rows = np.repeat(x, 5, axis=0)
        assert np.array_equal(picks(E, k, rows, bias, score, groups, max(1, groups // 2)), np.repeat(want, 5, axis=0))
