"""A cache's rule is replaced while its routing is still to come: the old bias may be overwritten on the cache's stream."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle.routing import Rule, route_by  # noqa: E402

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.pipeline import ExpertCache
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"


@pytest.mark.parametrize("side", [False, True])
def test_writes_after_set_router_come_after_the_routing(side):
    from synth import workloads as W
    from tests.harness import make_bank
    L, E, k, T = 2, 64, 4, 16
    w = W.QWEN35B_DECODE.replace(num_layers=L, num_experts=E, top_k=k, hidden=128, inter=128, tokens=T, num_slots=2 * E)
    bank, blobs = make_bank(w, 2)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    cache = ExpertCache(L, E, k, 128, 128, w.wdtype, 2 * E, T, bank, blobs, device=torch.device(DEV), stream=stream)
    rng = np.random.default_rng(1)
    try:
        for step in range(4):
            x, b = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal(E).astype(np.float32)
            logits, bias = torch.tensor(x, device=DEV), torch.tensor(b, device=DEV)
            idx, gw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
            torch.cuda.synchronize()
            cache.set_router(Router(E, k, score="sigmoid", bias=bias))
            with torch.cuda.stream(stream):
                torch.cuda._sleep(2_000_000)  # about a millisecond: the routing waits for it
                cache.route_classify(step % L, logits, idx, gw)
                cache.set_router(None if step % 2 else Router(E, k))
                bias.fill_(float("nan"))
            del bias
            with torch.cuda.stream(stream):
                other = [torch.full((E,), 1e30, device=DEV) for _ in range(8)]  # (one of them may get its memory)
            cache.synchronize()
            torch.cuda.synchronize()
            del other
            assert np.array_equal(idx.cpu().numpy(), route_by(Rule("sigmoid", b.astype(np.float64)), x, k)[0])
    finally:
        cache.close()


def test_a_rule_may_be_set_after_a_step_graph_and_many_times():
    """The event of the wait has been part of a graph's capture before."""
    from expert_cache_host_layer_gb300.pipeline import StepGraph
    from synth import workloads as W
    from tests.harness import make_bank
    L, E, k, T = 2, 64, 4, 2
    w = W.QWEN35B_DECODE.replace(num_layers=L, num_experts=E, top_k=k, hidden=128, inter=128, tokens=T, num_slots=2 * E)
    bank, blobs = make_bank(w, 2)
    cache = ExpertCache(L, E, k, 128, 128, w.wdtype, 2 * E, T, bank, blobs, device=torch.device(DEV))
    rng = np.random.default_rng(2)
    try:
        rules = [rng.standard_normal(E).astype(np.float32) for _ in range(3)]
        logits = [torch.tensor(rng.standard_normal((T, E)).astype(np.float32), device=DEV) for _ in range(L)]
        xs, ys = [torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV)] * L, [torch.empty(T, 128, device=DEV) for _ in range(L)]
        cache.set_router(Router(E, k, bias=torch.tensor(rules[0], device=DEV)))
        graph = StepGraph(cache, logits, xs, ys)
        for b in rules[1:]:
            cache.set_router(Router(E, k, bias=torch.tensor(b, device=DEV)))
            graph.launch()
            idx, gw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
            cache.synchronize()
            cache.route_classify(0, logits[0], idx, gw)
            cache.set_router(None)
            cache.synchronize()
            want = route_by(Rule("softmax", b.astype(np.float64)), logits[0].cpu().numpy(), k)[0]
            assert np.array_equal(idx.cpu().numpy(), want)
        graph.close()
    finally:
        cache.close()
