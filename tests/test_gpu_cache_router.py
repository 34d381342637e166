"""ExpertCache.set_router over the shapes that its kernel has variants for:
values a lane, groups, rows that are no whole vectors, more tokens than the
grid has warps for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle.routing import Rule, route_by  # noqa: E402

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.pipeline import ExpertCache
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"


def make_cache(T, L, E, k):
    from synth import workloads as W
    from tests.harness import make_bank
    C = 2 * min(T * k, E) + 3
    w = W.QWEN35B_DECODE.replace(num_layers=L, num_experts=E, top_k=k, hidden=128, inter=128, tokens=T, num_slots=C)
    bank, blobs = make_bank(w, 2)
    return C, ExpertCache(L, E, k, 128, 128, w.wdtype, C, T, bank, blobs, device=torch.device(DEV))


# values a lane 1 (16, and groups of 6), 2 (60 in 4), 4 (128), 8 (256), 16 (384), 32 (1024); 5000 and more rows: a warp's second
SHAPES = [(16, 2, 1, 1, 5), (30, 3, 5, 2, 7), (60, 4, 4, 2, 33), (128, 8, 1, 1, 12), (256, 8, 8, 4, 5000), (384, 8, 1, 1, 9),
          (1024, 32, 1, 1, 9), (1024, 9, 16, 5, 3), (64, 6, 2, 1, 10007)]


@pytest.mark.parametrize("E,k,groups,top_groups,T", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_picks_gates_and_decisions(E, k, groups, top_groups, T, score, bias):
    from oracle.cache import ExpertCacheOracle
    from tests.harness import compare_event
    L = 2
    rng = np.random.default_rng(E + T)
    b = (rng.standard_normal((L, E)) * (0.2 if score == "sigmoid" else 0.5 / E)).astype(np.float32) if bias else None
    C, cache = make_cache(T, L, E, k)
    ref = ExpertCacheOracle(L, E, C)
    group_top = 2 if groups > 1 else 1
    try:
        cache.set_router(Router(E, k, score=score, bias=None if b is None else torch.tensor(b, device=DEV), groups=groups,
                                top_groups=top_groups, group_top=group_top, scale=1.5))
        idx, gw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
        wide = torch.empty(T * E + 1, device=DEV)
        for event in range(4):
            l = event % L
            x = rng.standard_normal((T, E)).astype(np.float32)
            at = event // L  # the second time rows start at no 16-byte boundary
            logits = wide[at:at + T * E].view(T, E)
            logits.copy_(torch.tensor(x))
            cache.route_classify(l, logits, idx, gw)
            ridx, rw = route_by(Rule(score, None if b is None else b[l].astype(np.float64), groups, top_groups, group_top, True, 1.5),
                                x.astype(np.float64), k)
            errs = compare_event(cache.plan(l), ref.event(l, ridx), idx.cpu().numpy(), ridx, gw.cpu().numpy(), rw)
            assert not errs, (event, [e[0] for e in errs], str(errs[0][1])[:300])
    finally:
        cache.close()
