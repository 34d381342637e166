"""Routing rules (Router.route, ExpertCache.set_router) against the fp64 oracle.

Experts have to be the oracle's, in its order, also where values differ by less
than fp32 can tell.  Gates (u = 2^-24): an exponential is good to 2 ulp and its
argument's rounding, d u for an argument of size d; the denominator is a sum of at
most 32 terms in a lane and 5 levels, and quotients, the scale and the last
rounding add a few u:

    |w - exact| <= (64 + 4 d) u |w| + 2^-120 |scale|,

d the largest distance of a pick's logit from the row's largest (softmax) or 0.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle.routing import Rule, clean, route_by  # noqa: E402

if torch.cuda.is_available():
    import expert_cache_host_layer_gb300 as ft
    from expert_cache_host_layer_gb300.pipeline import ExpertCache, StepGraph
    from expert_cache_host_layer_gb300.router import Router

DEV = "cuda:0"
GUARD = 24


def router(rule, E, k):
    bias = None if rule.bias is None else torch.tensor(rule.bias, dtype=torch.float32, device=DEV)
    return Router(E, k, score=rule.score, bias=bias, groups=rule.groups, top_groups=rule.top_groups, group_top=rule.group_top,
                  renormalise=rule.renormalise, scale=rule.scale)


def run(rule, logits, k, r=None, stream=None):
    T, E = logits.shape
    idx = torch.full((T + 1, k), GUARD, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), float(GUARD), device=DEV)
    (r or router(rule, E, k)).route(logits, idx[:T], w[:T], stream=stream)
    torch.cuda.synchronize()
    assert (idx[T:] == GUARD).all() and (w[T:] == GUARD).all()
    return idx[:T].cpu().numpy(), w[:T].double().cpu().numpy()


def check(rule, logits, k, got):
    x = logits.double().cpu().numpy()
    idx, w = route_by(rule, x, k)
    assert np.array_equal(got[0], idx), np.flatnonzero((got[0] != idx).any(axis=1))[:5]
    x = clean(x)
    picked = np.take_along_axis(x, idx.astype(np.int64), axis=1)
    d = np.zeros_like(picked)
    if rule.score == "softmax":
        with np.errstate(invalid="ignore"):
            d = np.nan_to_num(x.max(axis=1, keepdims=True) - picked, nan=0.0, posinf=0.0)
    bound = (64 + 4 * np.minimum(d.max(axis=1, keepdims=True), 200)) * 2.0 ** -24 * np.abs(w) + 2.0 ** -120 * abs(rule.scale)
    assert (np.abs(got[1] - w) <= bound).all(), float(np.abs(got[1] - w).max())


def normal(T, E, seed=0, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=gen) * spread).to(DEV)


def f32(x):
    return np.asarray(x, dtype=np.float32).astype(np.float64)


SHAPES = [(1, 256, 8, 8, 4), (77, 256, 8, 8, 4), (5, 1, 1, 1, 1), (33, 16, 2, 1, 1), (9, 60, 4, 1, 1), (300, 72, 6, 1, 1),
          (40, 160, 6, 8, 3), (21, 60, 7, 4, 2), (13, 1024, 32, 1, 1), (12, 1024, 9, 16, 5), (17, 384, 8, 1, 1), (14, 96, 32, 32, 16),
          (700, 64, 8, 2, 1), (6147, 256, 8, 8, 4), (6146, 72, 6, 1, 1), (7000, 64, 8, 2, 1), (6145, 160, 6, 8, 3), (6500, 16, 2, 1, 1),
          (6144, 30, 1, 5, 1), (6149, 256, 8, 1, 1), (6143, 256, 8, 1, 1), (6500, 128, 16, 1, 1), (6500, 64, 5, 16, 3), (25, 27, 6, 9, 2), (8, 37, 37 // 2, 1, 1), (6, 640, 3, 5, 1)]


@pytest.mark.parametrize("T,E,k,groups,top_groups", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
def test_choice_and_gates(T, E, k, groups, top_groups, score, bias, group_top):
    rng = np.random.default_rng(T + E)
    b = f32(rng.standard_normal(E) * (0.2 if score == "sigmoid" else 0.5 / E)) if bias else None
    logits = normal(T, E, seed=E + k)
    for renormalise, scale in ((True, 1.0), (False, 2.5)):
        rule = Rule(score, b, groups, top_groups, group_top, renormalise, scale)
        check(rule, logits, k, run(rule, logits, k))
    half = logits.bfloat16()  # few different values: many are equal
    check(rule, half, k, run(rule, half, k))


@pytest.mark.parametrize("E,groups", [(256, 8), (72, 1), (60, 4)])
def test_views_of_a_wider_tensor(E, groups):
    for extra, dtype in ((3, torch.float32), (8, torch.float32), (1, torch.bfloat16), (8, torch.bfloat16)):
        wide = normal(30, E + extra, seed=3).to(dtype)
        for at in sorted({0, 1, extra}):
            x = wide[:, at:at + E]
            rule = Rule("sigmoid", None, groups, max(1, groups // 2), 2)
            check(rule, x, 4, run(rule, x, 4))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(256, 8, 1), (256, 8, 8), (100, 6, 1), (64, 5, 4)])
def test_values_that_fp32_cannot_tell_apart(score, E, k, groups):
    """A bias that all but cancels the scores: s + bias is the same up to the bias's own fp32 rounding (some 1e-9), so the
    whole choice is one between values that are equal in fp32."""
    rng = np.random.default_rng(E)
    logits = f32(rng.standard_normal((1, E)))
    s = 1 / (1 + np.exp(-logits)) if score == "sigmoid" else np.exp(logits) / np.exp(logits).sum()
    rule = Rule(score, f32(0.75 - s[0]), groups, max(1, groups // 2), min(2, groups))
    x = torch.tensor(logits, dtype=torch.float32, device=DEV)
    check(rule, x, k, run(rule, x, k))
    x = x.repeat(6200, 1)
    check(rule, x, k, run(rule, x, k))
    # and where only some are: pairs of experts
    rule.bias = f32(np.where(np.arange(E) % 7 == 0, 0.75 - s[0], 0.0))
    check(rule, x, k, run(rule, x, k))


@pytest.mark.parametrize("T", [400, 6150])
def test_rows_with_close_values_among_many(T):
    """Rows of one call with and without such pairs, the pairs at every place of the choice."""
    rng = np.random.default_rng(8)
    E, k = 128, 8
    logits = f32(rng.standard_normal((T, E)))
    b = f32(rng.standard_normal(E) * 0.1)
    s = 1 / (1 + np.exp(-logits))
    for t in range(0, T, 2):  # the logit of another expert that gives it the same v, rounded to fp32
        order = np.argsort(-(s[t] + b))
        i, j = order[rng.integers(0, k + 2)], rng.integers(0, E)
        v = s[t, i] + b[i] - b[j]
        if 0.01 < v < 0.99:
            logits[t, j] = f32(np.log(v / (1 - v)))
    rule = Rule("sigmoid", b)
    x = torch.tensor(logits, dtype=torch.float32, device=DEV)
    check(rule, x, k, run(rule, x, k))
    rule = Rule("sigmoid", b, 8, 3, 2)
    check(rule, x, k, run(rule, x, k))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (8, 1), (8, 2)])
@pytest.mark.parametrize("copies", [1, 513])
def test_equal_logits_and_values_that_are_not_finite(score, bias, groups, group_top, copies):
    E, k = 256, 8
    x = np.round(np.random.default_rng(5).standard_normal((12, E)) * 2) / 2
    x[1] = 0.0
    x[2] = -np.inf
    x[3, ::2] = np.nan
    x[4, 5] = np.inf
    x[5, [9, 200, 30]] = np.inf
    x[6, :] = np.nan
    x[6, 77] = -3.0
    x[7, ::3] = -0.0
    x[8] = -200.0 - np.arange(E) / 8
    x[9] = 300.0 + np.arange(E) / 8
    x[10, :] = -np.inf
    x[10, [3, 250]] = 1.0
    x[11, 31::32] = np.nan
    b = None
    if bias:
        b = f32(np.round(np.random.default_rng(6).standard_normal(E) * 8) / 64)
        b[[4, 90]], b[7], b[8] = np.nan, np.inf, -np.inf
    rule = Rule(score, b, groups, max(1, groups // 2), group_top)
    logits = torch.tensor(x, dtype=torch.float32, device=DEV)
    one = run(rule, logits, k)
    check(rule, logits, k, one)
    many = run(rule, logits.repeat(copies, 1), k)  # enough rows for several to a warp
    assert all(np.array_equal(m, np.tile(o, (copies, 1))) for m, o in zip(many, one))


def test_far_biases():
    """Biases of size 30 and of size 1e-6: the order is that of the exact sums."""
    rng = np.random.default_rng(9)
    logits = torch.tensor(rng.standard_normal((200, 256)), dtype=torch.float32, device=DEV)
    many = logits.repeat(31, 1)
    for scale in (30.0, 1e-6, 1e30, 3e38):
        for groups in (1, 8):
            rule = Rule("sigmoid", f32(np.clip(rng.standard_normal(256), -1, 1) * scale), groups, max(1, groups // 2), 2 if groups > 1 else 1)
            check(rule, logits, 8, run(rule, logits, 8))
            check(rule, many, 8, run(rule, many, 8))
    rule.bias = f32(rng.integers(-2, 3, 256) * 4.0)  # whole steps apart: groups whose best two cancel
    check(rule, logits, 8, run(rule, logits, 8))


def test_on_another_stream_in_graphs_and_a_changing_bias():
    rng = np.random.default_rng(2)
    rule = Rule("sigmoid", f32(rng.standard_normal(256) * 0.1), 8, 4, 2)
    r = router(rule, 256, 8)
    x = normal(100, 256, seed=11)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(rule, x, 8, run(rule, x, 8, r, stream=side))
    idx, w = torch.empty(100, 8, dtype=torch.int32, device=DEV), torch.empty(100, 8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.route(x, idx, w)
    for seed in (12, 13):
        x.copy_(normal(100, 256, seed=seed))
        rule.bias = f32(rng.standard_normal(256) * 0.1)
        r.bias.copy_(torch.tensor(rule.bias))
        g.replay()
        torch.cuda.synchronize()
        check(rule, x, 8, (idx.cpu().numpy(), w.double().cpu().numpy()))


def test_refusals():
    r = Router(64, 4)
    x, idx, w = normal(3, 64), torch.zeros(3, 4, dtype=torch.int32, device=DEV), torch.zeros(3, 4, device=DEV)
    for args, text in (((x[:, :32], idx, w), "logits is"), ((x.half(), idx, w), "logits is"), ((x, idx.long(), w), "topk_idx"),
                       ((x, idx[:2], w), "topk_idx"), ((x, idx, w.bfloat16()), "topk_idx"), ((x.T.contiguous().T, idx, w), "contiguous"),
                       ((x.cpu(), idx, w), "GPU")):
        with pytest.raises(ValueError, match=text):
            r.route(*args)
    with pytest.raises(ValueError, match="cache's routing"):
        Router(64, 4, bias=torch.zeros(2, 64, device=DEV)).route(x, idx, w)
    r.route(x[:0], idx[:0], w[:0])


# ---------------------------------------------------------------- a cache's routing

def make_cache(T, L=3, E=256, k=8, C=600, hidden=128, inter=128):
    import synth
    from synth import workloads as W
    from tests.harness import make_bank
    w = W.QWEN35B_DECODE.replace(num_layers=L, num_experts=E, top_k=k, hidden=hidden, inter=inter, tokens=T, num_slots=C)
    bank, blobs = make_bank(w, 8)
    del synth
    return w, bank, blobs, ExpertCache(L, E, k, hidden, inter, w.wdtype, C, T, bank, blobs, device=torch.device(DEV))


def events(cache, rule_of, logits, L, E, k, T, ref):
    """One routing of every layer: picks, gates and the cache's decisions against the oracle's."""
    from tests.harness import compare_event
    idx, gw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    for l in range(L):
        cache.route_classify(l, logits[l], idx, gw)
        ridx, rw = route_by(rule_of(l), logits[l].double().cpu().numpy(), k)
        errs = compare_event(cache.plan(l), ref.event(l, ridx), idx.cpu().numpy(), ridx, gw.cpu().numpy(), rw)
        assert not errs, (l, errs[:3])


@pytest.mark.parametrize("T", [1, 4, 64])
def test_a_cache_routes_by_the_rule(T):
    from oracle.cache import ExpertCacheOracle
    L, E, k = 3, 256, 8
    w, bank, blobs, cache = make_cache(T)
    rng = np.random.default_rng(T)
    bias = f32(rng.standard_normal((L, E)) * 0.2)
    rule = Rule("sigmoid", None, 8, 4, 2, True, 2.5)

    def of(l):
        return Rule(rule.score, bias[l], 8, 4, 2, True, 2.5)
    ref = ExpertCacheOracle(L, E, w.num_slots)
    try:
        with pytest.raises(ValueError, match="of 256 experts"):
            cache.set_router(Router(E, 4))
        with pytest.raises(ValueError, match="bias"):
            cache.set_router(Router(E, k, bias=torch.zeros(L + 1, E, device=DEV)))
        for step in range(6):
            by_rule = step % 3 != 2  # the default in between
            cache.set_router(Router(E, k, score="sigmoid", bias=torch.tensor(bias, dtype=torch.float32, device=DEV), groups=8,
                                    top_groups=4, group_top=2, scale=2.5) if by_rule else None)
            logits = [normal(T, E, seed=100 * step + l) for l in range(L)]
            events(cache, of if by_rule else lambda l: Rule(), logits, L, E, k, T, ref)
    finally:
        cache.close()


def test_the_default_rule_is_the_default():
    """ft_route with the default rule: bit for bit the cache's own picks and gates."""
    T, L, E, k = 50, 1, 256, 8
    w, bank, blobs, cache = make_cache(T, L=L)
    try:
        x = normal(T, E, seed=4)
        x[::5] = (x[::5] * 4).round() / 4
        idx, gw = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
        cache.route_classify(0, x, idx, gw)
        cache.synchronize()
        got = run(Rule(), x, k)
        assert np.array_equal(got[0], idx.cpu().numpy()) and np.array_equal(got[1], gw.double().cpu().numpy())
    finally:
        cache.close()


def test_a_step_graph_keeps_its_rule():
    """Step graphs with and without a rule, each against the experts' products by the oracle."""
    from oracle import ffn as offn
    from tests.harness import bank_blob
    T, L, E, k = 2, 3, 64, 4
    w, bank, blobs, cache = make_cache(T, L=L, E=E, k=k, C=100)
    rule = Rule("sigmoid", f32(np.random.default_rng(1).standard_normal(E) * 0.3), 4, 2, 2, False, 1.5)
    try:
        logits, xs = [normal(T, E, seed=l) for l in range(L)], [normal(T, 128, seed=9 + l).bfloat16() for l in range(L)]
        ys = [[torch.empty(T, 128, device=DEV) for _ in range(L)] for _ in range(2)]
        cache.set_router(router(rule, E, k))
        by_rule = StepGraph(cache, logits, xs, ys[0])
        cache.set_router(None)
        plain = StepGraph(cache, logits, xs, ys[1])
        for step in range(3):
            for l in range(L):
                logits[l].copy_(normal(T, E, seed=50 + 10 * step + l))
            torch.cuda.synchronize()
            for g, y, of in ((by_rule, ys[0], rule), (plain, ys[1], Rule())):
                g.launch()
                cache.synchronize()
                for l in range(L):
                    idx, gates = route_by(of, logits[l].double().cpu().numpy(), k)
                    want = offn.moe_ffn(xs[l].double().cpu().numpy(), idx, gates, lambda e, l=l: offn.dequant_blob(
                        bank_blob(bank, w, blobs, l, e), 128, 128, w.wdtype))
                    assert np.abs(y[l].double().cpu().numpy() - want).max() <= 2e-2 * np.sqrt((want ** 2).mean())
        by_rule.close()
        plain.close()
    finally:
        cache.close()


def test_picks_feed_the_experts_without_a_cache():
    """route, then ft_moe_decode_ffn_static on its picks and gates."""
    from oracle import ffn as offn
    from tests.harness import bank_blob
    T, E, k, H = 4, 64, 4, 128
    w, bank, blobs, cache = make_cache(1, L=1, E=E, k=k, C=2 * k)
    cache.close()
    pool = bank.to(DEV)
    rule = Rule("softmax", None, 4, 2, 1, False, 4.0)
    x, logits = normal(T, H, seed=3).bfloat16(), normal(T, E, seed=2)
    slot = (torch.arange(E, dtype=torch.int32) % blobs).to(DEV)
    idx, gw, y = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV), torch.empty(T, H, device=DEV)
    router(rule, E, k).route(logits, idx, gw)
    ft.ft_moe_decode_ffn_static(H, 128, w.wdtype, E, k, pool.data_ptr(), blobs, slot.data_ptr(), idx.data_ptr(), gw.data_ptr(),
                                x.data_ptr(), T, y.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    ridx, gates = route_by(rule, logits.double().cpu().numpy(), k)
    want = offn.moe_ffn(x.double().cpu().numpy(), ridx, gates, lambda e: offn.dequant_blob(bank_blob(bank, w, blobs, 0, e), H, 128, w.wdtype))
    assert np.array_equal(idx.cpu().numpy(), ridx)
    assert np.abs(y.double().cpu().numpy() - want).max() <= 2e-2 * np.sqrt((want ** 2).mean())
