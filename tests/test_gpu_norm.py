"""RMSNorm.apply (ft_add_norm) against the fp64 oracle.

Error bounds (u = 2^-24, fp32's unit roundoff).  r is one fp32 sum: u |r|.  Its
mean square is a sum of at most 32 terms in a thread and 10 levels between
threads, a quotient and eps: off by at most 48 u of itself (2 u of them r's);
the inverse root halves that and adds u, and the two products 2 u more:

    |y - exact| <= 30 u |y|  <  2^-19 |y|,

and a bf16 result is rounded once, 2^-8 |y|.  A scale is a largest |y| over 448:
2^-19 of itself.  A code is y / scale, off by less than 2^-18 of itself, rounded
to 4 bits (2^-4 of the value, or half a step of 2^-9).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import norm as onorm  # noqa: E402

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300 import FtError
    from expert_cache_host_layer_gb300.norm import RMSNorm

DEV = "cuda:0"
BF, F, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ROUND = {BF: 2.0 ** -8, F: 0.0}
GUARD = 24.0


def host(t):
    return t.double().cpu().numpy()


def make(rows, hidden, xt, dt, wt, seed=0, pad=0):
    """Tensors with rows `pad` elements further apart than hidden."""
    gen = torch.Generator().manual_seed(seed)

    def matrix(t):
        m = torch.randn(rows, hidden + pad, generator=gen) * torch.exp(torch.randn(hidden + pad, generator=gen))
        return m.to(t).to(DEV)[:, :hidden]
    x = matrix(xt)
    delta = matrix(dt) if dt else None
    w = (1 + 0.3 * torch.randn(hidden, generator=gen)).to(wt).to(DEV) if wt else None
    return x, delta, w


def blank(rows, hidden, t, pad=0):
    """A tensor of guard values, and its view of hidden columns."""
    whole = torch.full((rows + 1, hidden + pad), GUARD, device=DEV).to(t)
    return whole, whole[:rows, :hidden]


def untouched(whole, rows, hidden):
    w = host(whole)
    return (w[rows:] == GUARD).all() and (w[:, hidden:] == GUARD).all()


def check(x, delta, w, out, total=None, scales=None, eps=1e-6, group=0):
    r, y = onorm.add_norm(host(x), None if delta is None else host(delta), None if w is None else host(w), eps)
    if total is not None:
        assert (np.abs(host(total) - r) <= (ROUND[total.dtype] * (1 + 2.0 ** -16) + 2.0 ** -24) * np.abs(r)).all()
    if scales is None:
        err = np.abs(host(out) - y)
        assert (err <= (ROUND[out.dtype] * (1 + 2.0 ** -16) + 2.0 ** -19) * np.abs(y)).all(), float((err / (np.abs(y) + 1e-300)).max())
        return
    _, s = onorm.quantise(y, group)
    got, codes = host(scales), host(out)
    assert (np.abs(got - s) <= 2.0 ** -19 * s).all()
    for g, at in enumerate(onorm.groups(y.shape[1], group)):
        q = np.divide(y[:, at], s[:, g:g + 1], out=np.zeros_like(y[:, at]), where=s[:, g:g + 1] > 0)
        err = np.abs(codes[:, at] - q)
        assert (err <= np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10) + 2.0 ** -18 * np.abs(q)).all()
        assert (np.abs(codes[:, at]).max(axis=1) == 448.0 * (s[:, g] > 0)).all()  # the largest is the largest code


SIZES = [(1, 8), (1, 2048), (3, 24), (5, 1800), (2, 16384), (64, 4096), (609, 264), (611, 1000), (1301, 128), (613, 16384)]


@pytest.mark.parametrize("rows,hidden", SIZES)
@pytest.mark.parametrize("xt,dt,wt,ot", [(BF, F, BF, BF), (BF, BF, F, BF), (F, BF, BF, F), (F, F, F, BF), (BF, None, None, F),
                                         (F, None, BF, BF), (BF, F, None, F), (BF, None, BF, BF)])
def test_sums_and_norms(rows, hidden, xt, dt, wt, ot):
    x, delta, w = make(rows, hidden, xt, dt, wt, seed=rows + hidden, pad=16)
    whole, out = blank(rows, hidden, ot, pad=8)
    all_total, total = blank(rows, hidden, xt, pad=40) if dt else (None, None)
    before = x.clone()
    RMSNorm(hidden, w, eps=1e-5).apply(x, out, delta=delta, total=total)
    assert torch.equal(x, before) and untouched(whole, rows, hidden) and (total is None or untouched(all_total, rows, hidden))
    check(x, delta, w, out, total, eps=1e-5)


@pytest.mark.parametrize("rows,hidden", [(1, 8), (1, 4096), (3, 24), (5, 1800), (2, 16384), (611, 1000), (1301, 136), (700, 2048)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("xt,dt", [(BF, F), (F, BF), (BF, None)])
def test_codes_and_scales(rows, hidden, group, xt, dt):
    x, delta, w = make(rows, hidden, xt, dt, BF, seed=rows * 3 + hidden + group)
    norm = RMSNorm(hidden, w, group=group)
    whole, out = blank(rows, hidden, F8, pad=8)
    all_scales, _ = blank(rows, norm.num_scales, F)
    scales = all_scales[:rows]
    total = torch.empty_like(x) if dt else None
    norm.apply(x, out, delta=delta, total=total, scales=scales)
    assert untouched(whole, rows, hidden) and (all_scales[rows:] == GUARD).all()
    check(x, delta, w, out, total, scales, group=group)


@pytest.mark.parametrize("rows", [3, 700])
def test_in_place(rows):
    """total = x, out = delta; then out = x."""
    x, delta, w = make(rows, 1024, BF, BF, F, seed=4)
    x0, delta0 = x.clone(), delta.clone()
    norm = RMSNorm(1024, w)
    norm.apply(x, delta, delta=delta, total=x)
    check(x0, delta0, w, delta, x)
    x, x0 = x0, x0.clone()
    norm.apply(x, x)
    check(x0, None, w, x)
    x, x0 = x0, x0.clone()
    norm.apply(x, x0_out := torch.empty_like(x), delta=delta0, total=delta0)
    check(x0, make(rows, 1024, BF, BF, F, seed=4)[1], w, x0_out, delta0)


def test_the_sum_is_not_rounded_before_the_norm():
    """1 + 2^-10 is not a bf16 number: total has 1, the norm the sum."""
    x = torch.ones(1, 512, dtype=BF, device=DEV)
    delta = torch.full((1, 512), 2.0 ** -10, device=DEV)
    delta[0, 0] = 3.0
    total, out = torch.empty_like(x), torch.empty(1, 512, device=DEV)
    RMSNorm(512, eps=0.0).apply(x, out, delta=delta, total=total)
    assert (total[0, 1:] == 1.0).all()
    check(x, delta, None, out, total, eps=0.0)


def test_rows_that_are_not_finite_and_rows_of_zeros():
    x, _, w = make(6, 512, F, None, F, seed=9)
    x[1], x[2, 40], x[3, 200], x[4] = 0.0, float("nan"), float("inf"), 1e-25
    norm = RMSNorm(512, w, group=128)
    for ot in (F, BF, F8):
        out = torch.empty(6, 512, device=DEV).to(ot)
        scales = torch.empty(6, 4, device=DEV) if ot == F8 else None
        norm.apply(x, out, scales=scales)
        if ot != F8:
            y = host(out)
            assert np.isnan(y[2]).all() and np.isnan(y[3, 200]) and (y[1] == 0).all()
            assert np.isfinite(y[4]).all() and (y[4] != 0).all() and (y[3, :200] == 0).all()
        else:
            y = host(out) * host(scales).repeat(128, axis=1)
            assert np.isnan(y[2]).all() and np.isnan(y[3, 128:256]).all() and (y[1] == 0).all() and np.isfinite(host(scales)[1]).all()
            assert (y[3, :128] == 0).all() and np.isfinite(y[4]).all()
        keep = [0, 5]
        check(x[keep], None, w, out[keep], None, None if scales is None else scales[keep], group=128)


def test_many_rows_and_few_of_them():
    """The same call gives the same bits; a few of its rows alone take another split over threads, within the bounds too."""
    x, delta, w = make(700, 2048, BF, F, BF, seed=2)
    out = torch.empty_like(x)
    norm = RMSNorm(2048, w)
    norm.apply(x, out, delta=delta)
    again = torch.empty_like(x)
    norm.apply(x, again, delta=delta)
    assert torch.equal(out, again)
    part = torch.empty_like(x[5:9])
    norm.apply(x[5:9], part, delta=delta[5:9])
    check(x[5:9], delta[5:9], w, part)


def test_on_another_stream_in_a_graph_and_at_the_same_time():
    x, delta, w = make(300, 2048, BF, F, BF, seed=3)
    norm = RMSNorm(2048, w)
    want, total = torch.empty_like(x), torch.empty_like(x)
    norm.apply(x, want, delta=delta, total=total)
    side = torch.cuda.Stream()
    outs = [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    norm.apply(x, outs[0], delta=delta, stream=side)
    norm.apply(x, outs[1], delta=delta)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm.apply(x, outs[0], delta=delta, total=total)
        norm.apply(total, outs[1])
    for seed in (5, 6):
        x.copy_(make(300, 2048, BF, F, BF, seed=seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(x, delta, w, outs[0], total)
        check(total, None, w, outs[1])


def test_rows_far_apart():
    """Offsets beyond 32 bits: two rows 2^31 + 2^30 elements apart."""
    far = (1 << 31) + (1 << 30)
    space = torch.empty(far + 64, dtype=BF, device=DEV)
    x = space.as_strided((2, 64), (far, 1))
    x.copy_(make(2, 64, BF, None, None, seed=8)[0])
    out = torch.empty(2, 64, dtype=BF, device=DEV)
    RMSNorm(64).apply(x, out)
    check(x, None, None, out)
    RMSNorm(64).apply(out.clone(), x)
    check(out, None, None, x)


def test_refusals():
    x, delta, w = make(4, 64, BF, F, F)
    out = torch.empty_like(x)
    norm = RMSNorm(64, w)
    for args, kw, text in (((x[:, :32], out), {}, "rows, 64"), ((x.half(), out), {}, "x is a"), ((x, out[:2]), {}, "out is"),
                           ((x, out.half()), {}, "out is"), ((x, out), dict(delta=delta[:2]), "delta is"),
                           ((x, out), dict(total=out), "goes with delta"), ((x, out), dict(delta=delta, total=delta), "total is"),
                           ((x, out), dict(scales=torch.empty(4, 1, device=DEV)), "scales go"), ((x, out.to(F8)), {}, "scales go"),
                           ((x, out.to(F8)), dict(scales=torch.empty(4, 2, device=DEV)), "scales is"),
                           ((x.cpu(), out), {}, "GPU"), ((x, out.cpu()), {}, "device"),
                           ((torch.empty(64, 64, dtype=BF, device=DEV).T[:4], out), {}, "contiguous")):
        with pytest.raises(ValueError, match=text):
            norm.apply(*args, **kw)
    for n in (0,):
        norm.apply(x[:n], out[:n], delta=delta[:n], total=x[:n])


def test_rows_that_are_not_contiguous():
    """Broadcast and strided columns, of every tensor."""
    x, out = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV)
    norm = RMSNorm(64)
    for bad in (torch.zeros(4, 1, device=DEV).expand(4, 64), torch.zeros(4, 128, device=DEV)[:, ::2], torch.zeros(64, 4, device=DEV).T):
        for args, kw in (((bad, out), {}), ((x, bad), {}), ((x, out), dict(delta=bad)), ((x, out), dict(delta=x, total=bad))):
            with pytest.raises(ValueError, match="contiguous"):
                norm.apply(*args, **kw)
    with pytest.raises(FtError, match="row stride"):
        norm.apply(x, out, delta=torch.zeros(1, 64, device=DEV).expand(4, 64))  # a row for all: not taken
