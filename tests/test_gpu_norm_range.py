"""RMSNorm.apply where the mean square is next to nothing: rows of zeros and of
tiny values, with an eps of zero.

mean r^2 + eps counts as 2^-126 at least, so that its inverse root, 2^63 then, is a
number: y = r w 2^63 for such rows.  Bounds as in test_gpu_norm.py: 2^-19 |y| and an
output's rounding; a mean above 2^-126 whose squares are below it has lost 2^-24 of
itself to their steps of 2^-149 (hidden roundings of half a step each, of a sum of
2^-126 hidden at least), which the bound has room for.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from expert_cache_host_layer_gb300.norm import RMSNorm

DEV = "cuda:0"
BF, F, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ROUND = {BF: 2.0 ** -8, F: 0.0}


def host(t):
    return t.double().cpu().numpy()


def exact(x, w, eps):
    return x * w / np.sqrt(np.maximum((x * x).mean(axis=1, keepdims=True) + eps, 2.0 ** -126))


def rows(hidden, xt):
    """Zeros, one magnitude from row to row down to the least of fp32, and an ordinary row."""
    gen = torch.Generator().manual_seed(hidden)
    x = torch.randn(12, hidden, generator=gen)
    size = [0.0, 1e-17, 1e-18, 2.0 ** -62, 2.0 ** -64, 1e-20, 1e-25, 1e-30, 1e-35, 1e-38, 1e-44, 1.0]
    return (x * torch.tensor(size)[:, None]).to(xt).to(DEV), (1 + 0.3 * torch.randn(hidden, generator=gen)).to(DEV)


@pytest.mark.parametrize("hidden", [8, 512, 2048])
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("ot", [BF, F])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-6])
def test_zeros_and_tiny_rows(hidden, xt, ot, eps):
    x, w = rows(hidden, xt)
    for many in (1, 100):
        out = torch.empty(12 * many, hidden, dtype=ot, device=DEV)
        RMSNorm(hidden, w, eps=eps).apply(x.repeat(many, 1), out)
        y, got = exact(host(x), host(w), float(np.float32(eps))), host(out).reshape(many, 12, hidden)
        assert (got[:, 0] == 0).all()
        # (products r w below 2^-126 are steps of 2^-149, which the inverse root enlarges; bf16's are 2^-133)
        slack = 2.0 ** -149 * np.minimum(2.0 ** 63, (eps or 2.0 ** -126) ** -0.5) + (2.0 ** -134 if ot == BF else 0.0)
        assert (np.abs(got - y) <= (ROUND[ot] * (1 + 2.0 ** -16) + 2.0 ** -19) * np.abs(y) + slack).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("xt", [BF, F])
def test_zeros_and_tiny_rows_in_codes(group, eps, xt):
    """Scales are numbers, a row of zeros has codes of zero, and codes times scales are the norm."""
    x, w = rows(512, xt)
    norm = RMSNorm(512, w, eps=eps, group=group)
    out, scales = torch.empty(12, 512, device=DEV).to(F8), torch.empty(12, norm.num_scales, device=DEV)
    norm.apply(x, out, scales=scales)
    c, s = host(out), host(scales)
    assert np.isfinite(c).all() and np.isfinite(s).all() and (c[0] == 0).all()
    y = exact(host(x), host(w), float(np.float32(eps)))
    wide = 512 // norm.num_scales
    most = np.abs(y).reshape(12, -1, wide).max(axis=2)
    # max |r w| below 2^-100 counts as that
    root = np.sqrt(np.maximum((host(x) ** 2).mean(axis=1, keepdims=True) + float(np.float32(eps)), 2.0 ** -126))
    want = np.maximum(most, 2.0 ** -100 / root) / 448
    assert (np.abs(s - want) <= 2.0 ** -19 * want).all()
    err = np.abs(c * s.repeat(wide, axis=1) - y)
    assert (err <= (2.0 ** -4 + 2.0 ** -17) * np.abs(y) + (2.0 ** -10 + 2.0 ** -27) * want.repeat(wide, axis=1)).all()


def test_a_nan_stays_one():
    for eps in (0.0, 1e-6):
        x, w = rows(512, F)
        x[3, 7], x[11, 100] = float("nan"), float("nan")
        out = torch.empty_like(x)
        RMSNorm(512, w, eps=eps).apply(x, out)
        y = host(out)
        assert np.isnan(y[[3, 11]]).all() and np.isfinite(np.delete(y, [3, 11], axis=0)).all()
