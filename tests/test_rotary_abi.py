"""CPU checks of the rotary calls' argument validation, the frequencies and the oracle's pins."""
import ctypes
import math

import numpy as np
import pytest

from oracle import rotary as orot
from test_kv_abi import batch, pages

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def rotary(**kw):
    f = dict(turns=1 << 20, rot_dim=64, interleaved=0, scale=1.0)
    f.update(kw)
    return ft.ft_rotary(**f)


def rotate(r=None, T=3, pos=4096, heads=4, dim=64, x=8192, xt=256, xh=64, out=16384, ot=256, oh=64):
    ft.ft_rotate(r or rotary(), ft.ft_rotate_args(pos, x, xt, xh, out, ot, oh, T, heads, dim))


def append(p=None, b=None, r=None, k=4096, kt=256, kh=128, v=8192, vt=256, vh=128, heads=8, q=16384, qt=1024, qh=128, out=32768,
           ot=1024, oh=128):
    ft.ft_kv_append_rotary(p or pages(), b or batch(), r or rotary(),
                           ft.ft_append_args(k, kt, kh, v, vt, vh, q, qt, qh, out, ot, oh, heads))


BAD = [(dict(turns=None), "INVALID_ARG", "turns"), (dict(turns=(1 << 20) + 4), "INVALID_ARG", "turns"),
       (dict(rot_dim=0), "UNSUPPORTED", "rot_dim"), (dict(rot_dim=24), "UNSUPPORTED", "rot_dim"),
       (dict(rot_dim=144), "UNSUPPORTED", "rot_dim"), (dict(scale=float("nan")), "INVALID_ARG", "scale"),
       (dict(scale=float("inf")), "INVALID_ARG", "scale")]


@pytest.mark.parametrize("kw,status,text", BAD)
def test_rotary(kw, status, text):
    for call in (lambda r: rotate(r, dim=128, xt=512, xh=128, ot=512, oh=128), lambda r: append(r=r)):
        with pytest.raises(ft.FtError, match=text) as e:
            call(rotary(**kw))
        assert e.value.status == getattr(ft, "FT_ERR_" + status)


@pytest.mark.parametrize("kw,text", [
    (dict(dim=8), "head_dim"), (dict(dim=72), "head_dim"), (dict(dim=528), "head_dim"), (dict(dim=48), "rot_dim"),
    (dict(heads=0), "num_heads"), (dict(heads=8193), "num_heads"), (dict(T=-1), "num_tokens"), (dict(pos=None), "positions"),
    (dict(x=None), "x is null"), (dict(x=8200), "x must"), (dict(xt=257), "x must"), (dict(xh=4), "x must"),
    (dict(out=None), "out is null"), (dict(ot=0), "positive"), (dict(oh=-64), "positive"), (dict(oh=12), "out must"),
])
def test_rotate(kw, text):
    with pytest.raises(ft.FtError, match=text):
        rotate(**kw)


@pytest.mark.parametrize("kw,text", [
    (dict(p=pages(head_dim=96)), "head_dim"), (dict(b=batch(max_q_len=0)), "max_q_len"), (dict(heads=-1), "num_q_heads"),
    (dict(heads=8193), "num_q_heads"), (dict(k=None), "k is null"), (dict(kt=3), "k must"), (dict(v=8196), "v must"),
    (dict(q=None), "q is null"), (dict(qh=1), "q must"), (dict(out=None), "q_out is null"), (dict(ot=0), "positive"),
    (dict(oh=-128), "positive"),
])
def test_append(kw, text):
    with pytest.raises(ft.FtError, match=text):
        append(**kw)


def test_nothing_to_do_is_not_an_error():
    rotate(T=0, pos=None, x=None, out=None)
    append(b=batch(num_tokens=0, max_q_len=0), k=None, v=None, q=None, out=None)
    assert ctypes.sizeof(ft.ft_rotary) == 24
    lib = ft.library()
    assert lib.ft_rotate(ctypes.addressof(rotary()), None, None) == ft.FT_ERR_INVALID_ARG
    assert lib.ft_kv_append_rotary(ctypes.addressof(pages()), ctypes.addressof(batch()), None, None, None) == ft.FT_ERR_INVALID_ARG


def test_frequencies():
    from expert_cache_host_layer_gb300.rotary import Rotary, frequencies
    assert frequencies(16, 10000.0)[:2] == [1.0, 10000.0 ** -0.125]
    assert np.allclose(frequencies(64, 500.0, "linear", 4.0), 500.0 ** (-np.arange(32) / 32) / 4, rtol=1e-14)
    for d, base, factor, length in ((128, 1e4, 8.0, 4096), (64, 1e6, 32.0, 32768), (32, 150.0, 2.0, 300)):
        got = frequencies(d, base, "yarn", factor, length)
        assert np.allclose(got, orot.yarn(d, base, factor, length), rtol=1e-12)
        assert got[0] == 1.0 and math.isclose(got[-1], base ** (-(d - 2) / d) / factor, rel_tol=1e-12)
    for kw, text in ((dict(scaling="cubic"), "scaling"), (dict(base=0.0), "base"), (dict(base=-2.0), "base"), (dict(scaling="yarn", factor=2.0), "original_length"),
                     (dict(scaling="linear", factor=0.5), "factor")):
        with pytest.raises(ValueError, match=text):
            frequencies(64, **kw)
    for args, kw, text in (((24,), {}, "multiple of 16"), ((0,), {}, "multiple of 16"), ((16,), dict(frequencies=[1.0]), "frequencies"),
                           ((16,), dict(frequencies=[math.inf] * 8), "frequencies"), ((16,), dict(device="cpu"), "GPU")):
        with pytest.raises(ValueError, match=text):
            Rotary(*args, **kw)


def test_oracle_pins():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = [np.pi / 2, np.pi]
    y = orot.rotate(x, [1], quarter)                       # pairs (1, 3), (2, 4): a quarter turn, half a turn
    assert np.allclose(y.ravel(), [-3, -2, 1, -4, 5, 6], atol=1e-15)
    y = orot.rotate(x, [1], quarter, interleaved=True, scale=2.0)   # pairs (1, 2), (3, 4)
    assert np.allclose(y.ravel(), [-4, 2, -6, -8, 5, 6], atol=1e-14)
    assert np.allclose(orot.rotate(orot.rotate(x, [7], quarter), [-7], quarter), x, atol=1e-13)
    assert orot.reach(-x, quarter).ravel().tolist() == [4, 6, 4, 6, 0, 0]


def test_without_a_gpu_calls_report_it():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    for call in (rotate, append, lambda: ft.ft_add_norm(ft.ft_norm(None, 0, 64, 1e-6, 0),
                                                        ft.ft_norm_args(3, 4096, 64, None, 0, None, 0, 8192, 64)),
                 lambda: ft.ft_route(ft.ft_router(0, 1, 1, 1, 1, 1.0, None, 0), ft.ft_route_args(4096, 64, 8192, 12288, 0, 3, 64, 4))):
        with pytest.raises(ft.FtError) as e:
            call()
        assert e.value.status == ft.FT_ERR_CUDA
