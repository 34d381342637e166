"""CPU checks of ft_add_norm's argument validation, its torch wrapper's, and its oracle's pins."""
import ctypes

import numpy as np
import pytest

from oracle import norm as onorm

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def call(rows=3, x=4096, xs=64, xt=ft.FT_BF16, delta=8192, ds=64, dt=ft.FT_F32, total=12288, ts=64, out=16384, os=64,
         ot=ft.FT_BF16, scales=None, weight=1 << 20, weight_dtype=ft.FT_BF16, hidden=64, eps=1e-6, group=0):
    ft.ft_add_norm(ft.ft_norm(weight, weight_dtype, hidden, eps, group),
                   ft.ft_norm_args(rows, x, xs, delta, ds, total, ts, out, os, scales, xt, dt, ot))


@pytest.mark.parametrize("kw,status,text", [
    (dict(hidden=0), "UNSUPPORTED", "hidden"), (dict(hidden=60), "UNSUPPORTED", "hidden"),
    (dict(hidden=16392), "UNSUPPORTED", "hidden"), (dict(eps=-1.0), "INVALID_ARG", "eps"),
    (dict(eps=float("nan")), "INVALID_ARG", "eps"), (dict(eps=float("inf")), "INVALID_ARG", "eps"),
    (dict(rows=-1), "INVALID_ARG", "num_rows"), (dict(rows=1 << 31), "INVALID_ARG", "num_rows"),
    (dict(weight_dtype=ft.FT_FP8E4M3), "INVALID_ARG", "weight_dtype"), (dict(weight=(1 << 20) + 8), "INVALID_ARG", "weight"),
    (dict(xt=ft.FT_FP8E4M3), "INVALID_ARG", "x_dtype"), (dict(dt=7), "INVALID_ARG", "delta_dtype"),
    (dict(delta=None), "INVALID_ARG", "total goes"), (dict(ot=3), "INVALID_ARG", "out_dtype"),
    (dict(ot=ft.FT_FP8E4M3, group=16), "UNSUPPORTED", "group"), (dict(ot=ft.FT_FP8E4M3), "INVALID_ARG", "scales"),
    (dict(ot=ft.FT_FP8E4M3, scales=4098), "INVALID_ARG", "scales"),
    (dict(x=None), "INVALID_ARG", "x is null"), (dict(x=4104), "INVALID_ARG", "x must be"),
    (dict(xs=68), "INVALID_ARG", "x must be"), (dict(xs=56), "INVALID_ARG", "below hidden"),
    (dict(ds=0), "INVALID_ARG", "delta: row stride"), (dict(total=12290), "INVALID_ARG", "total must be"),
    (dict(ts=65), "INVALID_ARG", "total must be"), (dict(out=None), "INVALID_ARG", "out is null"),
    (dict(os=-64), "INVALID_ARG", "out: row stride"),
])
def test_refusals(kw, status, text):
    with pytest.raises(ft.FtError, match=text) as e:
        call(**kw)
    assert e.value.status == getattr(ft, "FT_ERR_" + status)


def test_nothing_to_do_is_not_an_error():
    call(rows=0, x=None, out=None, total=None, delta=None)
    lib, norm, args = ft.library(), ft.ft_norm(None, 0, 64, 1e-6, 0), ft.ft_norm_args()
    assert lib.ft_add_norm(None, ctypes.addressof(args), None) == ft.FT_ERR_INVALID_ARG
    assert lib.ft_add_norm(ctypes.addressof(norm), None, None) == ft.FT_ERR_INVALID_ARG
    assert ctypes.sizeof(ft.ft_norm) == 24 and ctypes.sizeof(ft.ft_norm_args) == 96


def test_packed_arguments_are_the_structures():
    """What the torch wrappers pack, field by field."""
    from expert_cache_host_layer_gb300 import norm, paged_kv, rotary, router
    for pack, cls in ((norm._pack, ft.ft_norm_args), (rotary._pack, ft.ft_rotate_args), (paged_kv._append_args, ft.ft_append_args),
                      (router._pack, ft.ft_route_args)):
        n = len(cls._fields_)
        raw = pack(*range(1, n + 1))
        assert len(raw) == ctypes.sizeof(cls)
        c = cls.from_buffer_copy(raw)
        assert [getattr(c, f) for f, _ in cls._fields_] == list(range(1, n + 1))


def test_the_torch_wrapper_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    from expert_cache_host_layer_gb300.norm import RMSNorm
    with pytest.raises(ValueError, match="weight"):
        RMSNorm(64, torch.ones(64))  # not on a GPU
    x = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="GPU"):
        RMSNorm(64).apply(x, x)
    assert RMSNorm(1000, group=128).num_scales == 8 and RMSNorm(1000).num_scales == 1


def test_oracle_pins():
    r, y = onorm.add_norm([[1.0, 2.0]], [[2.0, 2.0]], [1.0, 0.5], eps=0.0)  # r = 3, 4: mean square 12.5
    assert r.tolist() == [[3.0, 4.0]]
    assert np.allclose(y, [[3.0 / np.sqrt(12.5), 2.0 / np.sqrt(12.5)]], rtol=1e-15)
    codes, s = onorm.quantise(np.array([[448.0, -1.0, 0.0, 0.0, 0.0, 17.0]]), group=2)
    assert s.tolist() == [[1.0, 0.0, 17.0 / 448.0]] and codes.tolist() == [[448.0, -1.0, 0.0, 0.0, 0.0, 448.0]]
    assert [g.stop - g.start for g in onorm.groups(300, 128)] == [128, 128, 44]
