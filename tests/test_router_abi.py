"""CPU checks of the routing rule's argument validation, its torch wrapper's, and its oracle's pins."""
import ctypes

import numpy as np
import pytest

from oracle import routing as orouting
from oracle.routing import Rule, route_by

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def route(E=64, k=4, T=3, logits=4096, stride=64, dtype=ft.FT_F32, idx=8192, w=12288, score=ft.FT_SCORE_SIGMOID, groups=4,
          top_groups=2, group_top=2, scale=1.0, bias=16384):
    ft.ft_route(ft.ft_router(score, groups, top_groups, group_top, 1, scale, bias, 0),
                ft.ft_route_args(logits, stride, idx, w, dtype, T, E, k))


@pytest.mark.parametrize("kw,status,text", [
    (dict(E=0), "INVALID_ARG", "num_experts"), (dict(E=1025), "INVALID_ARG", "num_experts"), (dict(k=0), "INVALID_ARG", "top_k"),
    (dict(k=33), "INVALID_ARG", "top_k"), (dict(E=4, k=5, groups=1, top_groups=1), "INVALID_ARG", "top_k"),
    (dict(score=2), "INVALID_ARG", "score"), (dict(groups=0), "INVALID_ARG", "num_groups"),
    (dict(groups=33, E=66), "INVALID_ARG", "num_groups"), (dict(groups=5), "INVALID_ARG", "divisor"),
    (dict(top_groups=0), "INVALID_ARG", "top_groups"), (dict(top_groups=5), "INVALID_ARG", "top_groups"),
    (dict(group_top=0), "INVALID_ARG", "group_top"), (dict(group_top=3), "INVALID_ARG", "group_top"),
    (dict(E=4, k=1), "INVALID_ARG", "group_top"), (dict(k=32, top_groups=1), "INVALID_ARG", "beyond the 16 experts"),
    (dict(E=1017, groups=9), "UNSUPPORTED", "at most 576"), (dict(E=1023, groups=31), "UNSUPPORTED", "at most 992"),
    (dict(scale=float("nan")), "INVALID_ARG", "scale"), (dict(bias=16386), "INVALID_ARG", "bias"),
    (dict(T=-1), "INVALID_ARG", "num_tokens"), (dict(T=(1 << 30) + 1), "INVALID_ARG", "num_tokens"), (dict(dtype=2), "INVALID_ARG", "logits_dtype"), (dict(logits=None), "INVALID_ARG", "null"),
    (dict(idx=None), "INVALID_ARG", "null"), (dict(w=None), "INVALID_ARG", "null"), (dict(logits=4098), "INVALID_ARG", "aligned"),
    (dict(idx=8194), "INVALID_ARG", "aligned"), (dict(stride=63), "INVALID_ARG", "logits_stride"),
])
def test_refusals(kw, status, text):
    with pytest.raises(ft.FtError, match=text) as e:
        route(**kw)
    assert e.value.status == getattr(ft, "FT_ERR_" + status)


def test_nothing_to_do_is_not_an_error():
    route(T=0, logits=None, idx=None, w=None)
    lib = ft.library()
    args = ft.ft_route_args(None, 8, None, None, 0, 0, 8, 2)
    assert lib.ft_route(None, ctypes.addressof(args), None) == ft.FT_ERR_INVALID_ARG
    assert lib.ft_route(ctypes.addressof(ft.ft_router(0, 1, 1, 1, 1, 1.0, None, 0)), None, None) == ft.FT_ERR_INVALID_ARG
    assert lib.ft_cache_set_router(None, None) == ft.FT_ERR_INVALID_ARG
    assert ctypes.sizeof(ft.ft_router) == 40


def test_the_torch_wrapper_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    from expert_cache_host_layer_gb300.router import Router
    with pytest.raises(ValueError, match="score"):
        Router(8, 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        Router(8, 2, bias=torch.zeros(8))  # not on a GPU
    with pytest.raises(ValueError, match="GPU"):
        Router(8, 2).route(torch.zeros(1, 8), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2))


def test_oracle_default_is_the_plain_choice():
    rng = np.random.default_rng(0)
    x = np.round(rng.standard_normal((50, 24)) * 4) / 4
    x[0, :3] = np.nan
    idx, w = route_by(Rule(), x, 5)
    ridx, rw = orouting.route(x, 5)
    assert (idx == ridx).all() and np.allclose(w, rw, rtol=1e-14)


def test_oracle_pins():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))  # softmax 1/8, 2/8, 4/8, 1/8
    idx, w = route_by(Rule(renormalise=False, scale=8.0), x, 3)
    assert idx.tolist() == [[2, 1, 0]] and np.allclose(w, [[4.0, 2.0, 1.0]])
    idx, w = route_by(Rule(bias=np.array([0.5, 0.0, 0.0, 0.25])), x, 2)      # v = 5/8, 2/8, 4/8, 3/8: gates without the bias
    assert idx.tolist() == [[0, 2]] and np.allclose(w, [[0.2, 0.8]])
    x = np.array([[3.0, -9.0, 2.0, 2.0, 1.0, 2.5]])                          # groups of two: best 3, 2, 2.5; sums of s 0.95, 1.76, 1.66
    assert route_by(Rule("sigmoid", groups=3, top_groups=1), x, 2)[0].tolist() == [[0, 1]]
    assert route_by(Rule("sigmoid", groups=3, top_groups=2), x, 3)[0].tolist() == [[0, 5, 4]]
    assert route_by(Rule("sigmoid", groups=3, top_groups=2, group_top=2), x, 3)[0].tolist() == [[5, 2, 3]]
    idx, w = route_by(Rule("sigmoid"), np.full((1, 4), -np.inf), 2)
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
    idx, w = route_by(Rule("sigmoid"), np.array([[0.0, np.inf, np.nan]]), 2)
    assert idx.tolist() == [[1, 0]] and np.allclose(w, [[2 / 3, 1 / 3]])
