"""CPU checks: an output of the rotary calls in its input's place."""
import pytest

from test_kv_abi import batch, pages
from test_rotary_abi import rotary

ft = pytest.importorskip("expert_cache_host_layer_gb300")
torch = pytest.importorskip("torch")


def rotate(T=3, heads=4, x=8192, xt=256, xh=64, out=8192, ot=256, oh=64):
    ft.ft_rotate(rotary(), ft.ft_rotate_args(4096, x, xt, xh, out, ot, oh, T, heads, 64))


def append(heads=8, q=16384, qt=1024, qh=128, out=16384, ot=1024, oh=128, tokens=None):
    b = batch() if tokens is None else batch(num_tokens=tokens)
    ft.ft_kv_append_rotary(pages(), b, rotary(), ft.ft_append_args(4096, 256, 128, 8192, 256, 128, q, qt, qh, out, ot, oh, heads))


@pytest.mark.parametrize("call,kw,text", [
    (rotate, dict(ot=512), "out may be"), (rotate, dict(xh=192, xt=64), "out may be"), (rotate, dict(xt=0), "out may be"),
    (rotate, dict(T=1, oh=128), "out may be"), (rotate, dict(heads=1, xt=128), "out may be"),
    (append, dict(ot=2048), "q_out may be"), (append, dict(qh=0), "q_out may be"),
    (append, dict(out=4096), "k or v"), (append, dict(out=8192), "k or v"),
])
def test_refused(call, kw, text):
    with pytest.raises(ft.FtError, match=text) as e:
        call(**kw)
    assert e.value.status == ft.FT_ERR_INVALID_ARG


@pytest.mark.parametrize("call,kw", [(rotate, {}), (rotate, dict(T=1, ot=512)), (rotate, dict(heads=1, oh=128)), (rotate, dict(out=32768, ot=512)),
                                     (append, {}), (append, dict(out=32768, ot=2048)), (append, dict(heads=1, oh=256)),
                                     (append, dict(heads=0, q=None, out=None))])
def test_allowed(call, kw):
    """As far as the launch, which reports that there is no GPU."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    with pytest.raises(ft.FtError) as e:
        call(**kw)
    assert e.value.status == ft.FT_ERR_CUDA
