"""CPU checks: which tensors of ft_add_norm may be one another's memory."""
import pytest

ft = pytest.importorskip("expert_cache_host_layer_gb300")
torch = pytest.importorskip("torch")

X, DELTA, TOTAL, OUT = 4096, 1 << 16, 1 << 17, 1 << 18


def call(rows=3, x=X, xs=64, xt=ft.FT_BF16, delta=DELTA, ds=64, dt=ft.FT_BF16, total=TOTAL, ts=64, out=OUT, os=64, ot=ft.FT_BF16,
         scales=None):
    ft.ft_add_norm(ft.ft_norm(None, 0, 64, 1e-6, 0), ft.ft_norm_args(rows, x, xs, delta, ds, total, ts, out, os, scales, xt, dt, ot))


@pytest.mark.parametrize("kw,text", [
    (dict(total=DELTA, xt=ft.FT_F32), "total may be delta"),   # would end beyond a bf16 delta
    (dict(total=DELTA, dt=ft.FT_F32), "total may be delta"),
    (dict(total=DELTA, ts=72), "total may be delta"), (dict(total=X, ts=128), "total may be x"),
    (dict(out=X, xt=ft.FT_F32), "out may be x"), (dict(out=X, ot=ft.FT_F32), "out may be x"), (dict(out=X, os=80), "out may be x"),
    (dict(out=X, ot=ft.FT_FP8E4M3, scales=1 << 19), "out may be x"),
    (dict(out=DELTA, dt=ft.FT_F32), "out may be delta"), (dict(out=DELTA, os=128), "out may be delta"),
    (dict(out=DELTA, rows=1, dt=ft.FT_F32), "out may be delta"),
    (dict(out=TOTAL), "one matrix"), (dict(out=X, total=X), "one matrix"), (dict(out=DELTA, total=DELTA), "one matrix"),
])
def test_refused(kw, text):
    with pytest.raises(ft.FtError, match=text) as e:
        call(**kw)
    assert e.value.status == ft.FT_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(), dict(total=X), dict(total=DELTA), dict(total=X, out=DELTA), dict(total=DELTA, out=X),
                                dict(out=X), dict(out=DELTA), dict(total=None, out=X, delta=None), dict(delta=X, total=X),
                                dict(rows=1, total=X, xs=8, ts=16), dict(rows=1, out=X, xs=8, os=24)])
def test_allowed(kw):
    """As far as the launch, which reports that there is no GPU."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    with pytest.raises(ft.FtError) as e:
        call(**kw)
    assert e.value.status == ft.FT_ERR_CUDA
