"""CPU checks of the ft_kv calls' argument validation: every refusal comes
before any CUDA call."""
import ctypes

import pytest

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def pages(**kw):
    f = dict(k=1 << 20, v=1 << 21, k_scale=1 << 22, v_scale=1 << 23, num_pages=10, num_kv_heads=2, head_dim=128,
             page_tokens=64, kv_dtype=ft.FT_KV_FP8E4M3)
    f.update(kw)
    return ft.ft_kv_pages(**f)


def batch(**kw):
    f = dict(q_start=1 << 20, kv_len=1 << 21, block_table=1 << 22, table_stride=4, num_seqs=3, num_tokens=5, max_q_len=2)
    f.update(kw)
    return ft.ft_kv_batch(**f)


def append(p, b, k=4096, kt=256, kh=128):
    ft.ft_kv_append(p, b, k, kt, kh, 8192, 256, 128)


def attend(p, b, heads=8, q=4096, qt=1024, qh=128, scale=0.1, causal=1, window=0, ws=4096, wsb=1 << 40):
    ft.ft_kv_attend(p, b, heads, q, qt, qh, 8192, 1024, 128, None, scale, causal, window, ws, wsb)


@pytest.mark.parametrize("kw,status,text", [
    (dict(kv_dtype=2), "INVALID_ARG", "kv_dtype"), (dict(head_dim=96), "UNSUPPORTED", "head_dim"),
    (dict(page_tokens=48), "UNSUPPORTED", "page_tokens"), (dict(page_tokens=8), "UNSUPPORTED", "page_tokens"),
    (dict(num_kv_heads=0), "INVALID_ARG", "num_kv_heads"), (dict(num_pages=0), "INVALID_ARG", "num_pages"),
    (dict(num_pages=1 << 24), "INVALID_ARG", "num_pages"), (dict(k=None), "INVALID_ARG", "null page"),
    (dict(v_scale=None), "INVALID_ARG", "null page"), (dict(v=(1 << 21) + 8), "INVALID_ARG", "16-byte"),
])
def test_pages(kw, status, text):
    for call in (append, attend, lambda p, b: ft.ft_kv_read(p, b, 4096, 9, 4096, 8192)):
        with pytest.raises(ft.FtError, match=text) as e:
            call(pages(**kw), batch())
        assert e.value.status == getattr(ft, "FT_ERR_" + status)
    assert ft.ft_kv_attend_workspace(pages(**kw), batch(), 8) == 0


@pytest.mark.parametrize("kw,text", [
    (dict(num_seqs=-1), "num_seqs"), (dict(num_seqs=5000), "num_seqs"), (dict(num_tokens=-1), "num_tokens"),
    (dict(num_seqs=0), "num_tokens"), (dict(max_q_len=0), "max_q_len"), (dict(table_stride=0), "table_stride"),
    (dict(table_stride=1 << 26), "table_stride"), (dict(kv_len=None), "null batch"),
])
def test_batch(kw, text):
    for call in (append, attend):
        with pytest.raises(ft.FtError, match=text):
            call(pages(), batch(**kw))


@pytest.mark.parametrize("call,kw,text", [
    (append, dict(k=4100), "k must be"), (append, dict(kt=257), "k must be"), (append, dict(kh=4), "k must be"),
    (append, dict(k=None), "k is null"), (attend, dict(q=4098), "q must be"), (attend, dict(q=None), "q is null"),
    (attend, dict(heads=7), "num_q_heads"), (attend, dict(heads=0), "num_q_heads"), (attend, dict(window=-1), "window"),
    (attend, dict(window=8, causal=0), "window"), (attend, dict(scale=float("nan")), "scale"),
    (attend, dict(ws=None), "workspace"), (attend, dict(ws=4100), "workspace"), (attend, dict(wsb=0), "workspace"),
])
def test_calls(call, kw, text):
    with pytest.raises(ft.FtError, match=text) as e:
        call(pages(), batch(), **kw)
    assert e.value.status == ft.FT_ERR_INVALID_ARG


def test_nothing_to_do_is_not_an_error():
    b = batch(num_tokens=0, max_q_len=0)
    append(pages(), b)
    attend(pages(), b)
    ft.ft_kv_read(pages(), b, 0, 0, 0, 0)
    none = batch(num_seqs=0, num_tokens=0, max_q_len=0, q_start=None, kv_len=None, block_table=None)
    append(pages(), none)
    attend(pages(), none)


def test_read_refusals():
    for args, text in (((None, 4, 4096, 8192), "kv_start"), ((4096, -1, 4096, 8192), "num_rows"),
                       ((4096, 1 << 31, 4096, 8192), "num_rows"), ((4096, 4, 4104, 8192), "k_out"),
                       ((4096, 4, 4096, None), "v_out")):
        with pytest.raises(ft.FtError, match=text):
            ft.ft_kv_read(pages(), batch(), *args)


def test_the_torch_wrapper_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
    i32 = torch.int32
    with pytest.raises(ValueError, match="int32"):
        KVBatch(torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32), 2, 1)
    with pytest.raises(ValueError, match="shapes"):
        KVBatch(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32), 2, 1)
    with pytest.raises(ValueError, match="rows are contiguous"):
        KVBatch(torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(4, 2, dtype=i32).T, 2, 1)
    b = KVBatch(torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 8, dtype=i32)[:, :4], 2, 1)
    assert b.c.table_stride == 8 and b.c.num_seqs == 2
    x = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one GPU"):
        KVPages(x, x.clone())
    with pytest.raises(ValueError, match="scales"):
        KVPages(x.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="bf16 or float8"):
        KVPages(x.float(), x.float())
    assert ctypes.sizeof(ft.ft_kv_pages) == 56 and ctypes.sizeof(ft.ft_kv_batch) == 48


def test_attend_refuses_what_its_kernels_do_not_take():
    with pytest.raises(ft.FtError, match="above 128") as e:
        attend(pages(num_kv_heads=1), batch(), heads=129)
    assert e.value.status == ft.FT_ERR_UNSUPPORTED
    with pytest.raises(ft.FtError, match="positive"):
        attend(pages(), batch(), qt=0)
    with pytest.raises(ft.FtError, match="scales are not"):
        attend(pages(k_scale=(1 << 22) + 8), batch())
