"""CPU checks of the ft_kv calls and their torch wrapper beside tests/test_kv_abi.py."""
import pytest

ft = pytest.importorskip("expert_cache_host_layer_gb300")


def test_a_stream_that_does_not_capture_has_no_number():
    assert ft.ft_stream_capture(0) == 0


def test_a_single_sequences_table_is_a_row_of_consecutive_entries():
    """A column of a wider table as the table of one sequence: its entries lie a row apart."""
    torch = pytest.importorskip("torch")
    from expert_cache_host_layer_gb300.paged_kv import KVBatch
    i32 = torch.int32
    wide = torch.arange(40, dtype=i32).view(5, 8)
    start, n = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    for table in (wide[:, 3:4].T, wide[:1, ::2], wide[0].expand(1, 8)[:, ::3]):
        with pytest.raises(ValueError, match="rows are contiguous"):
            KVBatch(start, n, table, 0, 0)
    # one entry, one row of a wider table, and a row of its own: the row's stride is not used
    for table in (wide[2:3, 4:5], wide[2:3], wide[4:5, 2:6], wide[:, 3:4].T[:, 1:2], wide[0].expand(1, 8),
                  torch.empty_strided((1, 4), (1, 1), dtype=i32)):
        b = KVBatch(start, n, table, 0, 0)
        assert b.c.block_table == table.data_ptr() and b.c.table_stride == table.shape[1]
    two = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    for table in (wide[0].expand(2, 8), wide[0].as_strided((2, 4), (2, 1))):  # rows that overlap
        with pytest.raises(ValueError, match="rows are contiguous"):
            KVBatch(*two, table, 0, 0)
    b = KVBatch(*two, wide[1:3, 7:8], 0, 0)
    assert b.c.table_stride == 8


def attend(out=8192, heads=8, tokens=5, qt=1024, qh=128, ot=1024, oh=128):
    """Refused by the strides, or else by the workspace's size: nothing is launched."""
    p = ft.ft_kv_pages(k=1 << 20, v=1 << 21, k_scale=None, v_scale=None, num_pages=10, num_kv_heads=1, head_dim=128,
                       page_tokens=64, kv_dtype=ft.FT_KV_BF16)
    b = ft.ft_kv_batch(q_start=1 << 20, kv_len=1 << 21, block_table=1 << 22, table_stride=4, num_seqs=3,
                       num_tokens=tokens, max_q_len=2)
    ft.ft_kv_attend(p, b, heads, 4096, qt, qh, out, ot, oh, None, 0.1, 1, 0, 4096, 0)


@pytest.mark.parametrize("kw", [dict(ot=0), dict(oh=0), dict(ot=-1024), dict(oh=-128), dict(qt=0), dict(qh=0),
                                dict(qt=-1024), dict(qh=-128)])
def test_strides_of_queries_and_outputs_are_positive(kw):
    with pytest.raises(ft.FtError, match="strides must be positive") as e:
        attend(**kw)
    assert e.value.status == ft.FT_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(tokens=1, qt=0, ot=0), dict(tokens=1, qt=-8, ot=3), dict(heads=1, qh=0, oh=0),
                                dict(heads=1, tokens=1, qt=1, qh=2, ot=-1, oh=0)])
def test_strides_of_single_entries_are_not_used(kw):
    with pytest.raises(ft.FtError, match="are needed"):
        attend(**kw)


@pytest.mark.parametrize("heads,most,kv_heads", [(129, 1, 1), (258, 40, 2), (128, 1 << 24, 1), (8, 1 << 30, 2)])
def test_no_workspace_for_shapes_that_are_refused(heads, most, kv_heads):
    p = ft.ft_kv_pages(k=1 << 20, v=1 << 21, k_scale=None, v_scale=None, num_pages=10, num_kv_heads=kv_heads, head_dim=128,
                       page_tokens=64, kv_dtype=ft.FT_KV_BF16)
    b = ft.ft_kv_batch(q_start=1 << 20, kv_len=1 << 21, block_table=1 << 22, table_stride=4, num_seqs=3, num_tokens=5,
                       max_q_len=most)
    assert ft.ft_kv_attend_workspace(p, b, heads) == 0
    with pytest.raises(ft.FtError) as e:
        ft.ft_kv_attend(p, b, heads, 4096, 128 * heads, 128, 8192, 128 * heads, 128, None, 0.1, 1, 0, 4096, 1 << 40)
    assert e.value.status == ft.FT_ERR_UNSUPPORTED
    b.max_q_len = 1
    assert (ft.ft_kv_attend_workspace(p, b, 128 * kv_heads) > 0) and ft.ft_kv_attend_workspace(p, b, 0) == 0
