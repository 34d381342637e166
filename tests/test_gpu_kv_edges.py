"""GPU parity of the key/value cache and its attention where NaN, negative
positions, strides or capture could go wrong (oracle: fp64; bounds: tests/kv_harness.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv import DEV, _clean_status, harness, make  # noqa: E402,F401


def place(c, s, j):
    """(page, slot) of token j of sequence s."""
    return int(c.table[s, j // c.sp.page]), j % c.sp.page


def nan_key(c, s, j):
    """Token j's key becomes NaN throughout."""
    page, slot = place(c, s, j)
    if c.sp.fp8:
        c.pages.k_scale[page, :, slot] = 255
    else:
        c.pages.k[page, :, slot] = float("nan")
    c.vals[0][page, :, slot] = np.nan


# ---------------------------------------------------------------- NaN scores

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("q_len,kv_len,at", [(1, 1, 0), (1, 17, 16), (1, 33, 32), (1, 65, 64), (2, 34, 33),
                                             (1, 5000, 4999), (40, 40, 39), (40, 129, 128)])
def test_a_key_of_nan_without_neighbours(fp8, group, q_len, kv_len, at):
    """The only token that a warp has to do with: out and lse of the rows that see it are NaN."""
    c = make([q_len], [kv_len], 2, group, 64, 16, fp8)
    nan_key(c, 0, at)
    out, lse = c.attend()
    assert torch.isnan(lse[-1]).all() and torch.isnan(out[-1]).all()
    c.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group,q_len,kv_len", [(4, 1, 1), (4, 1, 40), (8, 2, 700), (4, 1, 20000), (4, 60, 200)])
def test_a_query_of_nan(fp8, group, q_len, kv_len):
    """One head's query is NaN: its out and lse are, its neighbours' are not."""
    c = make([q_len], [kv_len], 2, group, 128, 16, fp8)
    c.q[-1, 1, 7] = np.nan
    out, lse = c.attend(q=torch.from_numpy(c.q).bfloat16().to(DEV))
    assert torch.isnan(lse[-1, 1]) and torch.isnan(out[-1, 1]).all()
    assert torch.isfinite(lse[-1, 0]) and torch.isfinite(out[-1, 2]).all()
    c.check(out, lse, rows=[0, 1, -1])


# ---------------------------------------------------------------- negative positions

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,kv_len", [([4, 40], [2, 13]), ([200], [60]), ([3], [1]), ([16, 1], [4, 900]),
                                          ([300], [290]), ([2, 2], [0, 2])])
def test_negative_positions_see_nothing_without_the_causal_mask(fp8, q_len, kv_len):
    c = make(q_len, kv_len, 2, 4, 64, 16, fp8)
    out, lse = c.attend(causal=False)
    for s, (m, n) in enumerate(zip(q_len, kv_len)):
        t, none = int(c.q_start[s]), max(0, m - n)
        assert (out[t:t + none] == 0).all() and torch.isneginf(lse[t:t + none]).all()
        if n:
            assert torch.isfinite(lse[t + none:t + m]).all()
    c.check(out, lse, causal=False)


# ---------------------------------------------------------------- codes of NaN

@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads,group,q_len,kv_len,at,window", [
    (2, 4, 60, 200, 170, 0), (2, 4, 60, 200, 30, 150), (2, 8, 300, 300, 129, 0), (1, 8, 2, 200, 199, 0),
    (1, 8, 2, 200, 40, 159), (1, 2, 4, 90, 87, 0), (2, 4, 150, 600, 20, 0), (2, 1, 1500, 1500, 1400, 0)])
def test_a_code_of_nan_reaches_only_rows_that_see_it(which, dim, kv_heads, group, q_len, kv_len, at, window):
    """Codes 0x7f and 0xff in columns 5 and 40 of a token that only some rows see."""
    c = make([q_len], [kv_len], kv_heads, group, dim, 16, fp8=True)
    page, slot = place(c, 0, at)
    t = (c.pages.k, c.pages.v)[which].view(torch.uint8)
    t[page, :, slot, 5], t[page, :, slot, 40] = 0x7f, 0xff
    c.vals[which][page, :, slot, 5] = c.vals[which][page, :, slot, 40] = np.nan
    out, lse = c.attend(window=window)
    first = at - (kv_len - q_len)
    rows = {0, q_len - 1, *range(first - 2, first + 3)}
    if window:
        last = first + window - 1
        rows |= set(range(last - 2, last + 3))
    c.check(out, lse, window=window, rows=sorted(r for r in rows if 0 <= r < q_len))


@pytest.mark.parametrize("group,q_len,kv_len", [(4, 1, 70), (8, 2, 300), (4, 50, 133)])
def test_codes_of_nan_in_places_that_no_sequence_owns(group, q_len, kv_len):
    c = make([q_len, q_len], [kv_len, kv_len + 9], 2, group, 128, 32, fp8=True, poison=False)
    free = torch.from_numpy(~c.owned(c.pages.num_pages)).to(DEV)
    for t in (c.pages.k, c.pages.v):
        t.view(torch.uint8)[free] = 0x7f
    c.check(*c.attend())


# ---------------------------------------------------------------- strides

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,kv_len,group", [([1, 1], [80, 500], 4), ([3, 150], [80, 151], 4), ([70], [333], 1)])
def test_queries_stored_by_head(fp8, q_len, kv_len, group):
    """q's head stride is above its token stride."""
    c = make(q_len, kv_len, 2, group, 128, 16, fp8)
    by_head = torch.full((c.Hq + 1, c.T, 136), 7.0, dtype=torch.bfloat16, device=DEV)
    by_head[1:, :, :128] = c.q_dev.transpose(0, 1)
    c.check(*c.attend(q=by_head[1:, :, :128].transpose(0, 1)))


@pytest.mark.parametrize("fp8", [False, True])
def test_strides_of_single_entries(fp8):
    """One token, one key head: whatever stride a view gives such a dimension, it is not used."""
    c = make([1], [80], 1, 1, 64, 16, fp8)
    out = torch.full((1, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    odd = [t.as_strided((1, 1, 64), (s0, s1, 1)) for t, s0, s1 in ((c.q_dev, 3, 0), (out, 0, 5))]
    _, lse = c.attend(q=odd[0], out=odd[1])
    c.check(out, lse)
    x = c.q_dev.as_strided((1, 1, 64), (1, 3, 1))
    c.pages.append(c.batch, x, x)
    page, slot = place(c, 0, 79)
    if not fp8:
        assert torch.equal(c.pages.k[page, 0, slot], c.q_dev[0, 0]) and torch.equal(c.pages.v[page, 0, slot], c.q_dev[0, 0])
    else:
        from oracle import kv as okv
        codes, e = okv.quantise(c.q[0, 0])
        assert int(c.pages.v_scale[page, 0, slot]) == int(e)
        np.testing.assert_array_equal(c.pages.v[page, 0, slot].double().cpu().numpy(), codes)


# ---------------------------------------------------------------- rows of no sequence

@pytest.mark.parametrize("fp8", [False, True])
def test_append_leaves_rows_before_the_first_sequence_alone(fp8):
    """q_start[0] = 4: rows 0..3 are nobody's, and no token of the cache changes for them."""
    from expert_cache_host_layer_gb300 import FT_ERR_INVALID_ARG, FtError
    from expert_cache_host_layer_gb300.paged_kv import KVBatch
    c = make([6], [40], 2, 4, 64, 16, fp8, poison=False)
    before = [t.clone() for t in (c.pages.k.view(torch.uint8), c.pages.v.view(torch.uint8))]
    b = KVBatch(torch.tensor([4, 6], dtype=torch.int32, device=DEV), c.batch.kv_len, c.batch.block_table, 6, 6)
    x = torch.ones(6, 2, 64, dtype=torch.bfloat16, device=DEV)
    c.pages.append(b, x, x)
    for t, old in zip((c.pages.k, c.pages.v), before):
        page, slot = place(c, 0, 37)  # the last token that is not new
        assert torch.equal(t.view(torch.uint8)[page, :, :slot + 1], old[page, :, :slot + 1])
        assert not torch.equal(t.view(torch.uint8)[page, :, slot + 1], old[page, :, slot + 1])
    with pytest.raises(FtError) as e:
        c.pages.check()
    assert e.value.status == FT_ERR_INVALID_ARG


@pytest.mark.parametrize("q_len,kv_len", [([1, 1], [80, 500]), ([3, 150], [80, 151])])
def test_rows_after_the_last_sequence_are_left_alone(q_len, kv_len):
    """A batch padded to a fixed number of rows, as a captured step has it."""
    from expert_cache_host_layer_gb300.paged_kv import KVBatch
    c = make(q_len, kv_len, 2, 4, 64, 16)
    T = c.T + 5
    b = KVBatch(c.batch.q_start, c.batch.kv_len, c.batch.block_table, T, max(q_len))
    q = torch.ones(T, c.Hq, 64, dtype=torch.bfloat16, device=DEV)
    q[:c.T] = c.q_dev
    out, lse = torch.full_like(q, 7.0), torch.full((T, c.Hq), 7.0, device=DEV)
    c.pages.attend(b, q, out, lse=lse)
    assert (out[c.T:] == 7.0).all() and (lse[c.T:] == 7.0).all()
    c.check(out[:c.T], lse[:c.T], rows=[0, 1, -1])
    before = c.pages.k.clone()
    x = torch.ones(T, 2, 64, dtype=torch.bfloat16, device=DEV)
    c.pages.append(b, x, x)
    changed = (c.pages.k.view(torch.int16) != before.view(torch.int16)).any(-1).any(1)
    assert int(changed.sum()) == c.T


# ---------------------------------------------------------------- rows of a tile that are nobody's

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [-0.2, 0.2])
@pytest.mark.parametrize("group,dim", [(5, 128), (3, 128), (7, 64), (12, 128), (100, 64)])
def test_results_do_not_depend_on_what_ran_before(fp8, scale, group, dim):
    """128 rows of a tile hold 128 / group tokens' heads and some rows more, which
    keep what other calls left there: nobody's result may change by a bit for it."""
    c = make([211], [1417], 3, group, dim, 16, fp8, sharp=0.3)
    others = [make([300], [600], 3, 4, dim, 16, fp8, sharp=s) for s in (30.0, 300.0, 0.01)]
    first = c.attend(scale=scale, causal=False)
    for other in others * 3:
        other.attend(scale=scale)
        again = c.attend(scale=scale, causal=False)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_a_sequence_does_not_notice_the_next_ones_queries(fp8, group):
    """Rows after a sequence's last in its tile are the next one's queries."""
    c = make([70, 200], [900, 300], 2, group, 64, 16, fp8, sharp=0.3)
    first = c.attend()
    for k in (30.0, 300.0, -7.0):
        q = c.q_dev.clone()
        q[70:] *= k
        again = c.attend(q=q)
        assert torch.equal(first[0][:70], again[0][:70]) and torch.equal(first[1][:70], again[1][:70])
