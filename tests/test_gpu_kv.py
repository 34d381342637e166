"""GPU parity of the paged key/value cache and its attention with the fp64
oracle (bounds: tests/kv_harness.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import kv as okv  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _clean_status():
    from expert_cache_host_layer_gb300 import ft_kv_status
    yield
    ft_kv_status()


def harness():
    import kv_harness
    return kv_harness


def make(*a, **k):
    h = harness()
    return h.Case(h.Spec(*a, **k))


# ---------------------------------------------------------------- append and read

def held(pages):
    """(codes' values, exponent bytes) or (values, None) of a cache's k and v, on the host."""
    vals = [t.double().cpu().numpy() for t in (pages.k, pages.v)]
    sc = [t.cpu().numpy() for t in (pages.k_scale, pages.v_scale)] if pages.k_scale is not None else [None, None]
    return list(zip(vals, sc))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim,page,heads", [(128, 64, 4), (64, 16, 5), (128, 256, 1), (64, 128, 3)])
@pytest.mark.parametrize("q_len,kv_len", [([1], [1]), ([1], [1001]), ([5, 0, 1, 300], [5, 17, 64, 431]),
                                          ([3, 4], [2, 700]), ([1] * 40, list(range(1, 41)))])
def test_append(fp8, dim, page, heads, q_len, kv_len):
    c = make(q_len, kv_len, kv_heads=heads, dim=dim, page=page, fp8=fp8, poison=False)
    rng = np.random.default_rng(9)
    h = harness()
    x = h.bf16(rng.standard_normal((c.T, 3 * heads, dim)) * np.exp(rng.normal(0, 6, (c.T, 3 * heads, 1))))
    dev = torch.from_numpy(x).bfloat16().to(DEV)
    before = held(c.pages)
    c.pages.append(c.batch, dev[:, heads:2 * heads], dev[:, 2 * heads:])  # views of one wider tensor
    after = held(c.pages)
    for which in range(2):
        want, want_e = before[which]
        for s, (m, n) in enumerate(zip(q_len, kv_len)):
            for i in range(m):
                p = n - m + i
                if p < 0:
                    continue
                at = (c.table[s, p // page], slice(None), p % page)
                new = x[c.q_start[s] + i, heads * (1 + which):heads * (2 + which)]
                if fp8:
                    want[at], want_e[at] = okv.quantise(new)
                else:
                    want[at] = new
        np.testing.assert_array_equal(after[which][0], want)
        if fp8:
            np.testing.assert_array_equal(after[which][1], want_e)


def test_append_extreme_vectors():
    """Zeros, subnormals, the largest values, infinities and NaN."""
    big, tiny = 3.3895313892515355e38, 9.183549615799121e-41
    rows = [np.zeros(64), np.full(64, tiny), np.full(64, -tiny), np.full(64, big), np.linspace(-big, big, 64),
            np.r_[np.inf, np.ones(63)], np.r_[np.ones(63), np.nan], np.r_[1e-30, np.zeros(63)],
            np.r_[448.0, np.full(63, 1.0)], np.r_[450.0, np.full(63, 1.0)], np.r_[-2.0 ** -118, np.zeros(63)]]
    x = harness().bf16(np.array(rows))[:, None, :]
    c = make([len(rows)], [len(rows)], kv_heads=1, group=1, dim=64, page=16, fp8=True, poison=False)
    dev = torch.from_numpy(x).bfloat16().to(DEV)
    c.pages.append(c.batch, dev, dev)
    codes, e = okv.quantise(x)
    for vals, sc in held(c.pages):
        at = c.table[0, 0]
        np.testing.assert_array_equal(vals[at, 0, :len(rows)], codes[:, 0])
        np.testing.assert_array_equal(sc[at, 0, :len(rows)], e[:, 0])
    out = [torch.empty(len(rows), 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    c.pages.read(c.batch, torch.tensor([0, len(rows)], dtype=torch.int32, device=DEV), *out)
    np.testing.assert_array_equal(out[0].double().cpu().numpy()[:, 0], okv.dequantise(codes, e)[:, 0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim,page,heads", [(128, 64, 4), (64, 16, 3), (128, 16, 1)])
@pytest.mark.parametrize("kv_len", [[1], [0, 5, 0], [130, 17, 64, 999], [33] * 20])
def test_read(fp8, dim, page, heads, kv_len):
    c = make([0] * len(kv_len), kv_len, kv_heads=heads, dim=dim, page=page, fp8=fp8)
    room = [n + (s % 3) for s, n in enumerate(kv_len)]  # some sequences leave rows over: those are zeros
    start = np.concatenate([[0], np.cumsum(room)]).astype(np.int32)
    k, v = (torch.full((int(start[-1]), heads, dim), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.pages.read(c.batch, torch.from_numpy(start).to(DEV), k, v)
    for got, which in ((k, 0), (v, 1)):
        want = np.zeros(got.shape)
        for s, n in enumerate(kv_len):
            want[start[s]:start[s] + n] = c.sequence(s)[which]
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)


# ---------------------------------------------------------------- attention

SHAPES = [  # kv_heads, group, dim, page
    (2, 4, 128, 64), (1, 8, 128, 16), (3, 1, 64, 16), (2, 3, 64, 32), (1, 16, 128, 128), (1, 32, 128, 64),
    (5, 5, 128, 256), (8, 2, 64, 128)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kv_heads,group,dim,page", SHAPES)
@pytest.mark.parametrize("kv_len", [[1], [15, 16, 17], [127, 128, 129, 64], [700, 1, 2049]])
def test_single_tokens(fp8, kv_heads, group, dim, page, kv_len):
    c = make([1] * len(kv_len), kv_len, kv_heads, group, dim, page, fp8, sharp=2.0)
    c.check(*c.attend())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kv_heads,group,dim,page", SHAPES[:6])
@pytest.mark.parametrize("q_len,kv_len", [([2], [2]), ([33], [33]), ([130], [400]), ([3, 0, 1, 65], [70, 9, 300, 65])])
def test_chunks(fp8, kv_heads, group, dim, page, q_len, kv_len):
    c = make(q_len, kv_len, kv_heads, group, dim, page, fp8, sharp=2.0)
    c.check(*c.attend())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 17, 128, 500])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1], [1000, 5]), ([300, 1], [777, 600])])
def test_windows(fp8, window, q_len, kv_len):
    c = make(q_len, kv_len, 2, 3, 64, 16, fp8)
    c.check(*c.attend(window=window), window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len,kv_len", [([1, 1], [300, 40]), ([70, 9], [200, 9])])
def test_without_a_causal_mask(fp8, q_len, kv_len):
    c = make(q_len, kv_len, 2, 4, 128, 32, fp8)
    c.check(*c.attend(causal=False), causal=False)


def test_a_long_chunk_on_a_longer_context():
    c = make([517, 1], [4517, 3000], 2, 8, 128, 64, sharp=2.0)
    c.check(*c.attend(), rows=[0, 1, 15, 16, 31, 127, 128, 300, 515, 516])


@pytest.mark.parametrize("fp8", [False, True])
def test_one_long_sequence_split_over_the_card(fp8):
    c = make([1], [70001], 1, 8, 128, 64, fp8, sharp=3.0)
    c.check(*c.attend())


@pytest.mark.parametrize("fp8", [False, True])
def test_a_few_rows_on_a_long_sequence(fp8):
    c = make([5], [40003], 2, 8, 128, 16, fp8, sharp=3.0)
    c.check(*c.attend())


def test_many_short_sequences():
    rng = np.random.default_rng(4)
    n = rng.integers(1, 90, 600).tolist()
    c = make([1] * 600, n, 2, 4, 64, 16)
    c.check(*c.attend(), rows=[0])


def test_many_ragged_chunks():
    rng = np.random.default_rng(5)
    m = rng.integers(0, 60, 70)
    n = (m + rng.integers(0, 200, 70)).tolist()
    c = make(m.tolist(), n, 2, 4, 128, 16, fp8=True)
    c.check(*c.attend(), rows=[0, 7, 33, 59])


@pytest.mark.parametrize("q_len,kv_len", [([1, 1, 1], [0, 5, 0]), ([4, 40], [2, 13]), ([200], [60]), ([1], [0])])
def test_rows_that_see_nothing(q_len, kv_len):
    c = make(q_len, kv_len, 2, 4, 128, 16)
    out, lse = c.attend()
    c.check(out, lse)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_a_batch_without_tokens_writes_nothing():
    c = make([0, 0], [10, 0], 2, 4, 128, 16)
    out, lse = c.attend()
    assert out.numel() == 0 and lse.numel() == 0
    empty = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    c.pages.append(c.batch, empty, empty)


@pytest.mark.parametrize("q_len", [1, 2, 40])
def test_every_score_minus_infinity_is_like_seeing_nothing(q_len):
    c = make([q_len], [50], 1, 4, 64, 16)
    q = torch.ones_like(c.q_dev)
    c.q[:] = 1.0
    for j in range(50):
        c.set_token(0, j, 0, np.full((1, 64), -np.inf))
    out, lse = c.attend(q=q)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("kv_heads,group,q_len,kv_len,at,window", [
    (1, 4, 60, 200, 170, 0), (1, 4, 60, 200, 30, 150), (2, 8, 300, 300, 129, 0), (1, 8, 2, 200, 199, 0),
    (1, 8, 2, 200, 40, 159)])
def test_unseen_tokens_do_not_reach_a_row(value, which, kv_heads, group, q_len, kv_len, at, window):
    """A token that some rows see and others do not: the latter stay finite."""
    c = make([q_len], [kv_len], kv_heads, group, 64, 16)
    bad = np.zeros((kv_heads, 64))
    bad[:, 5] = value
    c.set_token(0, at, which, bad)
    if which == 0:
        c.q[:, :, 5] = np.abs(c.q[:, :, 5]) + 0.5  # an infinite key scores +inf or -inf, the same for every row
    out, lse = c.attend(window=window, q=torch.from_numpy(c.q).bfloat16().to(DEV))
    c.q = harness().bf16(c.q)
    rows = sorted({0, q_len - 1, *range(max(0, at - (kv_len - q_len) - 2), min(q_len, at - (kv_len - q_len) + 3)),
                   *(i for i in range(q_len) if abs(kv_len - q_len + i - window + 1 - at) < 3)})
    c.check(out, lse, window=window, rows=[r for r in rows if 0 <= r < q_len])


def test_a_token_of_nan_in_the_quantised_cache():
    c = make([40], [100], 1, 4, 128, 16, fp8=True)
    x = torch.ones(40, 1, 128, dtype=torch.bfloat16, device=DEV)
    y = x.clone()
    y[20, 0, 3] = float("inf")
    c.pages.append(c.batch, x, y)
    out, _ = c.attend()
    assert torch.isfinite(out[:20]).all() and torch.isnan(out[20:]).all()


def test_strided_queries_and_outputs():
    c = make([3, 50], [80, 51], 2, 4, 128, 16)
    wide = torch.zeros(c.T, 3 * c.Hq, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, c.Hq:2 * c.Hq] = c.q_dev
    heads_first = torch.full((c.Hq, c.T, 136), 7.0, dtype=torch.bfloat16, device=DEV)
    out = heads_first[:, :, :128].transpose(0, 1)
    _, lse = c.attend(q=wide[:, c.Hq:2 * c.Hq], out=out)
    c.check(out, lse)
    assert (heads_first[:, :, 128:] == 7.0).all()


def test_scale_and_no_lse():
    c = make([1, 20], [90, 50], 2, 4, 64, 16)
    c.check(*c.attend(scale=0.5), scale=0.5)
    out, _ = c.attend(scale=0.5)
    again = torch.empty_like(out)
    c.pages.attend(c.batch, c.q_dev, again, scale=0.5)
    assert torch.equal(out, again)


def test_large_scores_do_not_overflow():
    c = make([1, 30], [200, 300], 1, 8, 128, 32, sharp=300.0)
    out, lse = c.attend()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.check(out, lse)


@pytest.mark.parametrize("q_len,kv_len", [([1] * 7, [5000, 3, 900, 77, 12000, 1, 640]), ([300, 1], [2000, 9000])])
def test_results_do_not_vary(q_len, kv_len):
    c = make(q_len, kv_len, 2, 8, 128, 64, fp8=True)
    first = c.attend()
    for _ in range(5):
        again = c.attend()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_another_stream_and_a_graph():
    c = make([1, 40], [500, 90], 2, 4, 128, 16)
    want = c.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.attend(stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out = torch.empty_like(want[0])
    with torch.cuda.stream(side):
        c.pages.attend(c.batch, c.q_dev, out)  # the stream's workspace exists before the capture
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.pages.attend(c.batch, c.q_dev, out)
    # the replay reads the lengths anew: the second sequence loses its last ten tokens
    c.batch.kv_len.copy_(torch.tensor([500, 80], dtype=torch.int32))
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.sp.kv_len[1] = 80
    lse = torch.empty(c.T, c.Hq, dtype=torch.float32, device=DEV)
    again = torch.empty_like(out)
    c.pages.attend(c.batch, c.q_dev, again, lse=lse)
    assert torch.equal(out, again)
    c.check(out, lse)


def test_offsets_past_32_bits():
    """A cache of 2 x 5.4 GB whose sequences sit in its last pages."""
    from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
    pages = KVPages.empty(20500, 8, 128, 128, device=DEV)
    n, D = 300, 128
    table = torch.tensor([[20499, 20470, 20488], [0, 20480, 1]], dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(8)
    kv = [harness().bf16(rng.standard_normal((2 * n, 8, D))) for _ in range(2)]
    dev = [torch.from_numpy(x).bfloat16().to(DEV) for x in kv]
    lens = torch.tensor([n, n], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)
    pages.append(KVBatch(start, lens, table, 2 * n, n), *dev)
    out = [torch.empty_like(d) for d in dev]
    pages.read(KVBatch(start, lens, table, 2 * n, n), start, *out)
    assert torch.equal(out[0], dev[0]) and torch.equal(out[1], dev[1])
    for m in (1, 9):
        q = harness().bf16(rng.standard_normal((2 * m, 8, D)))
        got = torch.empty(2 * m, 8, D, dtype=torch.bfloat16, device=DEV)
        pages.attend(KVBatch(torch.tensor([0, m, 2 * m], dtype=torch.int32, device=DEV), lens, table, 2 * m, m),
                     torch.from_numpy(q).bfloat16().to(DEV), got)
        for s in range(2):
            want, _, bulk, reach = okv.attend(q[s * m:(s + 1) * m], kv[0][s * n:(s + 1) * n], kv[1][s * n:(s + 1) * n],
                                              float(np.float32(D ** -0.5)))
            u = harness().U
            tol = u * np.abs(want) + (u + 2 * (D + 16) * 2.0 ** -24 * reach[..., None] + 2.0 ** -12) * bulk
            assert (np.abs(got[s * m:(s + 1) * m].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("what", ["page", "length", "q_start", "max_q_len"])
def test_bad_device_data_is_reported(what):
    from expert_cache_host_layer_gb300 import FT_ERR_INVALID_ARG, FtError
    from expert_cache_host_layer_gb300.paged_kv import KVBatch
    c = make([1, 30], [40, 50], 2, 4, 128, 16)
    b = c.batch
    q_start, kv_len, table, most = b.q_start.clone(), b.kv_len.clone(), b.block_table.clone(), 30
    if what == "page":
        table[1, 1] = c.pages.num_pages
    elif what == "length":
        kv_len[1] = 10 ** 6
    elif what == "q_start":
        q_start[1] = -4
    else:
        most = 20
    bad = KVBatch(q_start, kv_len, table, c.T, most)
    x = torch.zeros(c.T, 2, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(c.T, c.Hq, 128, dtype=torch.bfloat16, device=DEV)
    calls = [lambda: c.pages.append(bad, x, x), lambda: c.pages.attend(bad, c.q_dev, out)]
    if what in ("page", "length"):
        start = torch.tensor([0, 40, 90], dtype=torch.int32, device=DEV)
        rows = torch.empty(90, 2, 128, dtype=torch.bfloat16, device=DEV)
        calls.append(lambda: c.pages.read(bad, start, rows, rows.clone()))
    for call in calls:
        call()
        with pytest.raises(FtError) as e:
            c.pages.check()
        assert e.value.status == FT_ERR_INVALID_ARG
        c.pages.check()  # reported once


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kv_heads,group,dim,page", [(2, 4, 128, 64), (3, 1, 64, 16), (1, 12, 128, 32), (2, 6, 64, 128)])
def test_long_and_short_sequences_in_one_batch(fp8, kv_heads, group, dim, page):
    """Chunks, single tokens, a few tokens and idle sequences side by side: each
    kernel takes its own, and nobody's rows are left out."""
    c = make([150, 1, 0, 2, 1, 40, 3, 1], [400, 900, 5, 31, 1, 40, 1200, 64], kv_heads, group, dim, page, fp8, sharp=2.0)
    out, lse = c.attend()
    assert not (out == 7.0).all(-1).any()  # every row has been written
    c.check(out, lse)


@pytest.mark.parametrize("q_len,kv_len,at", [(40, 100, 80), (200, 300, 290), (1, 300, 17), (2, 40, 39)])
def test_a_value_of_nan_in_the_quantised_cache(q_len, kv_len, at):
    """Rows that see the token are NaN, with a finite lse; the others do not notice."""
    c = make([q_len], [kv_len], 2, 4, 128, 16, fp8=True)
    clean, lse_clean = c.attend()
    page, slot = int(c.table[0, at // 16]), at % 16
    c.pages.v_scale[page, :, slot] = 255
    out, lse = c.attend()
    sees = max(0, at - (kv_len - q_len))
    assert torch.equal(out[:sees], clean[:sees])
    assert torch.isnan(out[sees:]).all()
    assert torch.equal(lse, lse_clean)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
@pytest.mark.parametrize("q_len", [1, 30])
def test_scales_that_are_not_positive(scale, q_len):
    for fp8 in (False, True):
        c = make([q_len], [70], 2, 4, 64, 16, fp8=fp8)
        c.check(*c.attend(scale=scale), scale=scale)


def test_many_query_heads_to_a_key_head():
    c = make([3, 1], [100, 50], 1, 100, 64, 16)
    c.check(*c.attend())


def test_large_batches_of_single_tokens_with_a_window():
    rng = np.random.default_rng(6)
    n = rng.integers(1, 3000, 200).tolist()
    c = make([1] * 200, n, 1, 8, 128, 16, fp8=True)
    c.check(*c.attend(window=200), window=200)


def test_the_workspace_is_left_as_it_was_found():
    """Counters are zero again after every call: calls of all shapes share a workspace."""
    from expert_cache_host_layer_gb300 import paged_kv
    shapes = [([1], [30000]), ([1] * 9, [700] * 9), ([64], [9000]), ([1, 300], [5000, 400])]
    cases = [make(q, n, 2, 8, 128, 64) for q, n in shapes]
    first = [c.attend()[0] for c in cases]
    for _ in range(3):
        for c, want in zip(reversed(cases), reversed(first)):
            assert torch.equal(c.attend()[0], want)
    torch.cuda.synchronize()
    ws = paged_kv._workspaces[(0, torch.cuda.current_stream().cuda_stream)]
    assert (ws[:640] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim,page,group,q_len,kv_len,window", [
    (128, 64, 4, [1900], [1900], 0), (64, 16, 1, [700, 1, 650], [900, 80, 4000], 500), (128, 128, 8, [130, 1], [20000, 9], 0)])
def test_divided_blocks_give_the_same_every_time(fp8, dim, page, group, q_len, kv_len, window):
    """Row blocks divided between CTAs, joined by whichever kernel comes to it, on a busy and on an idle GPU."""
    from expert_cache_host_layer_gb300 import paged_kv
    c = make(q_len, kv_len, 4, group, dim, page, fp8=fp8)
    first = c.attend(window=window)
    c.check(*first, window=window, rows=[0, 67, -1])
    scratch = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    for k in range(6):
        if k % 2:
            scratch.fill_(k)  # the L2 cache holds something else
        again = c.attend(window=window)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    ws = paged_kv._workspaces[(0, torch.cuda.current_stream().cuda_stream)]
    assert (ws[:640] == 0).all() and (ws[768:768 + 8 * 640] == 0).all()  # both kernels' counters


def test_a_workspace_serves_every_batch_of_its_sizes():
    """On a new stream: a chunk, then the chunk beside a single token."""
    side = torch.cuda.Stream()
    c = make([300], [300], 2, 4, 128, 64)
    d = make([300, 1], [300, 700], 2, 4, 128, 64)
    d.pages._needs = c.pages._needs  # as if both steps were of one layer
    torch.cuda.synchronize()
    for x in (c, d, c):
        got = x.attend(stream=side)
        side.synchronize()
        x.check(*got, rows=[0, 150, -1])


def test_a_captured_call_keeps_its_workspace():
    """A larger call on the stream leaves the workspace of a graph captured before it alone."""
    from expert_cache_host_layer_gb300 import paged_kv
    side = torch.cuda.Stream()
    c, big = make([1], [20000], 2, 4, 128, 64), make([200], [900], 2, 4, 128, 64)
    out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    want = c.attend(stream=side)[0]
    side.synchronize()
    key = (0, side.cuda_stream)
    before = paged_kv._workspaces[key]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.pages.attend(c.batch, c.q_dev, out)
    big.attend(stream=side)
    side.synchronize()
    assert paged_kv._workspaces[key] is not before and any(t is before for t in paged_kv._outgrown)
    out.fill_(7.0)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
