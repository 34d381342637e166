"""The workspaces of captured and of simultaneous attention calls (KVPages.attend)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv import DEV, _clean_status, make  # noqa: E402,F401

# divided between many CTAs, so that every call counts parts: token_kernel, chunk_kernel, both
SHAPES = [([1], [20000]), ([300], [3000]), ([300, 1], [900, 9000])]


def cases():
    made = [make(q, n, 2, 8, 128, 64, seed=k + 1) for k, (q, n) in enumerate(SHAPES)]
    want = [c.attend()[0] for c in made]
    torch.cuda.synchronize()
    return made, want


def captured(cs, stream=None, **kw):
    """A graph of one call of each case, and its outputs."""
    outs = [torch.empty(c.T, c.Hq, c.sp.dim, dtype=torch.bfloat16, device=DEV) for c in cs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, **({} if stream is None else {"stream": stream})):
        for c, out in zip(cs, outs):
            c.pages.attend(c.batch, c.q_dev, out, **kw)
    return g, outs


def test_graphs_are_replayed_in_any_order():
    """Warmed up on another stream than they are captured on; the last captured is replayed first."""
    made, want = cases()
    graphs = [captured([c]) for c in made] + [captured(made)]
    expected = [[w] for w in want] + [want]
    for g, outs in graphs:
        for out in outs:
            out.fill_(7.0)
    for k in (3, 2, 1, 0, 2, 3, 0):
        graphs[k][0].replay()
        torch.cuda.synchronize()
        for out, w in zip(graphs[k][1], expected[k]):
            assert torch.equal(out, w)
            out.fill_(7.0)


def test_graphs_of_one_stream_run_at_the_same_time():
    """Replayed on two streams, beside calls on the stream that they were captured on."""
    made, want = cases()
    home, other = torch.cuda.Stream(), torch.cuda.Stream()
    for c in made:
        c.attend(stream=home)
    home.synchronize()
    (ga, a), (gb, b) = captured(made, home), captured(made[::-1], home)
    direct = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for out in a + b + direct:
            out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            ga.replay()
        gb.replay()
        for c, out in zip(made, direct):
            c.pages.attend(c.batch, c.q_dev, out, stream=home)
        torch.cuda.synchronize()
        for out, w in zip(a + b[::-1] + direct, want * 3):
            assert torch.equal(out, w)


def test_a_capture_that_forks():
    """Calls on two streams of one capture have a workspace each."""
    made, want = cases()
    outs = [torch.empty_like(w) for w in want]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        made[0].pages.attend(made[0].batch, made[0].q_dev, outs[0])
        made[1].pages.attend(made[1].batch, made[1].q_dev, outs[1], stream=side)
        made[2].pages.attend(made[2].batch, made[2].q_dev, outs[2])
        main.wait_stream(side)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)


def test_captures_hold_one_workspace_a_stream():
    from expert_cache_host_layer_gb300 import paged_kv
    made, want = cases()
    captured(made[:1])
    held = len(paged_kv._captured), len(paged_kv._workspaces), len(paged_kv._outgrown)
    for _ in range(4):
        g, outs = captured(made)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        del g, outs
    assert held == (len(paged_kv._captured), len(paged_kv._workspaces), len(paged_kv._outgrown))


def test_a_workspace_of_the_callers_own():
    from expert_cache_host_layer_gb300 import FtError, paged_kv
    made, want = cases()
    held = len(paged_kv._captured), len(paged_kv._workspaces)
    for c, w in zip(made, want):
        ws = c.pages.new_workspace(c.batch, c.Hq)
        for _ in range(2):
            out = torch.full_like(w, 7.0)
            c.pages.attend(c.batch, c.q_dev, out, workspace=ws)
            assert torch.equal(out, w)
        g, outs = captured([c], workspace=ws)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], w)
        with pytest.raises(FtError, match="are needed"):
            c.pages.attend(c.batch, c.q_dev, out, workspace=ws[:-256])
        for bad in (ws.view(torch.int8), ws[::2], ws.cpu()):
            with pytest.raises(ValueError, match="workspace"):
                c.pages.attend(c.batch, c.q_dev, out, workspace=bad)
    assert held == (len(paged_kv._captured), len(paged_kv._workspaces))


def test_tensors_of_a_call_on_another_stream_may_be_dropped():
    """The stream is busy when the calls are made; what they read and write is dropped and its memory asked for again."""
    from expert_cache_host_layer_gb300.paged_kv import KVBatch
    c = make([3, 60], [400, 90], 2, 8, 128, 16)
    want, _ = c.attend()
    k_want, v_want = (torch.empty(490, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    start = torch.tensor([0, 400, 490], dtype=torch.int32, device=DEV)
    x = torch.randn(c.T, 2, 128, device=DEV).bfloat16()
    c.pages.read(c.batch, start, k_want, v_want)  # (before the new tokens are written over)
    side = torch.cuda.Stream()
    got, k_out, v_out = torch.empty_like(want), torch.empty_like(k_want), torch.empty_like(v_want)
    torch.cuda.synchronize()
    busy = torch.randn(8192, 8192, device=DEV)
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = (busy @ busy).mul_(1e-4)  # some 100 ms

    def batch():
        return KVBatch(*(t.clone() for t in (c.batch.q_start, c.batch.kv_len, c.batch.block_table)), c.T, 60)

    c.pages.attend(batch(), c.q_dev.clone(), got, stream=side)
    c.pages.read(batch(), start.clone(), k_out, v_out, stream=side)
    c.pages.append(batch(), x.clone(), x.clone(), stream=side)
    grabbed = []
    for like in (c.batch.q_start, c.batch.kv_len, c.batch.block_table, c.q_dev, x) * 20:
        grabbed.append(torch.zeros_like(like))  # on this stream, which does not wait
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(k_out, k_want) and torch.equal(v_out, v_want)
    k_new, v_new = torch.empty_like(k_want), torch.empty_like(v_want)
    c.pages.read(c.batch, start, k_new, v_new)
    assert torch.equal(k_new[397:400], x[:3]) and torch.equal(v_new[-60:], x[3:])


def test_calls_on_another_stream_can_be_captured():
    c = make([3, 60], [400, 90], 2, 8, 128, 16)
    want, _ = c.attend()
    side, out = torch.cuda.Stream(), torch.empty_like(c.attend()[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.pages.attend(c.batch, c.q_dev, out, stream=side)
    for _ in range(2):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
