"""Rotary positions (Rotary.rotate, KVPages.append with rotary) against the fp64 oracle.

Error bound (u = 2^-24): a turn's fraction is exact up to 2^-32 turns and the
table's own rounding (a double's), and the rest of at most pi / 4 is a float of
24 bits, so the angle is off by less than u; sine and cosine by 1 ulp, their
product with scale by one rounding more: 3 u |scale| each.  a cos - b sin adds
two roundings:

    |y - exact| <= 5 u |scale| (|a| + |b|)  <=  2^-21 |scale| (|a| + |b|),

and a bf16 result one of 2^-8 |y|.  (At positions near 2^31 the table's rounding,
2^-56 of a turn a position, and that of the oracle's product, 2^-53 of the angle,
add 8 u: 2^-20 in all.)  An e4m3 code adds 2^-4 of the value, or half
a step of 2^-9 times its scale 2^k, the least with max|y| <= 448 2^k up to that
error of max|y|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import kv as okv  # noqa: E402
from oracle import rotary as orot  # noqa: E402

if torch.cuda.is_available():
    import expert_cache_host_layer_gb300 as ft
    from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
    from expert_cache_host_layer_gb300.rotary import Rotary

DEV = "cuda:0"
U = 2.0 ** -8
GUARD = 24.0


def host(t):
    return t.double().cpu().numpy()


def bound(x, y, rot):
    r = orot.reach(x, rot.frequencies, rot.interleaved, rot.scale)
    return U * np.abs(y) + 2.0 ** -20 * r  # (2^-21, and the same rounded to bf16)


def check(x, positions, out, rot):
    y = orot.rotate(host(x), positions, rot.frequencies, rot.interleaved, rot.scale)
    err = np.abs(host(out) - y)
    assert (err <= bound(host(x), y, rot)).all(), float(err.max())


def normal(*shape, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).bfloat16().to(DEV)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


FAR = [0, 1, -1, 7, 4095, 100000, 1 << 20, (1 << 31) - 1, -(1 << 31), -12345]


@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (64, 16), (80, 32), (96, 96), (128, 128), (128, 48), (256, 112), (512, 512)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads", [(1, 1), (10, 3), (61, 17), (1300, 2), (3, 130)])
def test_rotate(dim, rot, interleaved, T, heads):
    r = Rotary(rot, base=1e4, interleaved=interleaved)
    x = normal(T, heads + 2, dim, seed=T + dim)[:, 1:1 + heads]  # a view, as of a projection's output
    pos = np.array((FAR * T)[:T] if T <= 10 else np.random.default_rng(T).integers(-100, 200000, T), dtype=np.int64)
    whole = torch.full((T + 1, heads + 1, dim), GUARD, dtype=torch.bfloat16, device=DEV)
    before = x.clone()
    r.rotate(ints(pos), x, whole[:T, :heads])
    assert torch.equal(x, before)
    check(x, pos, whole[:T, :heads], r)
    assert (whole[T:] == GUARD).all() and (whole[:, heads:] == GUARD).all()
    assert torch.equal(whole[:T, :heads, rot:], x[..., rot:])  # the rest is as it was
    r.rotate(ints(pos), x, x)
    assert torch.equal(x, whole[:T, :heads])


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=8.0, original_length=4096),
                                dict(scaling="yarn", factor=8.0, original_length=4096, scale=0.5),
                                dict(frequencies=[0.0, 3.0, 6.5, -1.0, 1e-7, 0.5, 0.25, 100.0], scale=-2.0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_scaled_and_given_frequencies(kw, interleaved):
    r = Rotary(16 if "frequencies" in kw else 64, base=5e5, interleaved=interleaved, **kw)
    x, pos = normal(40, 3, 64, seed=5), np.arange(40) * 2711
    out = torch.empty_like(x)
    r.rotate(ints(pos), x, out)
    check(x, pos, out, r)


def test_far_positions_keep_their_angles():
    """The slowest and the fastest pairs at the far end of a long context: fp32 angles would be off by 0.06 there."""
    r = Rotary(128, base=1e6)
    pos = np.arange(1048576 - 64, 1048576)
    x = torch.ones(64, 1, 128, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(x)
    r.rotate(ints(pos), x, out)
    check(x, pos, out, r)


def test_back_and_forth():
    """Rotated by p and then by -p: the same values, up to two bf16 roundings."""
    r = Rotary(64, interleaved=True)
    x = normal(50, 4, 64)
    pos = ints(np.arange(50) * 977)
    y, z = torch.empty_like(x), torch.empty_like(x)
    r.rotate(pos, x, y)
    r.rotate(-pos, y, z)
    reach = orot.reach(host(x), r.frequencies, True) + orot.reach(host(y), r.frequencies, True)
    assert (np.abs(host(z) - host(x)) <= (2 * U + 2.0 ** -19) * reach).all()


def test_values_that_are_not_finite():
    x = normal(2, 2, 64)
    x[0, 0, 3], x[1, 1, 40] = float("inf"), float("nan")
    out = torch.empty_like(x)
    r = Rotary(32)
    r.rotate(ints([3, 5]), x, out)
    y = host(out)
    assert not np.isfinite(y[0, 0, [3, 19]]).any() and np.isnan(y[1, 1, 40]) and np.isfinite(np.delete(y[0, 0], [3, 19])).all()
    assert np.isfinite(y[0, 1]).all() and np.isfinite(np.delete(y[1, 1], 40)).all()


# ---------------------------------------------------------------- into the cache

class Step:
    """A batch of new tokens, pages full of a guard value, and a table that has pages for the new tokens."""

    def __init__(self, q_len, kv_len, H=2, Hq=6, D=128, P=64, fp8=False, pad=0, seed=0):
        rng = np.random.default_rng(seed)
        self.q_len, self.kv_len, self.H, self.P, self.D, self.fp8 = q_len, kv_len, H, P, D, fp8
        need = [-(-max(n, 0) // P) for n in kv_len]
        n_pages = sum(need) + 2
        order = rng.permutation(n_pages)
        self.table = np.full((len(q_len), max([1] + need)), -1, dtype=np.int64)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.pages = KVPages.empty(n_pages, H, P, D, ft.FT_KV_FP8E4M3 if fp8 else ft.FT_KV_BF16)
        for t in (self.pages.k, self.pages.v):
            t.copy_(torch.full_like(t, GUARD, dtype=torch.float32).to(t.dtype))
        if fp8:
            self.pages.k_scale.fill_(77)
            self.pages.v_scale.fill_(77)
        self.T = sum(q_len) + pad
        self.starts = np.concatenate([[0], np.cumsum(q_len)])
        self.batch = KVBatch(ints(self.starts), ints(kv_len), ints(self.table), self.T, max(q_len))
        qkv = normal(self.T, Hq + 2 * H, D, seed=seed)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]

    def rows(self):
        """(row of the batch, position, page, slot) of the tokens that have a position; page -1: not stored."""
        for s, (m, n) in enumerate(zip(self.q_len, self.kv_len)):
            for i in range(m):
                p = n - m + i
                yield self.starts[s] + i, p, int(self.table[s, p // self.P]) if p >= 0 else -1, p % self.P

    def check(self, rot, q_out):
        rows = list(self.rows())
        t, pos = [r[0] for r in rows], np.array([r[1] for r in rows])
        if q_out is not None:
            check(self.q[t], pos, q_out[t], rot)
            rest = np.setdiff1d(np.arange(self.T), t)
            assert (q_out[rest] == GUARD).all()
        got = {n: host(getattr(self.pages, n)) for n in ("k", "v")}
        scales = {n: getattr(self.pages, n + "_scale").cpu().numpy() if self.fp8 else None for n in ("k", "v")}
        x = host(self.k)
        y = orot.rotate(x[t], pos, rot.frequencies, rot.interleaved, rot.scale)
        slack = 2.0 ** -21 * orot.reach(x[t], rot.frequencies, rot.interleaved, rot.scale)
        v = host(self.v)
        for i, (row, p, page, slot) in enumerate(rows):
            if page < 0:
                continue
            held = {n: got[n][page, :, slot].copy() for n in got}
            for n in got:
                got[n][page, :, slot] = GUARD
            if not self.fp8:
                assert (np.abs(held["k"] - y[i]) <= U * np.abs(y[i]) + 2 * slack[i]).all()
                assert (held["v"] == v[row]).all()
                continue
            codes, e = okv.quantise(v[row])
            assert (held["v"] == codes).all() and (scales["v"][page, :, slot] == e).all()
            for h in range(self.H):
                k = int(scales["k"][page, h, slot]) - 127
                most, off = np.abs(y[i, h]).max(), slack[i, h].max()
                assert most - off <= 448.0 * 2.0 ** k and (k == -110 or most + off > 448.0 * 2.0 ** (k - 1))
                err = np.abs(held["k"][h] * 2.0 ** k - y[i, h])
                assert (err <= np.maximum(2.0 ** -4 * np.abs(y[i, h]), 2.0 ** (k - 10)) + 1.0625 * slack[i, h]).all()
            scales["k"][page, :, slot] = scales["v"][page, :, slot] = 77
        for n in got:  # nothing else was written
            assert (got[n] == GUARD).all() and (scales[n] is None or (scales[n] == 77).all())

    def append(self, rot, queries=True, **kw):
        out = torch.full_like(self.q, GUARD) if queries else None
        self.pages.append(self.batch, self.k, self.v, rotary=rot, q=self.q if queries else None, q_out=out, **kw)
        self.pages.check()
        return out


BATCHES = [([1], [1]), ([1], [1000]), ([5, 0, 1, 70], [5, 9, 300, 131]), ([33, 1], [33, 64]), ([1] * 40, list(range(1, 41))),
           ([1500], [1700])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,P,H,Hq", [(128, 64, 2, 6), (64, 16, 3, 3), (128, 256, 1, 1), (64, 32, 5, 40)])
@pytest.mark.parametrize("q_len,kv_len", BATCHES)
def test_append(fp8, D, P, H, Hq, q_len, kv_len):
    for rot, interleaved in ((D, False), (D, True), (48, False), (16, True)):
        s = Step(q_len, kv_len, H=H, Hq=Hq, D=D, P=P, fp8=fp8, seed=len(q_len) + D)
        r = Rotary(rot, base=1e4, interleaved=interleaved, scale=1.25)
        s.check(r, s.append(r))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hq,D", [(8, 64, 128), (3, 50, 128), (30, 7, 64), (1, 200, 64)])
def test_more_heads_than_a_block_has_threads_for(fp8, H, Hq, D):
    """Several passes over a block's tokens; queries, keys and values in one warp."""
    for interleaved in (False, True):
        s = Step([40, 1, 9], [64, 200, 9], H=H, Hq=Hq, D=D, P=32, fp8=fp8, pad=3, seed=H)
        r = Rotary(48, base=1e4, interleaved=interleaved)
        s.check(r, s.append(r))


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_no_sequence_negative_positions_and_no_queries(fp8):
    r = Rotary(64)
    s = Step([3, 4], [10, 2], fp8=fp8, pad=5)  # the second's first two are at positions -2 and -1
    s.check(r, s.append(r))
    s = Step([3, 4], [10, 9], fp8=fp8, pad=5, seed=3)
    s.append(r, queries=False)
    s.check(r, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_no_turn_is_the_plain_append(fp8):
    """Frequencies of zero: the cache is bit for bit that of append without rotary, extremes among the values."""
    a, b = Step([70, 3], [90, 3], fp8=fp8), Step([70, 3], [90, 3], fp8=fp8)
    for s in (a, b):
        s.k[0, 0, 0], s.k[1, 0, 1], s.k[2, 1, 2], s.v[3, 1, 3] = float("inf"), 3.0e38, float("nan"), 2.0e38
        s.k[4], s.v[5], s.k[6] = 0.0, 0.0, 1e-38
    r = Rotary(128, frequencies=[0.0] * 64)
    out = a.append(r)
    b.pages.append(b.batch, b.k, b.v)
    for n in ("k", "v") + (("k_scale", "v_scale") if fp8 else ()):
        x, y = getattr(a.pages, n), getattr(b.pages, n)
        x, y = (x.view(torch.int16), y.view(torch.int16)) if x.dtype == torch.bfloat16 else (x.view(torch.uint8), y.view(torch.uint8))
        if n == "k" and not fp8:  # inf and NaN times sine 0 are NaN: the pair's other value too
            x, y = x.clone(), y.clone()
            page, slot = int(a.table[0, 20 // 64]), 20 % 64
            for t, h in ((0, 0), (2, 1)):
                x[page, h, slot + t] = y[page, h, slot + t] = 0
        assert torch.equal(x, y), n
    assert torch.equal(out, a.q)


def test_q_out_may_be_q_and_a_chunk_is_its_tokens():
    r = Rotary(128, base=5e5)
    whole, single = Step([30], [90], fp8=True), Step([30], [90], fp8=True)
    out = whole.append(r)
    q = single.q.clone()
    for i in range(30):
        b = KVBatch(ints([0, 1]), ints([61 + i]), ints(single.table), 1, 1)
        single.pages.append(b, single.k[i:i + 1], single.v[i:i + 1], rotary=r, q=q[i:i + 1], q_out=q[i:i + 1])
    assert torch.equal(out, q)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(whole.pages, n).view(torch.uint8), getattr(single.pages, n).view(torch.uint8))


def test_pages_out_of_range_are_not_written():
    for table, text in (([[0, 9], [1, 2]], "out of range"), ([[0, -1], [1, 2]], "out of range")):
        s = Step([100, 3], [100, 70])
        s.batch = KVBatch(ints(s.starts), ints(s.kv_len), ints(table), s.T, 100)
        with pytest.raises(ft.FtError, match=text):
            s.append(Rotary(64))
    s = Step([1], [1])
    s.append(Rotary(64))  # the word was cleared


def test_on_another_stream_and_in_graphs():
    r = Rotary(128)
    s = Step([40, 1, 1], [64, 200, 7], fp8=True)
    want = s.append(r)
    held = [getattr(s.pages, n).clone() for n in ("k", "k_scale")]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, x = torch.empty_like(want), torch.empty_like(want)
    s.pages.append(s.batch, s.k, s.v, rotary=r, q=s.q, q_out=out, stream=side)
    pos = ints([p for _, p, _, _ in s.rows()])
    r.rotate(pos, s.q, x, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(x, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.pages.append(s.batch, s.k, s.v, rotary=r, q=s.q, q_out=out)
        r.rotate(pos, out, x)
        r.rotate(-pos, x, x)
    s.pages.k_scale.fill_(77)
    out.fill_(GUARD)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(s.pages.k.view(torch.uint8), held[0].view(torch.uint8)) and torch.equal(s.pages.k_scale, held[1])


def test_heads_far_apart():
    """Offsets beyond 32 bits: two tokens 2^31 + 2^30 elements apart."""
    far = (1 << 31) + (1 << 30)
    x = torch.empty(far + 64, dtype=torch.bfloat16, device=DEV).as_strided((2, 1, 64), (far, 64, 1))
    x.copy_(normal(2, 1, 64))
    out = torch.empty(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    r = Rotary(64)
    r.rotate(ints([3, 9]), x, out)
    check(x, [3, 9], out, r)
    r.rotate(ints([3, 9]), x, x)
    assert torch.equal(x, out)


def test_refusals():
    r = Rotary(64)
    x, out, pos = normal(3, 2, 64), normal(3, 2, 64), ints([0, 1, 2])
    for args, text in (((pos, x.float(), out), "x is a"), ((pos, x[0], out), "x is a"), ((pos, x, out[:2]), "out is"),
                       ((pos, x, out.float()), "out is"), ((pos.long(), x, out), "positions"), ((pos[:2], x, out), "positions"),
                       ((pos.cpu(), x, out), "positions"), ((pos, x.cpu(), out), "x is a"),
                       ((pos, normal(3, 64, 64).transpose(1, 2)[:, :2], out), "contiguous")):
        with pytest.raises(ValueError, match=text):
            r.rotate(*args)
    with pytest.raises(ft.FtError, match="rot_dim"):
        r.rotate(pos, normal(3, 2, 32), normal(3, 2, 32))
    r.rotate(pos[:0], x[:0], out[:0])
    s = Step([3], [3])
    for kw, text in ((dict(q=s.q, q_out=s.q.clone()), "go with rotary"), (dict(rotary=r, q=s.q), "goes with q_out"),
                     (dict(rotary=r, q=s.q, q_out=s.q[:, :1]), "q_out is a")):
        with pytest.raises(ValueError, match=text):
            s.pages.append(s.batch, s.k, s.v, **kw)
