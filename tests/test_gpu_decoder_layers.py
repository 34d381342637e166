"""The example decoder with rotary positions and a routing rule: norm, append with rotary, attention, norm, routing and
experts one after the other, each against the fp64 oracle on the inputs that the GPU gave it.

The bounds are those of the operators' own tests: 2^-8 |y| + 2^-19 |y| for a norm, 2^-8 |y| + 2^-20 (|a| + |b|) for a
rotation, tests/kv_harness.py's for attention (over the keys and values that the cache holds, read back), 2e-2 of the
RMS for the experts.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import ffn as offn  # noqa: E402
from oracle import kv as okv  # noqa: E402
from oracle import norm as onorm  # noqa: E402
from oracle import rotary as orot  # noqa: E402
from oracle.routing import Rule, route_by  # noqa: E402
from test_gpu_decoder import example, host  # noqa: E402

U = 2.0 ** -8


def norm_is(norm, x, delta, total, out):
    r, y = onorm.add_norm(x, delta, None, norm.eps)
    assert (np.abs(out - y) <= (U + 2.0 ** -18) * np.abs(y)).all()
    if total is not None:
        assert (np.abs(total - r) <= (U + 2.0 ** -18) * np.abs(r)).all()


class Check:
    def __init__(self, d):
        self.d = d
        self.weights = d.bank.numpy().reshape(d.sh.layers * d.sh.experts, -1)

    def step(self, seqs, counts, seed):
        d, sh = self.d, self.d.sh
        gen = torch.Generator(device=d.dev).manual_seed(seed)
        x = torch.randn((sum(counts), sh.hidden), generator=gen, device=d.dev).bfloat16()
        record, batch = [], d.batch(seqs, counts)
        given = x.clone()
        out = d.step(batch, x, record)
        d.check()
        assert torch.equal(x, given)
        lengths = [d.length[s] for s in seqs]
        start = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        pos = np.concatenate([np.arange(n - m, n) for m, n in zip(counts, lengths)])
        rec = [{n: host(t) for n, t in r.items()} for r in record]
        for l, r in enumerate(rec):
            prev = rec[l - 1] if l else None
            norm_is(d.norms[l][0], prev["x2"] if l else host(x), prev["y"] if l else None, r["x"] if l else None, r["n1"])
            norm_is(d.norms[l][1], r["x"], r["o"], r["x2"], r["n"])
            rows = torch.from_numpy(start).to(d.dev)
            kv = [torch.empty((int(start[-1]), sh.kv_heads, sh.head_dim), dtype=torch.bfloat16, device=d.dev) for _ in range(2)]
            d.pages[l].read(batch, rows, *kv)
            self.layer(l, r, counts, lengths, start, pos, *map(host, kv))
        assert (np.abs(host(out) - rec[-1]["x2"] - rec[-1]["y"]) <= 2 * U * (np.abs(rec[-1]["x2"]) + np.abs(rec[-1]["y"]))).all()

    def layer(self, l, r, counts, lengths, start, pos, k_held, v_held):
        d, sh = self.d, self.d.sh
        rot = d.rotary
        k = r["k"]
        if rot is not None:
            q = orot.rotate(r["q0"], pos, rot.frequencies, rot.interleaved)
            assert (np.abs(r["q"] - q) <= U * np.abs(q) + 2.0 ** -20 * orot.reach(r["q0"], rot.frequencies, rot.interleaved)).all()
            k = orot.rotate(k, pos, rot.frequencies, rot.interleaved)
        off = 2.0 ** -20 * np.abs(r["k"]).max() * 2  # of a rotated key, before it is stored
        at = 0
        for s, (m, n) in enumerate(zip(counts, lengths)):
            ks, vs = k_held[start[s]:start[s + 1]], v_held[start[s]:start[s + 1]]
            for held, new in ((ks[n - m:], k[at:at + m]), (vs[n - m:], r["v"][at:at + m])):
                if sh.kv_dtype == example().FT_KV_BF16:
                    assert (np.abs(held - new) <= U * np.abs(new) + off).all()
                else:  # 4 bits of a value, or half a step of the head's scale (2^k < max / 224)
                    step = np.abs(new).max(axis=-1, keepdims=True) / 224 * 2.0 ** -10
                    assert (np.abs(held - new) <= np.maximum(2.0 ** -4 * np.abs(new), step * 1.01) + 1.0625 * off).all()
            scale = float(np.float32(sh.head_dim ** -0.5))
            o, _, bulk, reach = okv.attend(r["q"][at:at + m], ks, vs, scale, window=sh.window)
            dd = (sh.head_dim + 16) * 2.0 ** -24 * reach
            assert (np.abs(r["attention"][at:at + m] - o) <= U * np.abs(o) + (U + 2 * dd + 2.0 ** -12)[..., None] * bulk).all()
            at += m
        if d.experts.router is None:
            rule = Rule()
        else:
            rule = Rule("sigmoid", host(d.experts.router.bias[l]), 4, 2, 2, True, 2.5)
        idx, gates = route_by(rule, r["logits"], sh.top_k)
        want = offn.moe_ffn(r["n"], idx, gates, lambda e: offn.dequant_blob(
            self.weights[l * sh.experts + e], sh.hidden, sh.inter, example().FT_W_BF16))
        assert np.abs(r["y"] - want).max() <= 2e-2 * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("kv", ["FT_KV_BF16", "FT_KV_FP8E4M3"])
@pytest.mark.parametrize("rotary,router,window", [("half", "sigmoid", 0), ("interleaved", "softmax", 50), ("none", "sigmoid", 0)])
def test_layers(kv, rotary, router, window):
    ex = example()
    d = ex.Decoder(ex.Shape(layers=2, experts=16, slots=32, num_pages=24, max_tokens=256, window=window, rotary=rotary,
                            router=router, kv_dtype=getattr(ex, kv)))
    c = Check(d)
    c.step(["a"], [130], 1)                     # a prompt
    c.step(["a", "b"], [1, 70], 2)              # another beside a decoding sequence
    c.step(["b", "a", "c"], [33, 1, 5], 3)
    for i in range(2):
        c.step(["a", "b", "c"], [1, 1, 1], 4 + i)
    if kv == "FT_KV_BF16":                      # rotated keys leave and come back as they are
        kept = d.park("b")
        c.step(["c"], [90], 8)
        d.pages[0].check()
        batch = d.batch(["b"], [kept[0][0].shape[0]])
        for pages, held in zip(d.pages, kept):
            pages.append(batch, *(t.to(d.dev) for t in held))
        c.step(["a", "b", "c"], [1, 1, 1], 9)
    d.experts.close()
