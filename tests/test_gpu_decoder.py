"""The example decoder (examples/decoder.py): key/value cache, attention and
expert cache together, each layer's attention and expert output against the
fp64 oracle.

The oracle takes each layer's own inputs as the GPU had them (bf16 tensors), so
that a bound of one operator is not spent on the layers before it:
attention's is tests/kv_harness.py's, the experts' 2e-2 of the output's RMS.
"""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import ffn as offn  # noqa: E402
from oracle import kv as okv  # noqa: E402
from oracle import routing as orouting  # noqa: E402

U = 2.0 ** -8


def example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import decoder
    finally:
        sys.path.pop(0)
    return decoder


def host(t):
    return t.double().cpu().numpy()


class Check:
    """What each sequence's cache holds after every step, by the oracle."""

    def __init__(self, d):
        self.d, self.kv = d, {}
        self.weights = d.bank.numpy().reshape(d.sh.layers * d.sh.experts, -1)

    def step(self, seqs, counts, seed):
        d, sh = self.d, self.d.sh
        gen = torch.Generator(device=d.dev).manual_seed(seed)
        x = torch.randn((sum(counts), sh.hidden), generator=gen, device=d.dev).bfloat16()
        record = []
        d.step(d.batch(seqs, counts), x, record)
        d.check()
        for l, r in enumerate(record):
            self.layer(l, {n: host(t) for n, t in r.items()}, seqs, counts)

    def layer(self, l, r, seqs, counts):
        sh, at = self.d.sh, 0
        for s, m in zip(seqs, counts):
            new = [r["k"][at:at + m], r["v"][at:at + m]]
            if sh.kv_dtype == example().FT_KV_FP8E4M3:
                new = [okv.dequantise(*okv.quantise(t)) for t in new]
            old = self.kv.get((s, l))
            kv = self.kv[s, l] = new if old is None else [np.concatenate(p) for p in zip(old, new)]
            scale = float(np.float32(sh.head_dim ** -0.5))
            out, _, bulk, reach = okv.attend(r["q"][at:at + m], *kv, scale, window=sh.window)
            d = (sh.head_dim + 16) * 2.0 ** -24 * reach
            bound = U * np.abs(out) + (U + 2 * d + 2.0 ** -12)[..., None] * bulk
            err = np.abs(r["attention"][at:at + m] - out)
            assert (err <= bound).all(), (s, l, float((err / bound).max()))
            at += m
        idx, gates = orouting.route(r["logits"], sh.top_k)
        want = offn.moe_ffn(r["n"], idx, gates, lambda e: offn.dequant_blob(
            self.weights[l * sh.experts + e], sh.hidden, sh.inter, example().FT_W_BF16))
        assert np.abs(r["y"] - want).max() <= 2e-2 * np.sqrt((want ** 2).mean())


@pytest.mark.parametrize("kv", ["FT_KV_BF16", "FT_KV_FP8E4M3"])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts_chunks_and_single_tokens(kv, window):
    ex = example()
    d = ex.Decoder(ex.Shape(layers=2, experts=16, slots=32, num_pages=24, max_tokens=256, window=window,
                            kv_dtype=getattr(ex, kv)))
    c = Check(d)
    c.step(["a"], [130], 1)                     # a prompt
    c.step(["a", "b"], [1, 70], 2)              # another beside a decoding sequence
    c.step(["b", "a", "c"], [33, 1, 5], 3)      # the rest of it, and a short one
    for i in range(3):
        c.step(["a", "b", "c"], [1, 1, 1], 4 + i)
    kept = d.park("b")                          # its pages go back; other sequences move on, and take them
    free = len(d.free)
    c.step(["c"], [90], 8)
    c.step(["a", "c"], [1, 1], 9)
    assert len(d.free) < free
    d.resume("b", kept)
    again = d.park("b")
    for x, y in zip(kept, again):               # what was kept is what the cache holds again
        assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(x, y))
    d.resume("b", again)
    c.step(["a", "b", "c"], [1, 1, 1], 10)
    d.release("a")
    c.step(["b", "c"], [1, 4], 11)
