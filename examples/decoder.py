"""A decoder served with the framework: attention over the paged key/value
cache, and routed experts through the expert cache, layer after layer.

    python examples/decoder.py [--streams 4] [--prompt 300] [--steps 32] [--kv fp8|bf16]
                               [--rotary half|interleaved|none] [--router softmax|sigmoid]

Random weights (synthetic; no checkpoint): the point is the order of the calls.

    layer:  norm.apply(x, n, delta=y, total=x)        x += y of the layer before, n = the norm of the sum
            q, k, v = n Wqkv                          (library products)
            pages.append(batch, k, v, rotary, q, q)   rotate q and k to their positions, store k and v
            pages.attend(batch, q, a)                 attention over their sequences
            norm.apply(x, n, delta=a Wo, total=x)
            cache.route_classify / fetch_misses / moe_forward   the experts, chosen by the cache's routing rule: y

A step takes any mix of sequences: whole prompts or chunks of them beside
sequences that are one token further.  A sequence that has to give up its pages
is read back in bf16, kept by the host, and appended again later: the scales
are powers of two, so what comes back is what was there.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_cache_host_layer_gb300 import FT_KV_BF16, FT_KV_FP8E4M3, FT_W_BF16, ft_expert_bytes
from expert_cache_host_layer_gb300.norm import RMSNorm
from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
from expert_cache_host_layer_gb300.pipeline import ExpertCache, pinned_bank
from expert_cache_host_layer_gb300.rotary import Rotary
from expert_cache_host_layer_gb300.router import Router


@dataclasses.dataclass(frozen=True)
class Shape:
    layers: int = 4
    experts: int = 32
    top_k: int = 2
    hidden: int = 1024
    inter: int = 512
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    page_tokens: int = 64
    num_pages: int = 256
    max_tokens: int = 2048  # of a step
    slots: int = 64         # of the expert cache: half of the layers' experts
    kv_dtype: int = FT_KV_FP8E4M3
    window: int = 0
    rotary: str = "none"    # or half, interleaved
    router: str = "softmax"  # or sigmoid: with a bias for the choice, in the best two of four groups


class Decoder:
    """The layers' weights, pages and expert cache, and the sequences' page lists."""

    def __init__(self, shape: Shape, seed: int = 0, device: str = "cuda:0"):
        self.sh, self.dev = shape, torch.device(device)
        sh, gen = shape, torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen) * rows ** -0.5).bfloat16().to(self.dev)

        wide = (sh.q_heads + 2 * sh.kv_heads) * sh.head_dim
        self.wqkv = [weight(sh.hidden, wide) for _ in range(sh.layers)]
        self.wo = [weight(sh.q_heads * sh.head_dim, sh.hidden) for _ in range(sh.layers)]
        self.router = [weight(sh.hidden, sh.experts) for _ in range(sh.layers)]
        self.pages = [KVPages.empty(sh.num_pages, sh.kv_heads, sh.page_tokens, sh.head_dim, sh.kv_dtype, self.dev)
                      for _ in range(sh.layers)]
        blobs = sh.layers * sh.experts
        self.bank = pinned_bank(blobs * ft_expert_bytes(sh.hidden, sh.inter, FT_W_BF16))
        w = self.bank.view(torch.bfloat16).view(blobs, -1)
        for b in range(blobs):
            w[b] = (torch.randn(w.shape[1], generator=gen) * sh.hidden ** -0.5).bfloat16()
        self.experts = ExpertCache(sh.layers, sh.experts, sh.top_k, sh.hidden, sh.inter, FT_W_BF16, sh.slots,
                                   sh.max_tokens, self.bank, device=device)
        self.norms = [[RMSNorm(sh.hidden) for _ in range(2)] for _ in range(sh.layers)]  # (a model's have weights)
        self.rotary = None if sh.rotary == "none" else Rotary(sh.head_dim, interleaved=sh.rotary == "interleaved",
                                                              device=self.dev)
        if sh.router == "sigmoid":
            bias = (0.1 * torch.randn(sh.layers, sh.experts, generator=gen)).to(self.dev)
            self.experts.set_router(Router(sh.experts, sh.top_k, score="sigmoid", bias=bias, groups=4, top_groups=2,
                                           group_top=2, scale=2.5))
        self.free = list(range(sh.num_pages))
        self.length: dict = {}  # sequence -> tokens in the cache
        self.table: dict = {}   # sequence -> its pages

    # ---- the sequences' pages ------------------------------------------------
    def batch(self, seqs, counts) -> KVBatch:
        """counts[i] new tokens of seqs[i]: pages for them, and the step's description."""
        for s, m in zip(seqs, counts):
            self.length[s] = self.length.get(s, 0) + m
            own = self.table.setdefault(s, [])
            while len(own) * self.sh.page_tokens < self.length[s]:
                own.append(self.free.pop())
        width = max(len(self.table[s]) for s in seqs)
        table = [self.table[s] + [0] * (width - len(self.table[s])) for s in seqs]
        starts = [0]
        for m in counts:
            starts.append(starts[-1] + m)
        host = [torch.tensor(x, dtype=torch.int32) for x in (starts, [self.length[s] for s in seqs], table)]
        return KVBatch(*(x.to(self.dev) for x in host), num_tokens=starts[-1], max_q_len=max(counts))

    def release(self, s):
        self.free += self.table.pop(s)
        del self.length[s]

    # ---- one step ----------------------------------------------------------
    def step(self, batch: KVBatch, x: torch.Tensor, record: list | None = None) -> torch.Tensor:
        """x: bf16 [num_tokens, hidden], the new tokens' states; returns the last layer's.
        record (tests) receives each layer's intermediate tensors."""
        sh, T = self.sh, batch.num_tokens
        q_wide, k_wide = sh.q_heads * sh.head_dim, sh.kv_heads * sh.head_dim
        a = torch.empty((T, sh.q_heads, sh.head_dim), dtype=torch.bfloat16, device=self.dev)
        n, r = torch.empty_like(x), torch.empty_like(x)  # a norm, and the residual
        y = None
        for l in range(sh.layers):
            before, after = self.norms[l]
            if y is None:
                before.apply(x, n)
            else:
                before.apply(x, n, delta=y, total=r)
                x = r
            qkv = n @ self.wqkv[l]
            q = qkv[:, :q_wide].view(T, sh.q_heads, sh.head_dim)
            k = qkv[:, q_wide:q_wide + k_wide].view(T, sh.kv_heads, sh.head_dim)
            v = qkv[:, q_wide + k_wide:].view(T, sh.kv_heads, sh.head_dim)
            if record is not None:
                record.append({"x": x.clone(), "n1": n.clone(), "q0": q.clone()})
            if self.rotary is None:
                self.pages[l].append(batch, k, v)
            else:
                self.pages[l].append(batch, k, v, rotary=self.rotary, q=q, q_out=q)
            self.pages[l].attend(batch, q, a, window=sh.window)
            o = a.view(T, q_wide) @ self.wo[l]
            after.apply(x, n, delta=o, total=r)
            x = r
            logits = (n @ self.router[l]).float()
            y = torch.empty((T, sh.hidden), dtype=torch.float32, device=self.dev)
            self.experts.route_classify(l, logits)
            self.experts.fetch_misses(l)
            self.experts.moe_forward(l, n, y)
            if record is not None:
                record[-1] |= {"q": q, "k": k, "v": v, "attention": a.clone(), "o": o, "x2": x.clone(), "n": n.clone(),
                               "logits": logits, "y": y.clone()}
        return x + y.bfloat16()

    # ---- a sequence leaves its pages and comes back -------------------------
    def park(self, s) -> list:
        """Sequence s as host tensors (k, v) per layer; its pages are free afterwards."""
        batch, n = self.batch([s], [0]), self.length[s]
        rows = torch.tensor([0, n], dtype=torch.int32, device=self.dev)
        kept = []
        for pages in self.pages:
            kv = [torch.empty((n, self.sh.kv_heads, self.sh.head_dim), dtype=torch.bfloat16, device=self.dev)
                  for _ in range(2)]
            pages.read(batch, rows, *kv)
            kept.append([t.cpu() for t in kv])
        self.release(s)
        return kept

    def resume(self, s, kept: list):
        batch = self.batch([s], [kept[0][0].shape[0]])
        for pages, kv in zip(self.pages, kept):
            pages.append(batch, *(t.to(self.dev) for t in kv))

    def check(self):
        """Raise what the calls met on the device."""
        self.pages[0].check()
        self.experts.synchronize()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--streams", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--kv", choices=("fp8", "bf16"), default="fp8")
    ap.add_argument("--rotary", choices=("half", "interleaved", "none"), default="half")
    ap.add_argument("--router", choices=("softmax", "sigmoid"), default="softmax")
    a = ap.parse_args()
    sh = Shape(kv_dtype=FT_KV_FP8E4M3 if a.kv == "fp8" else FT_KV_BF16, rotary=a.rotary, router=a.router)
    d = Decoder(sh)
    gen = torch.Generator(device=d.dev).manual_seed(1)

    def states(n):  # stands for the embedding of sampled tokens
        return torch.randn((n, sh.hidden), generator=gen, device=d.dev).bfloat16()

    seqs = list(range(a.streams))
    for s in seqs:  # a prompt comes in beside the sequences that decode already
        m = max(1, a.prompt - 37 * s)
        counts = [1] * s + [m]
        d.step(d.batch(seqs[:s + 1], counts), states(sum(counts)))
    kept = d.park(seqs[-1])
    d.resume(seqs[-1], kept)
    d.check()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        x = d.step(d.batch(seqs, [1] * len(seqs)), states(len(seqs)))
    d.check()
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    st = d.experts.stats()
    print(f"{a.streams} streams of up to {max(d.length.values())} tokens, {a.kv} cache: "
          f"{a.streams * a.steps / dt:.0f} tokens/s, {1e3 * dt / a.steps:.2f} ms a step of {sh.layers} layers, "
          f"expert hits {st['hits']} of {st['unique_experts']}, |x| {x.float().norm(dim=1).mean():.1f}")


if __name__ == "__main__":
    main()
