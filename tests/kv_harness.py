"""Batches, caches and the fp64 comparison for the key/value cache tests.

Error bound of one output element (u = 2^-8, bf16's unit roundoff; s the
scores, p the probabilities): the output is rounded once (u |o|), each
probability is rounded to bf16 (u sum p|v|), and each score is a sum of D
products in fp32, off by at most d = (D + 16) 2^-24 max_j scale sum|q k_j|,
which changes the probabilities' ratios by at most 2 d; the fp32 sums and the
exponentials add less than 2^-12.  So

    |out - exact| <= u |o| + (u + 2 d + 2^-12) sum p|v|,
    |lse - exact| <= d + 2^-16 (1 + |lse|).
"""
import dataclasses

import numpy as np
import torch

from oracle import kv as okv

U = 2.0 ** -8


@dataclasses.dataclass
class Spec:
    q_len: list
    kv_len: list
    kv_heads: int = 2
    group: int = 4
    dim: int = 128
    page: int = 64
    fp8: bool = False
    seed: int = 1
    sharp: float = 1.0      # factor on q
    spare_pages: int = 3
    poison: bool = True     # NaN (byte 255) in every place of the cache that no sequence owns


def bf16(x: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().double().numpy()


class Case:
    """Host copies (fp64, bf16-exact) and device tensors of one batch."""

    def __init__(self, sp: Spec, device="cuda:0"):
        from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
        self.sp, self.device = sp, device
        rng = np.random.default_rng(sp.seed)
        S, T, H, D, P = len(sp.q_len), sum(sp.q_len), sp.kv_heads, sp.dim, sp.page
        need = [-(-n // P) for n in sp.kv_len]
        pages = sum(need) + sp.spare_pages
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((S, max([1] + need)), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (pages, H, P, D)
        kv = [rng.standard_normal(shape) for _ in range(2)]
        if sp.fp8:
            codes = [torch.from_numpy(x.astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn) for x in kv]
            exps = [rng.integers(120, 130, shape[:3]).astype(np.uint8) for _ in range(2)]
            if sp.poison:
                for e in exps:
                    e[~self.owned(pages)] = 255
            self.vals = [okv.dequantise(c.double().numpy(), e) for c, e in zip(codes, exps)]
            t = [c.to(device) for c in codes] + [torch.from_numpy(e).to(device) for e in exps]
        else:
            self.vals = [bf16(x) for x in kv]
            if sp.poison:
                for x in self.vals:
                    x[~self.owned(pages)] = np.nan
            t = [torch.from_numpy(x).bfloat16().to(device) for x in self.vals]
        self.pages = KVPages(*t)
        self.q = bf16(rng.standard_normal((T, H * sp.group, D)) * sp.sharp)
        self.q_dev = torch.from_numpy(self.q).bfloat16().to(device)
        self.q_start = np.concatenate([[0], np.cumsum(sp.q_len)]).astype(np.int32)
        dev = [torch.from_numpy(x).to(device) for x in (self.q_start, np.array(sp.kv_len, dtype=np.int32), self.table)]
        self.batch = KVBatch(*dev, T, max(sp.q_len))
        self.T, self.Hq = T, H * sp.group

    def owned(self, pages):
        """[pages, H, P] places that hold a token of some sequence."""
        sp = self.sp
        o = np.zeros((pages, sp.kv_heads, sp.page), dtype=bool)
        for s, n in enumerate(sp.kv_len):
            j = np.arange(n)
            o[self.table[s, j // sp.page], :, j % sp.page] = True
        return o

    def sequence(self, s):
        """k, v [n, H, D] of sequence s, fp64."""
        j = np.arange(self.sp.kv_len[s])
        return [x[self.table[s, j // self.sp.page], :, j % self.sp.page] for x in self.vals]

    def set_token(self, s, j, which, values):
        """Overwrite token j's key (0) or value (1) of sequence s in a bf16 cache."""
        page, slot = int(self.table[s, j // self.sp.page]), j % self.sp.page
        self.vals[which][page, :, slot] = values
        t = (self.pages.k, self.pages.v)[which]
        t[page, :, slot] = torch.as_tensor(values, dtype=torch.float64).to(t.dtype).to(t.device)

    def attend(self, scale=None, causal=True, window=0, out=None, stream=None, q=None):
        out = torch.full((self.T, self.Hq, self.sp.dim), 7.0, dtype=torch.bfloat16,
                         device=self.device) if out is None else out
        lse = torch.full((self.T, self.Hq), 7.0, dtype=torch.float32, device=self.device)
        self.pages.attend(self.batch, self.q_dev if q is None else q, out, lse=lse, scale=scale, causal=causal,
                          window=window, stream=stream)
        return out, lse

    def check(self, out, lse, scale=None, causal=True, window=0, rows=None):
        """Compare with the oracle; rows: only these new tokens of every sequence."""
        sp = self.sp
        scale = 1.0 / np.sqrt(sp.dim) if scale is None else scale
        scale = float(np.float32(scale))
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        worst = 0.0
        for s, (m, n) in enumerate(zip(sp.q_len, sp.kv_len)):
            k, v = self.sequence(s)
            picked = range(m) if rows is None else sorted({i % m for i in rows} if m else ())
            for i in picked:
                t = self.q_start[s] + i
                see = np.flatnonzero(okv.visible(n, m, causal, window)[i]) if n else np.zeros(0, dtype=int)
                o, l, bulk, reach = okv.attend(self.q[t:t + 1], k[see], v[see], scale, causal=False)
                d = (sp.dim + 16) * 2.0 ** -24 * np.where(np.isfinite(reach[0]), reach[0], 0.0)
                tol = U * np.abs(o[0]) + (U + 2 * d[:, None] + 2.0 ** -12) * bulk[0]
                fin = np.isfinite(o[0])
                assert (np.isnan(o[0]) == np.isnan(out[t])).all() and (o[0][~fin & ~np.isnan(o[0])] ==
                                                                      out[t][~fin & ~np.isnan(o[0])]).all(), (s, i)
                err = np.abs(np.where(fin, out[t] - o[0], 0.0))
                assert (err[fin] <= tol[fin] + 1e-30).all(), (s, i, float(err.max()), float(tol[fin].min()))
                worst = max(worst, float((err[fin] / (tol[fin] + 1e-30)).max(initial=0.0)))
                lf = np.isfinite(l[0])
                assert (np.isnan(l[0]) == np.isnan(lse[t])).all() and (l[0][~lf & ~np.isnan(l[0])] ==
                                                                      lse[t][~lf & ~np.isnan(l[0])]).all(), (s, i)
                assert (np.abs(lse[t] - l[0])[lf] <= (d + 2.0 ** -16 * (1 + np.abs(l[0])))[lf]).all(), (s, i)
        return worst
