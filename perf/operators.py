"""What the paged key/value cache and the attention over it have to do: the
cases, their inputs, each operator's plain form in torch, and the work a pass
cannot do without.

A layer's cache is ``k_pages`` and ``v_pages``, [pages, kv heads, page tokens,
head dim], in bf16 or as e4m3 codes with one power-of-two scale per token and
head (``k_scale``, ``v_scale``: the scale's exponent plus 127).  A batch is
described by ``q_start`` (where each sequence's new tokens begin), ``kv_len``
(its length, the new tokens included) and ``block_table`` (its pages in order).

    append  writes the new tokens' keys and values into their pages
    read    gives the keys and values of whole sequences back, in bf16
    attend  softmax(scale q k^T) v of the new tokens over their sequence

``own`` selects the package's kernels; otherwise ``run`` is the plain form.
"""
import math

import torch

own = False


def listed():
    return [
        # one decode stream: the new token of one layer, the smallest call of all
        _case("append", "append_token_b1_fp8", cache="fp8", seqs=1, new=1, past=(1000, 1000), kv_heads=4),
        # the 16,384-token prompt chunk of the prefill workload
        _case("append", "append_chunk_16384_fp8", cache="fp8", seqs=1, chunks=1, chunk=16384, past=(0, 0), kv_heads=8),
        # prompts of many lengths in one call, an odd number of heads, short pages
        _case("append", "append_ragged_d64_bf16", cache="bf16", seqs=37, chunks=37, chunk=733, past=(0, 900),
              kv_heads=5, dim=64, page=16),
        # long sequences leave the card (swapped out, or moved to another server)
        _case("read", "read_b8_fp8", cache="fp8", seqs=8, new=0, past=(4001, 32768), kv_heads=8),
        # a few short prefixes
        _case("read", "read_short_d64_bf16", cache="bf16", seqs=3, new=0, past=(17, 333), kv_heads=3, dim=64, page=32),
        # one decode stream with a short context: latency
        _case("attend", "attend_token_b1_bf16", cache="bf16", seqs=1, new=1, past=(1020, 1020), q_heads=16, kv_heads=4),
        # eight decode streams, some long, eight query heads to a key head
        _case("attend", "attend_token_b8_fp8", cache="fp8", seqs=8, new=1, past=(2000, 32500), q_heads=32, kv_heads=4),
        # a full decode batch of ordinary lengths
        _case("attend", "attend_token_b64_bf16", cache="bf16", seqs=64, new=1, past=(301, 8000), q_heads=32,
              kv_heads=8),
        # a later chunk of a long prompt
        _case("attend", "attend_chunk_2048_fp8", cache="fp8", seqs=1, chunks=1, chunk=2048, past=(14336, 14336),
              q_heads=16, kv_heads=4),
        # the 16,384-token prompt chunk from its beginning
        _case("attend", "attend_chunk_16384_bf16", cache="bf16", seqs=1, chunks=1, chunk=16384, past=(0, 0),
              q_heads=16, kv_heads=4),
        # prompts of several lengths under a sliding window, one query head to a key head
        _case("attend", "attend_window_d64_bf16", cache="bf16", seqs=5, chunks=5, chunk=1501, past=(0, 2300),
              q_heads=12, kv_heads=12, dim=64, page=16, window=1000),
        # continuous batching: one prompt chunk beside 32 decoding sequences
        _case("attend", "attend_mixed_fp8", cache="fp8", seqs=33, chunks=1, chunk=1000, new=1, past=(199, 6000),
              q_heads=32, kv_heads=8),
    ]


def _case(op, name=None, *, cache, seqs, past, kv_heads, new=1, chunks=0, chunk=0, q_heads=0, dim=128, page=64,
          causal=True, window=0):
    c = {"op": op, "cache": cache, "seqs": seqs, "new": new, "chunks": chunks, "chunk": chunk, "past_min": past[0],
         "past_max": past[1], "q_heads": q_heads or kv_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "causal": causal, "window": window}
    return c if name is None else {"name": name, **c}


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    cache, dim, page = rng.choice(["bf16", "fp8"]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    op = rng.choice(["append", "read", "attend", "attend", "attend", "attend"])
    if op == "append":
        seqs = log(1, 64)
        if rng.random() < 0.4:
            return _case(op, cache=cache, seqs=seqs, past=(1, log(1, 20000)), kv_heads=kv_heads, dim=dim, page=page)
        chunk = log(2, 16384)
        return _case(op, cache=cache, seqs=seqs, chunks=max(1, min(seqs, 16384 // chunk)), chunk=chunk,
                     new=rng.choice([0, 1]), past=(0, log(1, 3000)), kv_heads=kv_heads, dim=dim, page=page)
    if op == "read":
        most = log(20, 100000)
        seqs = log(1, max(1, min(64, 110000 // most)))
        return _case(op, cache=cache, seqs=seqs, new=0, past=(rng.randint(1, most), most), kv_heads=kv_heads, dim=dim,
                     page=page)
    group = rng.choice([1, 2, 3, 4, 6, 8])
    kv_heads = min(kv_heads, 32 // group)
    kind = rng.choice(["token", "token", "chunk", "chunk", "mixed"])
    causal = kind == "token" or rng.random() < 0.9
    window = rng.choice([0, 0, 0, log(64, 4000)]) if causal else 0
    if kind == "token":
        most = log(30, 60000)
        seqs = log(1, max(1, min(64, 260000 // most)))
        return _case(op, cache=cache, seqs=seqs, new=rng.choice([1, 1, 1, 2, 4]), past=(rng.randint(1, most), most),
                     q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page, window=window)
    chunk = log(20, 4000)
    chunks = 1 if kind == "mixed" else log(1, max(1, min(8, 6000 // chunk)))
    most = log(1, 8000)
    seqs = chunks if kind == "chunk" else chunks + log(1, 16)
    return _case(op, cache=cache, seqs=seqs, chunks=chunks, chunk=chunk, past=(rng.randint(0, most), most),
                 q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page, causal=causal, window=window)


# ---------------------------------------------------------------- lengths and work

def _lengths(c):
    """New tokens and length of each sequence: the past lengths spread evenly
    over the logarithm, out of order, the chunks a little different."""
    n, lo, hi = c["seqs"], c["past_min"], c["past_max"]
    q = [max(1, c["chunk"] - (i * c["chunk"]) // (c["chunks"] + 1)) if i < c["chunks"] else c["new"] for i in range(n)]
    at = [(i * 7 + 3) % n / max(1, n - 1) if n % 7 else i / max(1, n - 1) for i in range(n)]
    past = [min(hi, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** t)) - 1) if n > 1 else hi for t in at]
    return q, [p + m for p, m in zip(past, q)]


def _pairs(c):
    """(query, key) pairs of one head that the mask leaves, over the batch."""
    total = 0
    for m, n in zip(*_lengths(c)):
        if not c["causal"]:
            total += m * n
            continue
        first = n - m + 1  # keys the first new token sees without a window; one more for each later one
        w = c["window"] or n
        full = min(m, max(0, w - first))  # new tokens that see fewer than w keys
        total += full * first + full * (full - 1) // 2 + (m - full) * w
    return total


def _seen(c):
    """Keys of one head that some query sees, over the batch."""
    w = c["window"] if c["causal"] and c["window"] else 1 << 60
    return sum(min(n, w + m - 1) for m, n in zip(*_lengths(c)) if m)


def work(c):
    q, kv = _lengths(c)
    row = c["dim"] * 2 if c["cache"] == "bf16" else c["dim"] + 1  # bytes of one token's key (or value) of one head
    wide, h = 2 * c["dim"], c["kv_heads"]
    if c["op"] == "append":
        return {"bytes": sum(q) * h * 2 * (wide + row), "flops": 0}
    if c["op"] == "read":
        return {"bytes": sum(kv) * h * 2 * (wide + row), "flops": 0}
    rows = sum(q) * c["q_heads"]
    return {"bytes": _seen(c) * h * 2 * row + rows * (2 * wide + 4), "flops": _pairs(c) * c["q_heads"] * 4 * c["dim"]}


# ---------------------------------------------------------------- inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    q_len, kv_len = _lengths(c)
    T, S, Hq, H, D, P = sum(q_len), c["seqs"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    need = [-(-n // P) for n in kv_len]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.full((S, max(1, max(need))), -1, dtype=torch.int32)  # -1: no page there yet
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n

    # keys have loud and quiet channels, as trained models' keys do
    loud = torch.exp(0.5 * normal(H, 1, D))
    k_pages, v_pages = normal(pages, H, P, D).mul_(loud), normal(pages, H, P, D)
    k_scale = v_scale = None
    if c["cache"] == "fp8":
        (k_pages, k_scale), (v_pages, v_scale) = _quantise(k_pages), _quantise(v_pages)
    else:
        k_pages, v_pages = k_pages.bfloat16(), v_pages.bfloat16()
    # the new tokens' queries, keys and values side by side, as one projection writes them
    qkv = normal(T, Hq + 2 * H, D).bfloat16()

    def starts(lengths):
        return torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=dev)

    st = {"case": c, "k_pages": k_pages, "v_pages": v_pages, "k_scale": k_scale, "v_scale": v_scale,
          "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:],
          "q_start": starts(q_len), "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev),
          "block_table": table.to(dev), "num_tokens": T, "max_q_len": max(q_len), "max_kv_len": max(kv_len)}
    if c["op"] == "attend":
        st["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    if c["op"] == "read":
        st["kv_start"] = starts(kv_len)
        st["rows"] = sum(kv_len)
        st["k_out"], st["v_out"] = (torch.empty(sum(kv_len), H, D, dtype=torch.bfloat16, device=dev) for _ in "kv")
    if own:  # the two descriptions that a program keeps: the layer's cache, and the step's batch
        from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
        st["pages"] = KVPages(k_pages, v_pages, k_scale, v_scale)
        st["batch"] = KVBatch(st["q_start"], st["kv_len"], st["block_table"], T, st["max_q_len"])
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if c["op"] == "append":
        if own:
            st["pages"].append(st["batch"], st["k"], st["v"])
        else:
            _append(st)
        held = [st["k_pages"], st["v_pages"]]
        return held if c["cache"] == "bf16" else held + [st["k_scale"], st["v_scale"]]
    if c["op"] == "read":
        if own:
            st["pages"].read(st["batch"], st["kv_start"], st["k_out"], st["v_out"])
            return [st["k_out"], st["v_out"]]
        return _read(st)
    if own:
        st["pages"].attend(st["batch"], st["q"], st["out"], lse=st["lse"], causal=c["causal"], window=c["window"])
        return [st["out"], st["lse"]]
    return _attend(st)


def _power(e):
    """2^(e - 127) of exponent bytes, by the bits of a float; 255 is NaN."""
    e = e.to(torch.int32)
    return torch.where(e == 255, float("nan"), (e << 23).view(torch.float32))


def _quantise(x):
    """e4m3 codes and exponent bytes: the smallest power of two s (2^-110 at
    least) with max|x| <= 448 s, and x / s rounded to nearest even."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).clamp(min=-110)  # m 2^e <= 448 2^k = 0.875 2^(9 + k)
    return (x * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _places(st):
    """Sequence of each new token, and its position there."""
    q_start, t = st["q_start"].long(), torch.arange(st["num_tokens"], device=st["q"].device)
    s = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    return s, st["kv_len"].long()[s] - q_start[s + 1] + t


def _append(st):
    P = st["case"]["page"]
    s, pos = _places(st)
    page, slot = st["block_table"].long()[s, pos // P], pos % P
    k, v = st["k"].transpose(0, 1), st["v"].transpose(0, 1)
    if st["k_scale"] is None:
        st["k_pages"].transpose(0, 1)[:, page, slot] = k
        st["v_pages"].transpose(0, 1)[:, page, slot] = v
        return
    for x, pages, scales in ((k, st["k_pages"], st["k_scale"]), (v, st["v_pages"], st["v_scale"])):
        codes, e = _quantise(x)
        pages.view(torch.uint8).transpose(0, 1)[:, page, slot] = codes.view(torch.uint8)
        scales.transpose(0, 1)[:, page, slot] = e


def _values(pages, scales, *at):
    x = pages[at] if scales is None else pages.view(torch.uint8)[at].view(torch.float8_e4m3fn)
    return x.float() if scales is None else x.float() * _power(scales[at]).unsqueeze(-1)


def _read(st):
    P = st["case"]["page"]
    start, r = st["kv_start"].long(), torch.arange(st["rows"], device=st["q"].device)
    s = torch.searchsorted(start[1:].contiguous(), r, right=True)
    pos = r - start[s]
    page, slot = st["block_table"].long()[s, pos // P], pos % P
    h = torch.arange(st["case"]["kv_heads"], device=r.device)
    at = (page[:, None], h[None, :], slot[:, None])
    return [_values(st["k_pages"], st["k_scale"], *at).bfloat16(), _values(st["v_pages"], st["v_scale"], *at).bfloat16()]


def _attend(st):
    """The chunks' sequences, then those of single tokens: each group padded to its own longest."""
    c, n = st["case"], st["case"]["chunks"]
    parts = [_attend_part(st, 0, n), _attend_part(st, n, c["seqs"])]
    return [torch.cat([p[i] for p in parts if p is not None]) for i in range(2)]


def _attend_part(st, s0, s1):
    c = st["case"]
    q_len, kv_lens = (x[s0:s1] for x in _lengths(c))
    t0, T = sum(_lengths(c)[0][:s0]), sum(q_len)
    if T == 0:
        return None
    P, D, H, G = c["page"], c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    used = -(-max(kv_lens) // P)
    table = st["block_table"][s0:s1, :used].long().clamp(min=0)
    S, M, N, dev = s1 - s0, max(q_len), used * P, table.device
    q_start, kv_len = st["q_start"][s0:s1 + 1].long() - t0, st["kv_len"][s0:s1].long()
    # every sequence padded to the longest: queries [S, H, M * G, D], keys and values [S, H, N, D]
    i = torch.arange(M, device=dev)
    q = st["q"][t0:t0 + T][(q_start[:-1, None] + i).clamp(max=T - 1)]
    q = q.float().view(S, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, M * G, D)
    k = _values(st["k_pages"], st["k_scale"], table).transpose(1, 2).reshape(S, H, N, D)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    del k
    j = torch.arange(N, device=dev)
    pos = (kv_len - (q_start[1:] - q_start[:-1]))[:, None] + i  # [S, M]
    hide = (j >= kv_len[:, None])[:, None, :].expand(S, M, N)
    if c["causal"]:
        hide = hide | (j > pos[:, :, None])
        if c["window"]:
            hide = hide | (j <= pos[:, :, None] - c["window"])
    s.view(S, H, M, G, N).masked_fill_(hide[:, None, :, None, :], float("-inf"))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(st["v_pages"], st["v_scale"], table).transpose(1, 2).reshape(S, H, N, D)
    o = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    lse = (total.log() + top).squeeze(-1)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    at = t - q_start[seq]
    out = o.view(S, H, M, G, D)[seq, :, at].reshape(T, H * G, D).bfloat16()
    return [out, lse.view(S, H, M, G)[seq, :, at].reshape(T, H * G)]


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _held(pages, scales, s):
    """The values of pages s in 64 bits: [pages, heads, tokens, dim]."""
    x = pages[s].double()
    return x if scales is None else x * _two(scales[s].long() - 127).unsqueeze(-1)


def _two(n):
    """2^n in 64 bits, exactly, by the bits of a double."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x rounded to a value of 4 significant bits, steps of 2^-9 at least (ties to even)."""
    step = _two(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(x / step) * step


def exact(c, seed):
    st = prepare(c, seed)
    q_len, kv_len = _lengths(c)
    P, D, H, G = c["page"], c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    table = st["block_table"].long()
    if c["op"] == "append":
        out = []
        for x, pages, scales in ((st["k"], st["k_pages"], st["k_scale"]), (st["v"], st["v_pages"], st["v_scale"])):
            x, codes = x.double(), pages.double()
            t0 = 0
            for s, (m, n) in enumerate(zip(q_len, kv_len)):
                pos = torch.arange(n - m, n, device=x.device)
                new = x[t0:t0 + m]
                if scales is not None:
                    part, e = torch.frexp(new.abs().amax(-1) / 448.0)
                    e = torch.where(part > 0.5, e, e - 1).clamp(min=-110)  # the least e with max|x| <= 448 2^e
                    new = _e4m3(new / _two(e).unsqueeze(-1))
                    scales[table[s, pos // P], :, pos % P] = (e + 127).to(torch.uint8)
                codes[table[s, pos // P], :, pos % P] = new
                t0 += m
            out.append(codes)
        return out if c["cache"] == "bf16" else out + [st["k_scale"], st["v_scale"]]
    if c["op"] == "read":
        out = []
        for pages, scales in ((st["k_pages"], st["k_scale"]), (st["v_pages"], st["v_scale"])):
            rows = [_held(pages, scales, table[s, :-(-n // P)]).transpose(1, 2).reshape(-1, H, D)[:n]
                    for s, n in enumerate(kv_len)]
            out.append(torch.cat(rows))
        return out
    out = torch.zeros(st["num_tokens"], c["q_heads"], D, dtype=torch.float64, device=table.device)
    lse = torch.full((st["num_tokens"], c["q_heads"]), -math.inf, dtype=torch.float64, device=table.device)
    t0 = 0
    for s, (m, n) in enumerate(zip(q_len, kv_len)):
        if m and n:
            at = table[s, :-(-n // P)]
            k = _held(st["k_pages"], st["k_scale"], at).transpose(0, 1).reshape(H, -1, D)[:, :n]
            v = _held(st["v_pages"], st["v_scale"], at).transpose(0, 1).reshape(H, -1, D)[:, :n]
            for a in range(0, m, 2048):
                b = min(m, a + 2048)
                pos = torch.arange(n - m + a, n - m + b, device=at.device)[:, None]
                hi = n - m + b if c["causal"] else n
                lo = max(0, n - m + a - c["window"] + 1) if c["causal"] and c["window"] else 0
                j = torch.arange(lo, hi, device=at.device)
                see = torch.ones_like(j > pos)
                if c["causal"]:
                    see = j <= pos
                    if c["window"]:
                        see &= j > pos - c["window"]
                for h in range(c["q_heads"]):
                    z = st["q"][t0 + a:t0 + b, h].double() @ k[h // G, lo:hi].T / math.sqrt(D)
                    z = z.masked_fill(~see, -math.inf)
                    lse[t0 + a:t0 + b, h] = torch.logsumexp(z, -1)
                    out[t0 + a:t0 + b, h] = torch.softmax(z, -1) @ v[h // G, lo:hi]
        t0 += m
    return [out, lse]
