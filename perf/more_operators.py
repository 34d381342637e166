"""What a decoder's layer does between its products, its attention and its
experts: the cases, their inputs, each operator's plain form in torch, and the
work a pass cannot do without.

    norm           the residual's addition and the root-mean-square norm of the sum,
                   in bf16, or in e4m3 with a scale per row or per group of channels
    rotate         rotary positions of queries or keys
    rotary_append  the new tokens' queries rotated, their keys rotated and stored in the
                   paged cache (bf16, or e4m3 with power-of-two scales), their values stored
    route          experts and gates of each token: softmax or sigmoid scores, a bias for
                   the choice, groups, top-k, renormalised and scaled weights

``own`` selects the package's kernels; otherwise ``run`` is the plain form.
"""
import math

import torch

own = False

_FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"": 0, "bf16": 2, "f32": 4, "fp8": 1}


def listed():
    return [
        # one decode stream: the experts' output joins the residual before the next layer's attention
        _norm("norm_token_b1", rows=1, hidden=2048, delta="f32"),
        # a decode batch whose next product takes e4m3 rows
        _norm("norm_b64_fp8", rows=64, hidden=4096, delta="bf16", out="fp8"),
        # the 16,384-token prompt chunk of the prefill workload, after its experts
        _norm("norm_chunk_16384", rows=16384, hidden=2048, delta="f32"),
        # an odd number of tokens and channels, an fp32 residual, e4m3 by groups of 128
        _norm("norm_ragged_fp8_groups", rows=4099, hidden=1800, x="f32", delta="bf16", out="fp8", group=128),
        # queries and keys of a decode batch at far positions: interleaved pairs, half of each head
        _rotate("rotate_b32_interleaved", tokens=32, heads=20, dim=128, rot=64, interleaved=True, most=500000),
        # a long chunk with an odd number of tokens, a third of each head, positions stretched by four
        _rotate("rotate_chunk_8191", tokens=8191, heads=24, dim=96, rot=32, scaling="linear", factor=4.0, most=120000),
        # one decode stream's new token: the smallest call
        _append("rotary_append_token_b1_fp8", cache="fp8", seqs=1, new=1, past=1000, q_heads=16, kv_heads=4),
        # a full decode batch, contexts longer than the model was first trained on
        _append("rotary_append_b64_bf16", cache="bf16", seqs=64, new=1, past=100000, q_heads=32, kv_heads=8,
                scaling="yarn", factor=32.0),
        # the 16,384-token prompt chunk
        _append("rotary_append_chunk_16384_fp8", cache="fp8", seqs=1, new=16384, past=0, q_heads=16, kv_heads=4),
        # one decode stream's token over 256 experts, sigmoid scores, a bias, the best 4 of 8 groups
        _route("route_token_b1_groups", tokens=1, experts=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
               group_top=2, scale=2.5),
        # the 16,384-token prompt chunk over the same experts
        _route("route_chunk_16384_groups", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
               top_groups=4, group_top=2, scale=2.5),
        # an odd number of tokens and few experts: plain softmax gates from bf16 logits
        _route("route_ragged_1237_bf16", tokens=1237, experts=72, top_k=6, logits="bf16", renormalise=False),
    ]


def _case(op, name, **kw):
    return {"name": name, "op": op, **kw} if name else {"op": op, **kw}


def _norm(name=None, *, rows, hidden, x="bf16", delta="", out="bf16", group=0, weight="bf16", eps=1e-6):
    return _case("norm", name, rows=rows, hidden=hidden, x=x, delta=delta, out=out, group=group, weight=weight, eps=eps)


def _rotate(name=None, *, tokens, heads, dim, rot, interleaved=False, base=10000.0, scaling="none", factor=1.0, most):
    return _case("rotate", name, tokens=tokens, heads=heads, dim=dim, rot=rot, interleaved=interleaved, base=base,
                 scaling=scaling, factor=factor, most=most)


def _append(name=None, *, cache, seqs, new, past, q_heads, kv_heads, dim=128, page=64, rot=0, interleaved=False,
            base=1000000.0, scaling="none", factor=1.0):
    return _case("rotary_append", name, cache=cache, seqs=seqs, new=new, past=past, q_heads=q_heads, kv_heads=kv_heads,
                 dim=dim, page=page, rot=rot or dim, interleaved=interleaved, base=base, scaling=scaling, factor=factor)


def _route(name=None, *, tokens, experts, top_k, logits="f32", score="softmax", bias=False, groups=1, top_groups=1,
           group_top=1, renormalise=True, scale=1.0):
    return _case("route", name, tokens=tokens, experts=experts, top_k=top_k, logits=logits, score=score, bias=bias,
                 groups=groups, top_groups=top_groups, group_top=group_top, renormalise=renormalise, scale=scale)


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm", "rotate", "rotary_append", "rotary_append", "route", "route"])
    scaling = rng.choice(["none", "none", "linear", "yarn"])
    factor = 1.0 if scaling == "none" else float(rng.choice([2, 4, 8, 32]))
    base = rng.choice([10000.0, 500000.0, 1000000.0])
    if op == "norm":
        hidden = 8 * log(8, 1024)
        out = rng.choice(["bf16", "bf16", "f32", "fp8", "fp8"])
        return _norm(rows=log(1, min(16384, 16384 * 1024 // hidden)), hidden=hidden, x=rng.choice(["bf16", "bf16", "f32"]),
                     delta=rng.choice(["", "bf16", "f32"]), out=out, group=rng.choice([0, 32, 64, 128]) if out == "fp8" else 0,
                     weight=rng.choice(["", "bf16", "f32"]), eps=rng.choice([1e-5, 1e-6]))
    if op == "rotate":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        heads = log(1, 64)
        return _rotate(tokens=log(1, min(16384, 8191 * 24 * 96 // (heads * dim))), heads=heads, dim=dim,
                       rot=16 * rng.randint(1, dim // 16), interleaved=rng.random() < 0.5, base=base, scaling=scaling,
                       factor=factor, most=log(10, 1000000))
    if op == "rotary_append":
        dim, kv_heads, group = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 8])
        wide = (2 * group + 4) * kv_heads * dim
        cap = 16384 * 48 * 128 // wide
        seqs = log(1, min(64, cap))
        return _append(cache=rng.choice(["bf16", "fp8"]), seqs=seqs, new=1 if rng.random() < 0.4 else log(1, min(16384, cap // seqs)),
                       past=log(1, 200000), q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                       page=rng.choice([16, 32, 64, 128]), rot=16 * rng.randint(1, dim // 16) if rng.random() < 0.4 else dim,
                       interleaved=rng.random() < 0.4, base=base, scaling=scaling, factor=factor)
    groups = rng.choice([1, 1, 4, 8])
    experts = groups * rng.choice([16, 20, 32]) if groups > 1 else rng.choice([16, 60, 64, 72, 128, 160, 256, 384])
    top_groups = rng.randint(1, groups)
    return _route(tokens=log(1, min(16384, 16384 * 256 // experts)), experts=experts,
                  top_k=rng.randint(1, min(16, experts // groups * top_groups)), logits=rng.choice(["f32", "f32", "bf16"]),
                  score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                  group_top=rng.choice([1, 2]), renormalise=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]))


# ---------------------------------------------------------------- work

def _scales(c):
    """Scales of a row of an e4m3 output."""
    return -(-c["hidden"] // (c["group"] or c["hidden"]))


def _lengths(c):
    """New tokens and past ones of each sequence: the lengths spread out, none alike."""
    n = c["seqs"]
    new = [max(1, c["new"] - i * c["new"] // (4 * n)) for i in range(n)]
    return new, [c["past"] - (i * 7 % n) * c["past"] // (2 * n) for i in range(n)]


def work(c):
    if c["op"] == "norm":
        row = c["hidden"] * (_SIZE[c["x"]] * (2 if c["delta"] else 1) + _SIZE[c["delta"]] + _SIZE[c["out"]])
        row += 4 * _scales(c) if c["out"] == "fp8" else 0
        return {"bytes": c["rows"] * row + c["hidden"] * _SIZE[c["weight"]], "flops": 0}
    if c["op"] == "rotate":
        return {"bytes": c["tokens"] * (c["heads"] * c["dim"] * 4 + 4), "flops": 0}
    if c["op"] == "rotary_append":
        held = c["dim"] * 2 if c["cache"] == "bf16" else c["dim"] + 1
        return {"bytes": sum(_lengths(c)[0]) * (c["q_heads"] * 4 * c["dim"] + c["kv_heads"] * 2 * (2 * c["dim"] + held)),
                "flops": 0}
    return {"bytes": c["tokens"] * (c["experts"] * _SIZE[c["logits"]] + c["top_k"] * 8) + (4 * c["experts"] if c["bias"] else 0),
            "flops": 0}


# ---------------------------------------------------------------- inputs

def _frequencies(c):
    """Radians that a token turns each pair by, as Python floats."""
    d, base, f = c["rot"], c["base"], c["factor"]
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if c["scaling"] == "linear":
        return [x / f for x in freq], 1.0
    if c["scaling"] == "yarn":  # pairs that turn often in the first training's length stay, slow ones are stretched

        def pair(turns):  # the index of the pair that turns so often
            return d * math.log(_ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(base))

        low, high = max(0, math.floor(pair(32.0))), min(d - 1, math.ceil(pair(1.0)))
        slow = [min(1.0, max(0.0, (i - low) / max(0.001, high - low))) for i in range(d // 2)]
        return [x * (1 - s) + x / f * s for x, s in zip(freq, slow)], 0.1 * math.log(f) + 1.0
    return freq, 1.0


_ORIGINAL = 4096  # tokens of the first training's contexts


def _own_rotary(c):
    from expert_cache_host_layer_gb300.rotary import Rotary
    return Rotary(c["rot"], base=c["base"], interleaved=c["interleaved"], scaling=c["scaling"], factor=c["factor"],
                  original_length=_ORIGINAL)


def prepare(c, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": c}
    if c["op"] == "norm":
        R, H = c["rows"], c["hidden"]
        # a residual stream with some loud channels and rows of different sizes
        st["x"] = (normal(R, H) * torch.exp(normal(H)) * torch.exp(0.3 * normal(R, 1))).to(_FLOATS[c["x"]])
        st["delta"] = (0.5 * normal(R, H)).to(_FLOATS[c["delta"]]) if c["delta"] else None
        st["weight"] = (1.0 + 0.2 * normal(H)).to(_FLOATS[c["weight"]]) if c["weight"] else None
        fp8 = c["out"] == "fp8"
        st["total"] = torch.empty_like(st["x"]) if c["delta"] else None
        st["out"] = torch.empty(R, H, dtype=torch.float8_e4m3fn if fp8 else _FLOATS[c["out"]], device=dev)
        st["scales"] = torch.empty(R, _scales(c), dtype=torch.float32, device=dev) if fp8 else None
        if own:  # the weight and how its output is wanted: made once per norm of a model
            from expert_cache_host_layer_gb300.norm import RMSNorm
            st["norm"] = RMSNorm(H, st["weight"], eps=c["eps"], group=c["group"])
    elif c["op"] == "rotate":
        T = c["tokens"]
        st["x"] = normal(T, c["heads"], c["dim"]).bfloat16()
        st["out"] = torch.empty_like(st["x"])
        first = torch.randint(0, max(1, c["most"] - T), (1,), generator=gen, device=dev)
        far = torch.randint(0, c["most"] + 1, (T,), generator=gen, device=dev)
        # a chunk's positions follow each other, a batch's are anywhere
        st["positions"] = (first + torch.arange(T, device=dev) if T > 64 else far).to(torch.int32)
    elif c["op"] == "rotary_append":
        new, past = _lengths(c)
        T, S, Hq, H, D, P = sum(new), c["seqs"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        first = [p // P for p in past]
        need = [-(-(p + m) // P) - f for p, m, f in zip(past, new, first)]
        shared = 64  # pages of a long prefix that the sequences share: they hold what came before
        pages = shared + sum(need)
        own_pages = shared + torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32).cpu()
        table = torch.zeros((S, max(f + n for f, n in zip(first, need))), dtype=torch.int32)
        at = 0
        for s in range(S):
            table[s, :first[s]] = torch.arange(first[s], dtype=torch.int32) % shared
            table[s, first[s]:first[s] + need[s]] = own_pages[at:at + need[s]]
            at += need[s]
        shape = (pages, H, P, D)
        if c["cache"] == "fp8":
            st["k_pages"], st["v_pages"] = (normal(*shape).to(torch.float8_e4m3fn) for _ in "kv")
            st["k_scale"], st["v_scale"] = (torch.randint(119, 122, shape[:3], generator=gen, device=dev).to(torch.uint8)
                                            for _ in "kv")
        else:
            st["k_pages"], st["v_pages"] = (normal(*shape).bfloat16() for _ in "kv")
            st["k_scale"] = st["v_scale"] = None
        # queries, keys and values side by side, as one projection writes them; keys with loud and quiet channels
        qkv = normal(T, Hq + 2 * H, D)
        qkv[:, Hq:Hq + H] *= torch.exp(0.5 * normal(H, D))
        qkv = qkv.bfloat16()
        st |= {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + H], "v": qkv[:, Hq + H:], "block_table": table.to(dev),
               "q_start": torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device=dev),
               "kv_len": torch.tensor([p + m for p, m in zip(past, new)], dtype=torch.int32, device=dev),
               "q_out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)}
        if own:  # the layer's cache and the step's batch, as a program keeps them
            from expert_cache_host_layer_gb300.paged_kv import KVBatch, KVPages
            st["pages"] = KVPages(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
            st["batch"] = KVBatch(st["q_start"], st["kv_len"], st["block_table"], T, max(new))
    else:
        T, E = c["tokens"], c["experts"]
        # some experts are asked for more often than others; the bias works against that
        wanted = 0.5 * normal(E)
        st["logits"] = (normal(T, E) + wanted).to(_FLOATS[c["logits"]])
        st["bias"] = (0.1 * normal(E) - 0.1 * wanted) * (1.0 if c["score"] == "sigmoid" else 1.0 / E) if c["bias"] else None
        st["idx"] = torch.empty(T, c["top_k"], dtype=torch.int32, device=dev)
        st["w"] = torch.empty(T, c["top_k"], dtype=torch.float32, device=dev)
        if own:  # the layer's routing rule
            from expert_cache_host_layer_gb300.router import Router
            st["router"] = Router(E, c["top_k"], score=c["score"], bias=st["bias"], groups=c["groups"],
                                  top_groups=c["top_groups"], group_top=c["group_top"], renormalise=c["renormalise"],
                                  scale=c["scale"])
    if c["op"] in ("rotate", "rotary_append"):
        freq, factor = _frequencies(c)
        st["freq"], st["factor"] = torch.tensor(freq, dtype=torch.float64, device=dev), factor
        if own:
            st["rotary"] = _own_rotary(c)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if op == "norm":
        if not own:
            return _plain_norm(st)
        st["norm"].apply(st["x"], st["out"], delta=st["delta"], total=st["total"], scales=st["scales"])
        return [st["total"], st["out"], st["scales"]]
    if op == "rotate":
        if not own:
            return _turn(st["x"], *_angles(st, st["positions"]), st["case"]).bfloat16()
        st["rotary"].rotate(st["positions"], st["x"], st["out"])
        return st["out"]
    if op == "rotary_append":
        if own:
            st["pages"].append(st["batch"], st["k"], st["v"], rotary=st["rotary"], q=st["q"], q_out=st["q_out"])
        else:
            _plain_append(st)
        # (the scales' exponent bytes are float8_e8m0fnu numbers)
        held = [] if st["k_scale"] is None else [st[n].view(torch.float8_e8m0fnu) for n in ("k_scale", "v_scale")]
        return [st["q_out"], st["k_pages"], st["v_pages"], *held]
    if not own:
        return _plain_route(st)
    st["router"].route(st["logits"], st["idx"], st["w"])
    return [st["idx"], st["w"]]


def _plain_norm(st):
    c = st["case"]
    x = st["x"].float()
    total = None
    if c["delta"]:
        x = x + st["delta"].float()
        total = x.to(st["x"].dtype)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c["eps"])
    if st["weight"] is not None:
        y = y * st["weight"].float()
    if c["out"] != "fp8":
        return [total, y.to(_FLOATS[c["out"]]), None]
    R, H, G = c["rows"], c["hidden"], _scales(c)
    wide = c["group"] or H
    y = torch.nn.functional.pad(y, (0, G * wide - H)).view(R, G, wide)
    scales = y.abs().amax(-1) / 448.0
    return [total, (y / scales.unsqueeze(-1)).view(R, -1)[:, :H].to(torch.float8_e4m3fn), scales]


def _angles(st, positions):
    """cos and sin of the tokens' angles (products in 64 bits: at far positions 32 would lose the turn's fraction)."""
    a = positions.double().unsqueeze(-1) * st["freq"]
    return (a.cos() * st["factor"]).float().unsqueeze(1), (a.sin() * st["factor"]).float().unsqueeze(1)


def _turn(x, cos, sin, c):
    """x [tokens, heads, dim] with its first `rot` channels rotated, in 32 bits."""
    x = x.float()
    r = x[..., :c["rot"]]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else r.chunk(2, -1)
    r = (a * cos - b * sin, b * cos + a * sin)
    r = torch.stack(r, -1).flatten(-2) if c["interleaved"] else torch.cat(r, -1)
    return torch.cat([r, x[..., c["rot"]:]], -1)


def _quantise(x):
    """e4m3 codes and exponent bytes: the smallest power of two s (2^-110 at
    least) with max|x| <= 448 s, and x / s rounded to nearest even."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = (e - 9 + (m > 0.875).int()).clamp(min=-110)  # m 2^e <= 448 2^k = 0.875 2^(9 + k)
    return (x * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_append(st):
    c, q_start = st["case"], st["q_start"].long()
    t = torch.arange(st["q"].shape[0], device=q_start.device)
    s = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    pos = st["kv_len"].long()[s] - q_start[s + 1] + t
    page, slot = st["block_table"].long()[s, pos // c["page"]], pos % c["page"]
    trig = _angles(st, pos)
    st["q_out"].copy_(_turn(st["q"], *trig, c))
    for x, pages, scales in ((_turn(st["k"], *trig, c), st["k_pages"], st["k_scale"]),
                             (st["v"].float(), st["v_pages"], st["v_scale"])):
        if scales is None:
            pages.transpose(0, 1)[:, page, slot] = x.bfloat16().transpose(0, 1)
            continue
        codes, e = _quantise(x)
        pages.view(torch.uint8).transpose(0, 1)[:, page, slot] = codes.view(torch.uint8).transpose(0, 1)
        scales.transpose(0, 1)[:, page, slot] = e.transpose(0, 1)


def _best(x, k):
    """The k largest of each row, the lowest index first among equals."""
    return torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :k]


def _plain_route(st):
    """In 64 bits: experts lie next to the border of the choice."""
    c = st["case"]
    T, E, G = c["tokens"], c["experts"], c["groups"]
    logits = st["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    key = score if st["bias"] is None else score + st["bias"].double()
    if G > 1:
        parts = key.view(T, G, E // G)
        of = torch.sort(parts, dim=-1, descending=True)[0][..., :c["group_top"]].sum(-1)
        in_best = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, _best(of, c["top_groups"]), True)
        key = parts.masked_fill(~in_best.unsqueeze(-1), float("-inf")).view(T, E)
    idx = _best(key, c["top_k"])
    w = score.gather(-1, idx)
    if c["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    return [idx.to(torch.int32), (w * c["scale"]).float()]


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _two(n):
    """2^n in 64 bits, exactly, by the bits of a double."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x rounded to a value of 4 significant bits, steps of 2^-9 at least (ties to even), no further than 448."""
    step = _two(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_turn(st, x, positions):
    """The pairs as complex numbers times the tokens' e^(i angle)."""
    c = st["case"]
    x, half = x.double().clone(), c["rot"] // 2
    turn = torch.polar(torch.full_like(st["freq"], st["factor"]).expand(len(positions), -1).contiguous(),
                       positions.double()[:, None] * st["freq"])[:, None]
    re, im = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, half), slice(half, c["rot"]))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * turn
    x[..., re], x[..., im] = z.real, z.imag
    return x


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "norm":
        x = st["x"].double()
        if c["delta"]:
            x = x + st["delta"].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["hidden"] + c["eps"])
        y = y if st["weight"] is None else st["weight"].double() * y
        total = x if c["delta"] else None
        if c["out"] != "fp8":
            return [total, y, None]
        wide = c["group"] or c["hidden"]
        codes, scales = torch.empty_like(y), torch.empty(c["rows"], _scales(c), dtype=torch.float64, device=y.device)
        for g in range(_scales(c)):
            part = y[:, g * wide:(g + 1) * wide]
            scales[:, g] = part.abs().amax(-1) / 448.0
            codes[:, g * wide:(g + 1) * wide] = _e4m3(part / scales[:, g:g + 1])
        return [total, codes, scales]
    if c["op"] == "rotate":
        return _exact_turn(st, st["x"], st["positions"])
    if c["op"] == "rotary_append":
        new, past = _lengths(c)
        pos = torch.cat([torch.arange(p, p + m, device=st["q"].device) for p, m in zip(past, new)])
        q, k, v = _exact_turn(st, st["q"], pos), _exact_turn(st, st["k"], pos), st["v"].double()
        P, table, held, scaled = c["page"], st["block_table"].long(), [], []
        for x, pages, scales in ((k, st["k_pages"], st["k_scale"]), (v, st["v_pages"], st["v_scale"])):
            pages, t0 = pages.double(), 0
            scales = None if scales is None else _two(scales.long() - 127)
            for s, m in enumerate(new):
                one, p = x[t0:t0 + m], pos[t0:t0 + m]
                if scales is not None:
                    part, e = torch.frexp(one.abs().amax(-1) / 448.0)
                    e = _two(torch.where(part > 0.5, e, e - 1).clamp(min=-110))  # the least 2^e with max|x| <= 448 2^e
                    one = _e4m3(one / e.unsqueeze(-1))
                    scales[table[s, p // P], :, p % P] = e
                pages[table[s, p // P], :, p % P] = one
                t0 += m
            held.append(pages)
            scaled += [] if scales is None else [scales]
        return [q, *held, *scaled]
    # route: the experts that the choice falls on are whole numbers; their weights, token by token of a loop over picks
    x = st["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    key = p.clone() if st["bias"] is None else p + st["bias"].double()
    if c["groups"] > 1:
        parts = key.view(c["tokens"], c["groups"], -1)
        of = parts.topk(c["group_top"], dim=-1)[0].sum(-1)
        above = (of.unsqueeze(1) > of.unsqueeze(2)).sum(-1)  # groups before this one: better, or equal and lower
        above += torch.tril(of.unsqueeze(1) == of.unsqueeze(2), -1).sum(-1)
        key = torch.where((above < c["top_groups"]).unsqueeze(-1), parts, -math.inf).reshape(c["tokens"], -1)
    w = torch.empty(c["tokens"], c["top_k"], dtype=torch.float64, device=x.device)
    for j in range(c["top_k"]):
        at = key.argmax(-1, keepdim=True)
        w[:, j:j + 1] = p.gather(-1, at)
        key.scatter_(-1, at, -math.inf)
    return [None, (w / w.sum(-1, keepdim=True) if c["renormalise"] else w) * c["scale"]]
