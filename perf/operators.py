"""Cases of the attention half of a decode layer: INT4 projections, the cache write with norms and rotation, the cache
read and the paged attention of one new token.

Head counts and widths are those of the stacks this repository runs (d_model 4096 with 128-wide heads, d_model 8192 with
64-wide heads) or generic.  A cache is four tensors: the codes of K and V, [pages, kv heads, page size, row] ("hnd") or
[pages, page size, kv heads, row] ("nhd"), and the scales of the two quantised formats.
"""
import math

import torch

own = False

FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------
def _matvec(name, n, k, tokens, x, y, norm=False, add=False):
    return {"name": name, "op": "matvec", "n": n, "k": k, "tokens": tokens, "x": x, "y": y, "norm": norm, "add": add}


def _append(name, tokens, seqs, heads, kv_heads, dim, io, cache, page, rotary, style="half", norm=False, start=0, pads=0,
            layout="hnd"):
    return {"name": name, "op": "append", "tokens": tokens, "seqs": seqs, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "io": io, "cache": cache, "page": page, "rotary": rotary, "style": style, "norm": norm, "start": start,
            "pads": pads, "layout": layout}


def _read(name, seqs, rows, kv_heads, dim, io, cache, page, layout="hnd"):
    return {"name": name, "op": "read", "seqs": seqs, "rows": rows, "kv_heads": kv_heads, "dim": dim, "io": io,
            "cache": cache, "page": page, "layout": layout}


def _attend(name, seqs, length, lens, heads, kv_heads, dim, io, cache, page, window=0, cap=0.0, layout="hnd"):
    return {"name": name, "op": "attend", "seqs": seqs, "length": length, "lens": lens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "io": io, "cache": cache, "page": page, "window": window, "cap": cap,
            "layout": layout}


def listed():
    return [
        # the key (or value) projection of 8 heads for one token: the smallest product of a layer, all latency
        _matvec("matvec 1024x4096 one token", 1024, 4096, 1, "f16", "f16"),
        # query, key and value of one token at once, straight from the fp32 residual with its norm
        _matvec("matvec 6144x4096 from the residual", 6144, 4096, 1, "f32", "f32", norm=True),
        # the output projection of a small batch, added to the fp32 residual
        _matvec("matvec 8192x8192 onto the residual", 8192, 8192, 13, "bf16", "f32", add=True),
        # the cache write of one decoded token far into a long text
        _append("append one token", 1, 1, 32, 8, 128, "bf16", "bf16", 64, 128, norm=True, start=30011),
        # the cache write of a decode batch, some of its places empty, and what the cache then holds
        _append("append a batch to i8", 32, 32, 128, 8, 64, "f16", "i8", 16, 64, start=4000, pads=3),
        # a prompt into a 4-bit cache, and the rows as the prompt's own attention has to see them
        _append("append a prompt to int4", 512, 1, 32, 8, 128, "f16", "int4g32", 64, 128, norm=True),
        # one sequence taken out of the cache, of odd length
        _read("read 701 rows of i8", 1, 701, 8, 64, "f16", "i8", 16),
        # the prefixes of a batch taken out of a 4-bit cache
        _read("read 8 prefixes of int4", 8, 4096, 8, 128, "bf16", "int4g32", 64),
        # the first words of an answer: a short text, a cache of its own for each head
        _attend("attend 200 positions", 1, 200, "full", 32, 32, 128, "f16", "f16", 16),
        # one user with a long text in a 4-bit cache
        _attend("attend 32768 positions of int4", 1, 32768, "full", 32, 8, 128, "f16", "int4g32", 64),
        # a decode batch of all lengths, an empty one and one of a single position among them
        _attend("attend a batch of ragged texts", 32, 8191, "ragged", 32, 8, 128, "bf16", "bf16", 64),
        # capped scores in a sliding window over an 8-bit cache, sixteen queries to a cached head
        _attend("attend in a window of i8", 16, 6000, "ragged", 128, 8, 64, "bf16", "i8", 16, window=4096, cap=30.0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["matvec", "append", "read", "attend"])
    io = rng.choice(["f16", "bf16"])
    cache = rng.choice(["f16" if io == "f16" else "bf16", "i8", "int4g32"])
    dim, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 5, 8, 16, 32])
    page, layout = rng.choice([8, 16, 32, 64, 128]), rng.choice(["hnd", "nhd"])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "matvec":
        x = rng.choice(["f32", "f16", "bf16"])
        n, k = _log(rng, 64, 16384), 32 * _log(rng, 8, 512)
        tokens = rng.choice([1, 1, 1, 2, 4, 8, rng.randint(3, 32)])
        while n * k > 8192 * 8192 or n * k * tokens > 13 * 8192 * 8192:
            n, tokens = n // 2 + 1, tokens // 2 + 1
        return _matvec(None, n, k, tokens, x, rng.choice([x, "f32"]), rng.random() < 0.4, rng.random() < 0.4)
    if op == "append":
        many = rng.random() < 0.5
        tokens = _log(rng, 2, 512) if many else rng.randint(1, 32)
        while tokens * group * kv_heads * dim > 512 * 32 * 128 and group > 1:
            group //= 2
        while tokens * group * kv_heads * dim > 512 * 32 * 128:
            tokens //= 2
        rotary = rng.choice([dim, dim, dim // 2, 0])
        return _append(None, tokens, 1 if many else tokens, group * kv_heads, kv_heads, dim, io, cache, page, rotary,
                       rng.choice(["half", "pairs"]), rng.random() < 0.5, _log(rng, 1, 32000), rng.choice([0, 0, tokens // 4]),
                       layout)
    if op == "read":
        seqs = _log(rng, 1, 8)
        rows = _log(rng, 1, 4096)
        while rows > 1 and seqs * rows * kv_heads * dim > 8 * 4096 * 8 * 128:
            rows //= 2
        return _read(None, seqs, rows, kv_heads, dim, io, cache, page, layout)
    seqs, length = _log(rng, 1, 32), _log(rng, 1, 32768)
    while length > 1 and seqs * length * kv_heads * dim * max(1, group // 4) > 16 * 8191 * 8 * 128:
        length //= 2
    return _attend(None, seqs, length, rng.choice(["full", "ragged"]), group * kv_heads, kv_heads, dim, io, cache, page,
                   rng.choice([0, 0, 1 + length // 3]), rng.choice([0.0, 0.0, 20.0]), layout)


def _lens(case):
    """The sequences' lengths: all alike, or spread evenly over 1 .. length with an empty and a single one among four."""
    n, top = case["seqs"], case["length"]
    if case["lens"] == "full":
        return [top] * n
    got = [1 + int(((i + 1) * 0.6180339887498949 % 1.0) * top) for i in range(n)]
    got[0] = top
    if n >= 4:
        got[1], got[2] = 0, 1
    return [min(x, top) for x in got]


def _row_bytes(case):
    """Bytes of one cached vector with its scales."""
    d, c = case["dim"], case["cache"]
    return {"f16": 2 * d, "bf16": 2 * d, "i8": d + 4, "int4g32": d // 2 + d // 16}[c]


def work(case):
    op = case["op"]
    if op == "matvec":
        n, k, t = case["n"], case["k"], case["tokens"]
        y = t * n * SIZE[case["y"]]
        return {"bytes": n * k // 2 + n * k // 16 + t * k * SIZE[case["x"]] + y * (2 if case["add"] else 1),
                "flops": 2 * t * n * k}
    d, hk, b = case["dim"], case["kv_heads"], SIZE[case["io"]]
    if op == "append":
        t = case["tokens"] - case["pads"]
        rows = 2 * t * hk * _row_bytes(case)
        moved = t * (2 * case["heads"] + 2 * hk) * d * b + rows
        if case["cache"] in ("i8", "int4g32"):
            moved += rows + 2 * t * hk * d * b
        return {"bytes": moved, "flops": 10 * t * (case["heads"] + 2 * hk) * d}
    if op == "read":
        n = 2 * case["seqs"] * case["rows"] * hk
        return {"bytes": n * (_row_bytes(case) + d * b), "flops": n * d}
    seen = sum(min(x, case["window"]) if case["window"] else x for x in _lens(case))
    q = case["seqs"] * case["heads"]
    return {"bytes": 2 * seen * hk * _row_bytes(case) + q * (2 * d * b + 4), "flops": 4 * seen * case["heads"] * d}


# ---------------------------------------------------------------------------------------------------------------------
# Formats (the writer's side, as the inputs are made)
# ---------------------------------------------------------------------------------------------------------------------
def _int4(w):
    """Last axis in groups of 32: s = fp16(max|w| / 7), q = round(w / s) in -8 .. 7, stored as q + 8, even element low."""
    g = w.double().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7).to(torch.float16)
    d = s.double().unsqueeze(-1)
    q = torch.where(d > 0, torch.round(g / torch.where(d > 0, d, 1.0)), 0.0).clamp(-8, 7)
    n = (q.flatten(-2) + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), s


def _i8(w):
    """Last axis a row: s = fp32(max|w| / 127), q = round(w / s) in -127 .. 127."""
    w = w.double()
    s = (w.abs().amax(-1) / 127).float()
    d = s.double().unsqueeze(-1)
    q = torch.where(d > 0, torch.round(w / torch.where(d > 0, d, 1.0)), 0.0).clamp(-127, 127)
    return q.to(torch.int8), s


def _encode(w, cache):
    if cache == "int4g32":
        return _int4(w)
    if cache == "i8":
        return _i8(w)
    return w.float().to(FLOAT[cache]), None


def _decode(codes, scale, cache):
    """The values that stored rows stand for, in 32 bits."""
    if cache == "int4g32":
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
        return (n.unflatten(-1, (-1, 32)) * scale.float().unsqueeze(-1)).flatten(-2)
    if cache == "i8":
        return codes.float() * scale.unsqueeze(-1)
    return codes.float()


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------
class _Handle:
    """A library handle that is released with the state that holds it."""

    def __init__(self, value, release):
        self.value, self.release = value, release

    def __del__(self):
        torch.cuda.synchronize()
        self.release(self.value)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _cache(case, g, pages, fill):
    """A cache without rows, or one full of them: channels of different sizes in K, as trained models have them."""
    hk, p, d = case["kv_heads"], case["page"], case["dim"]
    shape = (pages, hk, p) if case["layout"] == "hnd" else (pages, p, hk)
    if not fill:
        row, dtype = {"i8": (d, torch.int8), "int4g32": (d // 2, torch.uint8)}.get(case["cache"], (d, None))
        empty = lambda *n, t: torch.zeros(*shape, *n, device="cuda", dtype=t)  # noqa: E731
        codes = lambda: empty(row, t=dtype or FLOAT[case["cache"]])  # noqa: E731
        scale = {"i8": lambda: empty(t=torch.float32), "int4g32": lambda: empty(d // 32, t=torch.float16)}.get(case["cache"], lambda: None)
        return {"k": codes(), "v": codes(), "k_scale": scale(), "v_scale": scale()}
    size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    # in blocks of pages: the 64-bit arithmetic of the writer takes room
    block = max(1, (1 << 24) // (hk * p * d))
    got = [[], []]
    for a in range(0, pages, block):
        n = min(block, pages - a)
        for i in range(2):
            w = _normal(g, n, *shape[1:], d)
            got[i].append(_encode(w * size if i == 0 else w, case["cache"]))
    join = lambda i, j: torch.cat([x[j] for x in got[i]]) if got[i][0][j] is not None else None  # noqa: E731
    return {"k": join(0, 0), "v": join(1, 0), "k_scale": join(0, 1), "v_scale": join(1, 1)}


def _table(case, g, lens):
    """Pages of the sequences in random order over the cache, and how many the cache has; unused entries are -1."""
    p = case["page"]
    need = [-(-x // p) for x in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(need))
    at = torch.arange(width, device="cuda")
    need_d = torch.tensor(need, device="cuda")
    first = torch.cumsum(need_d, 0) - need_d
    idx = (first[:, None] + at).clamp(max=pages - 1)
    return torch.where(at < need_d[:, None], order[idx], -1).to(torch.int32).contiguous(), pages


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    op = case["op"]
    if op == "matvec":
        n, k, t = case["n"], case["k"], case["tokens"]
        q, sc = _int4(_normal(g, n, k, std=0.02))
        s = {"q": q, "scale": sc, "x": _normal(g, t, k, dtype=FLOAT[case["x"]]),
             "y": torch.zeros(t, n, device="cuda", dtype=FLOAT[case["y"]])}
        s["add"] = _normal(g, t, n, dtype=FLOAT[case["y"]]) if case["add"] else None
        return s
    io, d, hk = FLOAT[case["io"]], case["dim"], case["kv_heads"]
    if op == "append":
        t, n, h = case["tokens"], case["seqs"], case["heads"]
        step = torch.arange(t, device="cuda")
        # one sequence's tokens follow each other; a batch's sequences stand at different places
        pos = case["start"] + (step if n == 1 else (step * 37) % 97)
        top = int(case["start"] + (t if n == 1 else 97))
        table, pages = _table(case, g, [top if n == 1 else min(top, 8 * case["page"])] * n)
        if n > 1:
            pos = pos % (8 * case["page"])
        if case["pads"]:
            pos = torch.where(step >= t - case["pads"], -1, pos)
        qkv = _normal(g, t, (h + 2 * hk) * d, dtype=io)
        norm = case["norm"]
        weight = lambda: 1 + 0.2 * _normal(g, d) if norm else None  # noqa: E731
        s = {"table": table, "pos": pos.to(torch.int32), "q": qkv[:, :h * d].unflatten(1, (h, d)),
             "k_new": qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d)), "v_new": qkv[:, (h + hk) * d:].unflatten(1, (hk, d)),
             "q_norm": weight(), "k_norm": weight(), "q_out": torch.zeros(t, h, d, device="cuda", dtype=io),
             "seq": torch.zeros(t, device="cuda", dtype=torch.int32) if n == 1 else step.to(torch.int32)}
        s.update(_cache(case, g, pages, False))
        s["k_out"] = torch.zeros(t, hk, d, device="cuda", dtype=io)
        s["v_out"] = torch.zeros(t, hk, d, device="cuda", dtype=io)
        return s
    if op == "read":
        n, r = case["seqs"], case["rows"]
        table, pages = _table(case, g, [r] * n)
        s = {"table": table, "pos": torch.arange(r, device="cuda", dtype=torch.int32).repeat(n),
             "seq": torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(r)}
        s.update(_cache(case, g, pages, True))
        s["k_out"] = torch.zeros(n * r, hk, d, device="cuda", dtype=io)
        s["v_out"] = torch.zeros(n * r, hk, d, device="cuda", dtype=io)
        return s
    lens = _lens(case)
    table, pages = _table(case, g, lens)
    n, h = case["seqs"], case["heads"]
    s = {"table": table, "lens": torch.tensor(lens, device="cuda", dtype=torch.int32),
         "q": _normal(g, n, h, d, std=1.5, dtype=io), "out": torch.zeros(n, h, d, device="cuda", dtype=io),
         "lse": torch.zeros(n, h, device="cuda")}
    s.update(_cache(case, g, pages, True))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from activation_sparse_decode_threshold_b200 import binding as B
        s["B"] = B
        if case["op"] == "matvec":
            s["handle"] = _Handle(B.pi_int4_create(s["q"], s["scale"]), B.pi_int4_destroy)
        else:
            s["handle"] = _Handle(B.pi_attn_create(
                case.get("heads", case["kv_heads"]), case["kv_heads"], case["dim"], cache_dtype=case["cache"],
                page_size=case["page"], layout=case["layout"], rotary_dim=case.get("rotary", 0),
                rotary_pairs=case.get("style") == "pairs", rope_theta=10000.0, norm_eps=1e-6 if case.get("norm") else 0.0,
                window=case.get("window", 0), softcap=case.get("cap", 0.0)), B.pi_attn_destroy)
            s["cache"] = B.pi_kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    return {"matvec": _run_matvec, "append": _run_append, "read": _run_read, "attend": _run_attend}[s["case"]["op"]](s)


def _run_matvec(s):
    case = s["case"]
    if own:
        s["B"].pi_int4_matvec(s["handle"].value, s["x"], s["y"], add=s["add"], norm_eps=1e-6 if case["norm"] else 0.0)
        return s["y"]
    x = s["x"].float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    y = x @ _decode(s["q"], s["scale"], "int4g32").t()
    if case["add"]:
        y = y + s["add"].float()
    return y.to(FLOAT[case["y"]])


def _rotate(x, pos, rotary, style):
    """Pairs (i, i + rotary / 2), or (2i, 2i + 1), turned by pos * 10000^(-2i / rotary); x [tokens, heads, dim]."""
    if not rotary:
        return x
    freq = 10000.0 ** (torch.arange(0, rotary, 2, device=x.device, dtype=torch.float64) / -rotary)
    a = pos.double()[:, None, None] * freq
    c, n = torch.cos(a).to(x.dtype), torch.sin(a).to(x.dtype)
    r, rest = x[..., :rotary], x[..., rotary:]
    if style == "half":
        u, v = r.chunk(2, -1)
        r = torch.cat((u * c - v * n, v * c + u * n), -1)
    else:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack((u * c - v * n, v * c + u * n), -1).flatten(-2)
    return torch.cat((r, rest), -1)


def _slots(s, layout):
    """Index of each token's rows in a cache: tensors to index it with, and which tokens have one."""
    p = s["case"]["page"]
    live = s["pos"] >= 0
    pos = s["pos"].clamp(min=0).long()
    page = s["table"][s["seq"].long(), pos // p].long()
    return page, pos % p, live


def _write(s, name, scale, rows):
    """rows [tokens, kv heads, dim] into the cache, by the format's rule in 64 bits (codes lie next to borders)."""
    case = s["case"]
    page, off, live = _slots(s, case["layout"])
    codes, sc = _encode(rows, case["cache"])
    heads = torch.arange(case["kv_heads"], device=rows.device)
    at = (page[:, None], heads, off[:, None]) if case["layout"] == "hnd" else (page[:, None], off[:, None], heads)
    keep = live[:, None, None]
    s[name][at] = torch.where(keep, codes, s[name][at])
    if sc is not None:
        s[scale][at] = torch.where(keep if sc.dim() == 3 else keep[..., 0], sc, s[scale][at])


def _rows(s, name, scale):
    """The cache's rows of the tokens as values."""
    case = s["case"]
    page, off, live = _slots(s, case["layout"])
    heads = torch.arange(case["kv_heads"], device=page.device)
    at = (page[:, None], heads, off[:, None]) if case["layout"] == "hnd" else (page[:, None], off[:, None], heads)
    w = _decode(s[name][at], s[scale][at] if s[scale] is not None else None, case["cache"])
    return torch.where(live[:, None, None], w, 0.0).to(FLOAT[case["io"]])


def _run_append(s):
    case = s["case"]
    quantised = case["cache"] in ("i8", "int4g32")
    if own:
        B, h = s["B"], s["handle"].value
        B.pi_kv_append(h, s["cache"], s["table"], s["pos"], s["q"], s["k_new"], s["v_new"], s["q_out"], seq=s["seq"],
                       q_norm=s["q_norm"], k_norm=s["k_norm"])
        if quantised:
            B.pi_kv_read(h, s["cache"], s["table"], s["pos"], s["k_out"], s["v_out"], seq=s["seq"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}

    def turned(x, weight):
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.to(x.dtype)
        return _rotate(x, s["pos"].clamp(min=0), case["rotary"], case["style"])

    q = turned(s["q"].float(), s["q_norm"])
    q = torch.where(s["pos"][:, None, None] >= 0, q, 0.0).to(FLOAT[case["io"]])
    _write(s, "k", "k_scale", turned(s["k_new"].double(), s["k_norm"]))
    _write(s, "v", "v_scale", s["v_new"])
    if quantised:
        return {"q": q, "k": _rows(s, "k", "k_scale"), "v": _rows(s, "v", "v_scale")}
    return {"q": q, "k": s["k"], "v": s["v"]}


def _run_read(s):
    if own:
        s["B"].pi_kv_read(s["handle"].value, s["cache"], s["table"], s["pos"], s["k_out"], s["v_out"], seq=s["seq"])
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"k": _rows(s, "k", "k_scale"), "v": _rows(s, "v", "v_scale")}


def _gathered(s, name, scale):
    """The sequences' pages as values, [seqs, kv heads, positions, dim]; rows of no sequence are 0."""
    case = s["case"]
    page = s["table"].long()
    idx = page.clamp(min=0)
    w = _decode(s[name][idx], s[scale][idx] if s[scale] is not None else None, case["cache"])
    w = w * (page >= 0)[:, :, None, None, None]
    return (w.permute(0, 2, 1, 3, 4) if case["layout"] == "hnd" else w.permute(0, 3, 1, 2, 4)).flatten(2, 3)


def _run_attend(s):
    case = s["case"]
    if own:
        s["B"].pi_paged_attention(s["handle"].value, s["cache"], s["table"], s["lens"], s["q"], s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    n, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    q = s["q"].float().view(n, hk, h // hk, d)
    x = q @ _gathered(s, "k", "k_scale").transpose(2, 3) / math.sqrt(d)
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    at = torch.arange(x.shape[-1], device=x.device)
    top = s["lens"][:, None]
    seen = at < top
    if case["window"]:
        seen &= at >= top - case["window"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ _gathered(s, "v", "v_scale")) / torch.where(total > 0, total, 1.0)
    lse = m + torch.log(total)
    return {"out": o.reshape(n, h, d).to(FLOAT[case["io"]]), "lse": lse.reshape(n, h)}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "matvec":
        return _exact_matvec(case, s)
    if op == "append":
        return _exact_append(case, s)
    if op == "read":
        rows = [_exact_rows(case, s, "k", i) for i in range(case["seqs"])], [_exact_rows(case, s, "v", i) for i in range(case["seqs"])]
        return {"k": torch.cat(rows[0]), "v": torch.cat(rows[1])}
    return _exact_attend(case, s)


def _exact_matvec(case, s):
    x = s["x"].double()
    if case["norm"]:
        x = x / torch.sqrt(torch.einsum("tk,tk->t", x, x) / case["k"] + 1e-6)[:, None]
    low, high = (s["q"] % 16).double(), torch.div(s["q"], 16, rounding_mode="floor").double()
    scale = s["scale"].double().repeat_interleave(16, 1)
    y = torch.einsum("tk,nk->tn", x[:, 0::2], (low - 8) * scale) + torch.einsum("tk,nk->tn", x[:, 1::2], (high - 8) * scale)
    return y if s["add"] is None else y + s["add"].double()


def _exact_values(case, codes, scale):
    c = case["cache"]
    if c == "i8":
        return torch.einsum("...d,...->...d", codes.double(), scale.double())
    if c == "int4g32":
        out = torch.empty(*codes.shape[:-1], case["dim"], dtype=torch.float64, device=codes.device)
        out[..., 0::2] = (codes % 16).double() - 8
        out[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double() - 8
        return out * scale.double().repeat_interleave(32, -1)
    return codes.double()


def _exact_rows(case, s, name, seq):
    """All positions that sequence `seq` has pages for, [positions, kv heads, dim]; a read takes the first rows of them."""
    pages = s["table"][seq]
    pages = pages[pages >= 0].long()
    scale = s[name + "_scale"]
    w = _exact_values(case, s[name][pages], None if scale is None else scale[pages])
    w = (w.transpose(1, 2) if case["layout"] == "hnd" else w).reshape(-1, case["kv_heads"], case["dim"])
    return w[:case["rows"]] if case["op"] == "read" else w


def _exact_append(case, s):
    d, live = case["dim"], (s["pos"] >= 0).tolist()
    pos = s["pos"].double()

    def turned(x, weight):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + 1e-6) * weight.double()
        r = case["rotary"]
        out = x.clone()
        for i in range(r // 2):
            a, b = (i, i + r // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
            angle = pos * math.pow(10000.0, -2.0 * i / r)
            c, n = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            out[..., a] = x[..., a] * c - x[..., b] * n
            out[..., b] = x[..., b] * c + x[..., a] * n
        return out

    mask = torch.tensor(live, device="cuda")[:, None, None]
    q = torch.where(mask, turned(s["q"], s["q_norm"]), 0.0)
    rows = turned(s["k_new"], s["k_norm"]), s["v_new"].double()
    if case["cache"] in ("i8", "int4g32"):
        got = []
        for w in rows:
            n, top = (d, 127) if case["cache"] == "i8" else (32, 7)
            g = w.reshape(*w.shape[:-1], d // n, n)
            scale = (g.abs().amax(-1, keepdim=True) / top).to(torch.float32 if top == 127 else torch.float16).double()
            got.append(torch.where(mask, (torch.clamp(torch.round(g / scale), -127 if top == 127 else -8, top) * scale).reshape(w.shape), 0.0))
        return {"q": q, "k": got[0], "v": got[1]}
    caches = []
    for name, w in zip(("k", "v"), rows):
        full = s[name].double()
        for t in range(case["tokens"]):
            if live[t]:
                p = int(s["pos"][t])
                page = int(s["table"][int(s["seq"][t]), p // case["page"]])
                if case["layout"] == "hnd":
                    full[page, :, p % case["page"]] = w[t]
                else:
                    full[page, p % case["page"]] = w[t]
        caches.append(full)
    return {"q": q, "k": caches[0], "v": caches[1]}


def _exact_attend(case, s):
    n, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(n, h, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(_lens(case)):
        first = max(0, length - case["window"]) if case["window"] else 0
        if length == 0:
            continue
        k, v = (_exact_rows(case, s, name, i)[first:length] for name in ("k", "v"))
        q = s["q"][i].double().view(hk, h // hk, d)
        x = torch.einsum("kgd,pkd->kgp", q, k) / math.sqrt(d)
        if case["cap"]:
            x = torch.tanh(x / case["cap"]) * case["cap"]
        lse[i] = torch.logsumexp(x, -1).flatten()
        out[i] = torch.einsum("kgp,pkd->kgd", torch.softmax(x, -1), v).reshape(h, d)
    return {"out": out, "lse": lse}
