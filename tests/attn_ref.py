"""Plain 64-bit definitions of the attention half of a decode layer, in torch on
the CPU, with the error bounds that the tests hold the kernels to.

Every bound is made of roundings: a value rounded to type t is off by at most
half a step, HALF[t] relative to it; an fp32 operation by 2^-24; a sum of n
terms in fp32 by n 2^-24 of the sum of their magnitudes, in any order (twice
that on the tensor cores, which may cut off instead of rounding)."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}   # least step, halved
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def half_step(x: torch.Tensor, dtype) -> torch.Tensor:
    return x.abs() * HALF[dtype] + TINY[dtype]


# ---- formats --------------------------------------------------------------
def encode_int4(w):
    g = w.double().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 7).to(torch.float16)
    d = s.double().unsqueeze(-1)
    q = torch.where((d > 0) & d.isfinite(), torch.round(g / torch.where(d > 0, d, 1.0)), 0.0).clamp(-8, 7)
    n = (q.flatten(-2) + 8).to(torch.uint8)
    return (n[..., 0::2] | (n[..., 1::2] << 4)).contiguous(), s.contiguous()


def encode_i8(w):
    w = w.double()
    s = (w.abs().amax(-1) / 127).float()
    d = s.double().unsqueeze(-1)
    q = torch.where((d > 0) & d.isfinite(), torch.round(w / torch.where(d > 0, d, 1.0)), 0.0).clamp(-127, 127)
    return q.to(torch.int8).contiguous(), s.contiguous()


def encode(w, cache):
    if cache == "int4g32":
        return encode_int4(w)
    if cache == "i8":
        return encode_i8(w)
    return w.float().to(DT[cache]).contiguous(), None


def decode(codes, scale, cache):
    """Stored rows as the values they stand for, in 64 bits."""
    if cache == "int4g32":
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
        return (n.unflatten(-1, (-1, 32)) * scale.double().unsqueeze(-1)).flatten(-2)
    if cache == "i8":
        return codes.double() * scale.double().unsqueeze(-1)
    return codes.double()


# ---- a cache and its table ------------------------------------------------
class Cache:
    """A paged cache on `device`, filled with rows or empty, and its page table."""

    def __init__(self, g, lens, kv_heads, dim, cache, page, layout="hnd", fill=True, spare=2, device="cpu"):
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        self.kind, self.page, self.layout, self.heads, self.dim = cache, page, layout, kv_heads, dim
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        width = max(1, max(need))
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page, dim) if layout == "hnd" else (self.pages, page, kv_heads, dim)
        mk = (lambda: torch.randn(shape, generator=g)) if fill else (lambda: torch.zeros(shape))
        self.k, self.k_scale = encode(mk(), cache)
        self.v, self.v_scale = encode(mk(), cache)

    def rows(self, name, seq, first, last):
        """Positions [first, last) of a sequence: [positions, kv heads, dim] in 64 bits."""
        codes, scale = getattr(self, name).cpu(), getattr(self, name + "_scale")
        scale = None if scale is None else scale.cpu()
        out = torch.empty(max(0, last - first), self.heads, self.dim, dtype=torch.float64)
        for i, p in enumerate(range(first, last)):
            page, slot = int(self.table[seq, p // self.page]), p % self.page
            at = (page, slice(None), slot) if self.layout == "hnd" else (page, slot)
            out[i] = decode(codes[at], None if scale is None else scale[at], self.kind)
        return out

    def cuda(self):
        for n in ("k", "v", "k_scale", "v_scale"):
            t = getattr(self, n)
            setattr(self, n, None if t is None else t.cuda())
        self.table_dev = self.table.cuda()
        return self


# ---- operators ------------------------------------------------------------
def matvec(q, s, x, y_dtype, add=None, eps=0.0):
    """(y, bound) of y = add + W f(x)."""
    w, x = decode(q, s, "int4g32"), x.double()
    k = x.shape[1]
    if eps:
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    y = x @ w.t()
    mags = x.abs() @ w.abs().t()
    # 32 products of a group on the tensor cores, then at most K / 32 groups and 3 x 8 warps' sums in fp32, each scaled once
    bound = mags * (2 * 34 + k / 32 + 3 * 8 + 2) * U
    if eps:
        bound = bound + y.abs() * (k / 256 + 16 + 4) * U
    if add is not None:
        y = y + add.double()
        bound = bound + y.abs() * U
    return y, bound + half_step(y.abs() + bound, y_dtype)


def norm_rotate(x, pos, rotary, pairs, theta, eps, weight):
    """(values, magnitudes of what each value is a sum of) of one token's heads [heads, dim]."""
    x = x.double()
    if eps:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    out, mag = x.clone(), x.abs()
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rotary // 2)
        # theta is an fp32 number for the library
        ang = pos * float(torch.tensor(theta, dtype=torch.float32)) ** (-2.0 * i / rotary)
        c, s = math.cos(ang), math.sin(ang)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, mag


def attention(cache, seq, length, q, window=0, scale=0.0, cap=0.0):
    """(out, lse, bound of out, bound of lse) of one sequence, q [heads, dim]."""
    heads, dim = q.shape
    if length == 0:
        return (torch.zeros(heads, dim, dtype=torch.float64), torch.full((heads,), -math.inf, dtype=torch.float64),
                torch.zeros(heads, dim, dtype=torch.float64), torch.zeros(heads, dtype=torch.float64))
    first = max(0, length - window) if window else 0
    k, v = cache.rows("k", seq, first, length), cache.rows("v", seq, first, length)
    group = heads // cache.heads
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    scale = scale or 1 / math.sqrt(dim)
    s = torch.einsum("hd,phd->hp", q.double(), k) * scale
    # a score: products of q to 22 bits (16 for a bf16 cache, 24 for fp32 inputs' sake left out) with exact codes; dim of
    # them summed on the tensor cores in fp32, scaled, and multiplied by log2 e
    parts = 2.0 ** -16 if cache.kind == "bf16" else 2.0 ** -21
    delta = torch.einsum("hd,phd->hp", q.double().abs(), k.abs()) * abs(scale) * ((2 * dim + 8) * U + parts) + s.abs() * 4 * U
    if cap:
        s = cap * torch.tanh(s / cap)
        delta = delta + cap * 2.0 ** -21
    p = torch.softmax(s, -1)
    out = torch.einsum("hp,phd->hd", p, v)
    n = length - first
    # a weight: exp2 (2^-21), its parts (as above), a correction by the running maximum for each tile; sums of n terms
    rel = 2 * delta.amax(-1, keepdim=True) + 2.0 ** -21 + parts + (2 * n / 16 + 80) * U
    mags = torch.einsum("hp,phd->hd", p, v.abs())
    # parts of weights below the fp16 range: n times 2^-38 of the largest value
    bound = mags * rel + v.abs().amax() * n * 2.0 ** -38
    return out, torch.logsumexp(s, -1), bound, rel[:, 0] + torch.logsumexp(s, -1).abs() * 4 * U + 2.0 ** -20
