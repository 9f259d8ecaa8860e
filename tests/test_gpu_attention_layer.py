"""The attention half of a decode layer as it is used: projections, cache write,
attention and the projection onto the residual one after the other, with the
library's sparse FFN behind them, eager and replayed from a graph; and the paths
of the single kernels that only larger sizes take.

Every stage is held to its 64-bit definition (attn_ref.py) on the inputs that it
really had, which are the outputs of the kernel before it."""
import math

import pytest
import torch

import attn_ref as R
import gpu_util as G
from activation_sparse_decode_threshold_b200 import binding as B
from activation_sparse_decode_threshold_b200 import synth
from test_gpu_attention import append_case, attend, cache_of, check, check_attention, gen, layer, made, matrix  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


class Layer:
    """One layer's matrices and cache, and a buffer for each stage."""

    def __init__(self, made, g, d, heads, kv_heads, dim, cache, page, lens, tokens, io):
        self.heads, self.kv_heads, self.dim, self.io = heads, kv_heads, dim, io
        n = (heads + 2 * kv_heads) * dim
        self.w = [R.encode_int4(torch.randn(a, b, generator=g) / math.sqrt(b)) for a, b in ((n, d), (d, heads * dim))]
        self.m = [matrix(made, *w) for w in self.w]
        self.c = R.Cache(g, lens, kv_heads, dim, cache, page).cuda()
        self.cache = cache_of(self.c)
        self.norms = [(1 + 0.2 * torch.randn(dim, generator=g)).cuda() for _ in range(2)]
        mk = lambda *s: torch.zeros(*s, dtype=R.DT[io], device="cuda")  # noqa: E731
        self.qkv, self.q, self.o = mk(tokens, n), mk(tokens, heads, dim), mk(tokens, heads * dim)

    def step(self, a, r, pos, lens):
        h, k, d = self.heads, self.kv_heads, self.dim
        t = r.shape[0]
        part = lambda i, n: self.qkv[:, i * d:(i + n) * d].unflatten(1, (n, d))  # noqa: E731
        B.pi_int4_matvec(self.m[0], r, self.qkv, norm_eps=1e-6)
        B.pi_kv_append(a, self.cache, self.c.table_dev, pos, part(0, h), part(h, k), part(h + k, k), self.q,
                       q_norm=self.norms[0], k_norm=self.norms[1])
        B.pi_paged_attention(a, self.cache, self.c.table_dev, lens, self.q, self.o.unflatten(1, (h, d)))
        B.pi_int4_matvec(self.m[1], self.o, r, add=r)
        assert t == self.q.shape[0]

    def check(self, r_in, r_out, pos, lens, theta):
        h, k, d, io = self.heads, self.kv_heads, self.dim, R.DT[self.io]
        qkv, q, o = self.qkv.cpu(), self.q.cpu(), self.o.cpu()
        want, bound = R.matvec(*self.w[0], r_in, io, None, 1e-6)
        check(qkv, want, bound, "qkv")
        for t, p in enumerate(pos):
            x, mag = R.norm_rotate(qkv[t, :h * d].view(h, d), p, d, False, theta, 1e-6, self.norms[0].cpu())
            check(q[t], x, mag * (d / 32 + 5 + 8 + 6) * R.U + R.half_step(x, io), "q")
            x, _ = R.norm_rotate(qkv[t, h * d:(h + k) * d].view(k, d), p, d, False, theta, 1e-6, self.norms[1].cpu())
            for name, w in (("k", x), ("v", qkv[t, (h + k) * d:].view(k, d).double())):
                got = self.c.rows(name, t, p, p + 1)[0]
                codes, scale = R.encode(w, self.c.kind)
                exact = R.decode(codes, scale, self.c.kind)
                if scale is None:
                    check(got, w, R.half_step(w, R.DT[self.c.kind]) + w.abs() * R.U, name)
                else:
                    assert torch.equal(got, exact), name
        check_attention(self.c, lens, q, self.o.unflatten(1, (h, d)), self.lse(lens, q))
        want, bound = R.matvec(*self.w[1], o, torch.float32, r_in)
        check(r_out, want, bound, "residual")

    def lse(self, lens, q):
        return torch.stack([R.attention(self.c, s, n, q[s])[1].float() for s, n in enumerate(lens)])


@pytest.mark.parametrize("cache,io,tokens", [("bf16", "bf16", 3), ("f16", "f16", 1), ("i8", "f16", 5), ("int4g32", "f16", 2)])
def test_decode_steps_of_two_layers(made, cache, io, tokens):
    """Steps of growing texts through two layers on one handle, the sparse FFN behind each: first eager, then the same
    calls of the attention half replayed from a graph."""
    g = gen(tokens)
    cfg = synth.small(synth.CONFIGS["llama7b"], n_layers=2, d=512, F=1000, rank=64)
    ffn = G.create(cfg)
    for i in range(2):
        G.load(ffn, i, synth.make_layer(cfg, i, device="cuda"))
    heads, kv_heads, dim, page, theta = 6, 2, 64, 16, 10000.0
    lens = [29 + 7 * s for s in range(tokens)]
    room = [n + 8 for n in lens]
    a = layer(made, heads, kv_heads, dim, cache_dtype=cache, page_size=page, rotary_dim=dim, rope_theta=theta, norm_eps=1e-6)
    layers = [Layer(made, g, cfg.d, heads, kv_heads, dim, cache, page, room, tokens, io) for _ in range(2)]
    r = torch.randn(tokens, cfg.d, generator=g).cuda()
    pos, lens_dev = (torch.zeros(tokens, dtype=torch.int32, device="cuda") for _ in range(2))
    try:
        graphs = None
        for step in range(4):
            now = [n + step for n in lens]
            pos.copy_(torch.tensor(now))
            lens_dev.copy_(torch.tensor([n + 1 for n in now]))
            if step == 2:
                graphs = []
                for la in layers:
                    gr = torch.cuda.CUDAGraph()
                    keep = r.clone()
                    with torch.cuda.graph(gr):
                        la.step(a, r, pos, lens_dev)
                    r.copy_(keep)
                    graphs.append(gr)
            for i, la in enumerate(layers):
                before = r.clone()
                if graphs:
                    graphs[i].replay()
                else:
                    la.step(a, r, pos, lens_dev)
                after = r.clone()
                B.pi_sparse_ffn_decode_batch(ffn, i, i + 1, r)
                torch.cuda.synchronize()
                assert B.pi_attn_sync(a) == B.PI_OK and B.pi_sync(ffn) == B.PI_OK
                la.check(before.cpu(), after, now, [n + 1 for n in now], theta)
                alone = after.clone()
                B.pi_sparse_ffn_decode_batch(ffn, i, i + 1, alone)
                assert torch.equal(alone, r) and not torch.equal(r, after)
    finally:
        torch.cuda.synchronize()
        B.pi_ffn_destroy(ffn)


def test_steps_without_waiting_give_what_waiting_gives(made):
    """A hundred dependent calls in a row, each on the outputs of the one before, against the same with a wait after
    each: the same bits."""
    g = gen(42)
    heads, kv_heads, dim, d = 4, 4, 64, 256
    a = layer(made, heads, kv_heads, dim, cache_dtype="f16", page_size=8, rotary_dim=dim, norm_eps=1e-6)
    la = Layer(made, g, d, heads, kv_heads, dim, "f16", 8, [40, 40], 2, "f16")
    start = torch.randn(2, d, generator=g).cuda()
    empty = {n: getattr(la.c, n).clone() for n in ("k", "v")}
    got = []
    for wait in (True, False, False):
        for n, t in empty.items():
            getattr(la.c, n).copy_(t)
        r = start.clone()
        places = [torch.full((2,), i, dtype=torch.int32, device="cuda") for i in range(27)]
        torch.cuda.synchronize()
        for i in range(25):
            la.step(a, r, places[i], places[i + 1])
            r.mul_(0.5)
            if wait:
                torch.cuda.synchronize()
        got.append((r.clone(), la.c.k.clone()))
    for x, y in got[1:]:
        assert torch.equal(x, got[0][0]) and torch.equal(y, got[0][1])


# ---------------------------------------------------------------------------
# sizes that take other paths
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,k,tokens,x,y,eps,add", [
    (40000, 64, 1, "f16", "f16", 0.0, False),        # more row tiles than a CTA takes at once
    (38000, 96, 7, "f32", "f32", 1e-6, True),
    (600, 16384, 13, "bf16", "f32", 0.0, True),      # columns over a cluster
    (9000, 4096, 32, "f32", "f32", 1e-6, False),     # over a cluster, in several passes and rounds
    (300, 16416, 24, "f32", "bf16", 1e-6, True),     # parts of unequal size
    (2000, 65536, 4, "f16", "f32", 1e-6, False),
    (16, 131072, 32, "f32", "f32", 0.0, False),
])
def test_matvec_large(made, n, k, tokens, x, y, eps, add):
    g = torch.Generator(device="cuda").manual_seed(n + k)
    q, s = R.encode_int4(torch.randn(n, k, generator=g, device="cuda") * 0.05)
    xv = torch.randn(tokens, k, generator=g, device="cuda").to(R.DT[x])
    av = torch.randn(tokens, n, generator=g, device="cuda").to(R.DT[y]) if add else None
    m = matrix(made, q, s)
    out = torch.full((tokens, n), 7.0, dtype=R.DT[y], device="cuda")
    B.pi_int4_matvec(m, xv, out, add=av, norm_eps=eps)
    want, bound = R.matvec(q, s, xv, R.DT[y], av, eps)
    check(out, want.cpu(), bound.cpu())
    again = torch.zeros_like(out)
    B.pi_int4_matvec(m, xv, again, add=av, norm_eps=eps)
    assert torch.equal(out, again)


@pytest.mark.parametrize("cache,io,dim,rotary,pairs,eps,layout", [
    ("int4g32", "f16", 128, 128, False, 1e-6, "hnd"), ("i8", "bf16", 64, 64, True, 1e-6, "nhd"),
    ("bf16", "bf16", 64, 32, False, 0.0, "hnd"), ("f16", "f32", 128, 50, True, 1e-6, "nhd"),
    ("int4g32", "f32", 64, 0, False, 0.0, "hnd"), ("i8", "f32", 128, 6, False, 0.0, "hnd")])
def test_append_of_many_tokens(made, cache, io, dim, rotary, pairs, eps, layout):
    """More tokens than the GPU has SMs; heads that do not fill a warp's last vectors."""
    n = torch.cuda.get_device_properties(0).multi_processor_count + 13
    pos = [3 * i % 400 for i in range(n)]
    pos = [p if i % 17 else -1 for i, p in enumerate(pos)]
    append_case(made, io, cache, 9, 3, dim, 16, rotary, pairs, eps, layout, pos)


@pytest.mark.parametrize("lens", [[3000], [1500, 3, 0, 700]])
@pytest.mark.parametrize("cache,io,dim,kv_heads,group", [
    ("bf16", "bf16", 128, 2, 8), ("f16", "f16", 128, 1, 16), ("i8", "f16", 128, 2, 6), ("int4g32", "f16", 128, 1, 12),
    ("int4g32", "bf16", 64, 2, 8), ("f16", "f32", 64, 1, 7), ("bf16", "bf16", 64, 2, 16), ("i8", "bf16", 128, 1, 20),
    ("int4g32", "f32", 64, 1, 16), ("i8", "f32", 64, 3, 5)])
def test_attention_groups_over_many_warps(made, lens, cache, io, dim, kv_heads, group):
    c = R.Cache(gen(dim + group), lens, kv_heads, dim, cache, 32).cuda()
    a, q, out, lse = attend(made, c, lens, kv_heads * group, io)
    assert B.pi_attn_sync(a) == B.PI_OK
    check_attention(c, lens, q, out, lse)
    again, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    B.pi_paged_attention(a, cache_of(c), c.table_dev, torch.tensor(lens, dtype=torch.int32).cuda(), q.cuda(), again, lse=l2)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("cache", ["i8", "int4g32"])
def test_attention_rows_of_zeros(made, cache):
    """Rows with scale 0: alone in a text, before others and behind them."""
    lens = [40, 70, 70]
    c = R.Cache(gen(21), lens, 2, 128, cache, 16)
    for s, rows in ((0, range(40)), (1, range(33)), (2, range(50, 70))):
        for p in rows:
            page, slot = int(c.table[s, p // 16]), p % 16
            c.v_scale[page, :, slot] = 0
            c.k_scale[page, :, slot] = 0
            if cache == "i8":
                c.v[page, :, slot] = c.k[page, :, slot] = 0
            else:
                c.v[page, :, slot] = c.k[page, :, slot] = 0x88
    c.cuda()
    a, q, out, lse = attend(made, c, lens, 8, "f32")
    assert (out[0] == 0).all()
    check_attention(c, lens, q, out, lse)


def test_attention_an_infinite_scale_spoils_its_group_only(made):
    lens = [60, 60]
    for dim in (64, 128):
        c = R.Cache(gen(22), lens, 1, dim, "int4g32", 16)
        full = R.Cache(gen(22), lens, 1, dim, "int4g32", 16)
        page, slot = int(c.table[0, 2]), 5
        c.v_scale[page, 0, slot, 1] = INF
        c.v[page, 0, slot, 16:32] = 0x99      # codes of 1
        c.cuda()
        a, q, out, lse = attend(made, c, lens, 3, "f32")
        out = out.cpu()
        assert not out[0, :, 32:64].isfinite().any()
        for s in range(2):
            want, _, bound, _ = R.attention(full, s, 60, q[s])
            keep = [i for i in range(dim) if s or not 32 <= i < 64]
            check(out[s][:, keep], want[:, keep], bound[:, keep] + R.half_step(want[:, keep], torch.float32))


@pytest.mark.parametrize("cap", [1e-6, 0.5, 30.0, 64.0, 65.0, 1000.0, 1e6])
def test_capped_scores_of_all_sizes(made, cap):
    """One position: the log of the sum is its capped score.  Up to 64 the cap's formula is off by cap 2^-21, above it the
    score by a few of its own roundings (tanh 2 units of 2^-23, five products of 2^-24, products of 22 bits and their sum
    of 64 in 24)."""
    lens = [1, 1, 1]
    c = R.Cache(gen(31), lens, 1, 64, "f16", 8).cuda()
    for size in (0.01, 1.0, 40.0):
        q = size * torch.randn(3, 4, 64, generator=gen(32))
        a, q, out, lse = attend(made, c, lens, 4, "f32", q=q, softcap=cap)
        for s in range(3):
            k = c.rows("k", s, 0, 1)[0, 0]
            x = (q[s].double() @ k) / 8
            noise = (q[s].double().abs() @ k.abs()) / 8 * (2.0 ** -21 + 136 * R.U)
            want = cap * torch.tanh(x / cap)
            check(lse[s], want, noise + want.abs() * (2.0 ** -21 + 8 * R.U) + (cap * 2.0 ** -21 if cap <= 64 else 0.0), f"cap {cap} size {size}")


def test_sequences_that_share_pages(made):
    """A prefix in the pages of two sequences, read by both."""
    c = R.Cache(gen(23), [64, 64], 2, 64, "bf16", 16)
    c.table[1, :3] = c.table[0, :3]
    c.cuda()
    lens = [55, 64]
    a, q, out, lse = attend(made, c, lens, 4, "bf16")
    check_attention(c, lens, q, out, lse)


def test_two_handles_on_two_streams_at_once(made):
    """Attention calls of two handles that overlap on the GPU, many times: the bits of each alone."""
    lens = [700, 3, 250]
    c = R.Cache(gen(24), lens, 2, 64, "f16", 16).cuda()
    cache, n = cache_of(c), torch.tensor(lens, dtype=torch.int32).cuda()
    hs = [layer(made, 8, 2, 64, cache_dtype="f16", page_size=16) for _ in range(2)]
    qs = [torch.randn(3, 8, 64, generator=gen(i)).half().cuda() for i in range(2)]
    want = [torch.zeros_like(qs[0]) for _ in range(2)]
    for a, q, o in zip(hs, qs, want):
        B.pi_paged_attention(a, cache, c.table_dev, n, q, o)
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(qs[0]) for _ in range(8)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(8):
        for i in range(2):
            B.pi_paged_attention(hs[i], cache, c.table_dev, n, qs[i], outs[i][j], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_refused_sizes(made):
    c = R.Cache(gen(1), [20], 1, 64, "f16", 256).cuda()
    a = layer(made, 1, 1, 64, cache_dtype="f16", page_size=256)
    q, o = torch.zeros(1, 1, 64, device="cuda"), torch.zeros(1, 1, 64, device="cuda")
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(1, 2 ** 22 + 1, dtype=torch.int32, device="cuda")
    many = torch.zeros(65537, 1, dtype=torch.int32, device="cuda")
    for table, lens in ((wide, n), (many, n.expand(65537).contiguous())):
        with pytest.raises(B.PiError) as e:
            B.pi_paged_attention(a, cache_of(c), table, lens, q.expand(table.shape[0], 1, 64).contiguous(),
                                 o.expand(table.shape[0], 1, 64).contiguous())
        assert e.value.status == B.PI_ERR_INVALID_ARG
    with pytest.raises(B.PiError):
        B.pi_kv_read(a, cache_of(c), wide, n, q, o)
    # tiles of work beyond 2^30: 65536 sequences of 2^20 positions
    tall = torch.zeros(65536, 2 ** 12, dtype=torch.int32, device="cuda")
    with pytest.raises(B.PiError) as e:
        B.pi_paged_attention(a, cache_of(c), tall, n.expand(65536).contiguous(), q.expand(65536, 1, 64).contiguous(),
                             o.expand(65536, 1, 64).contiguous())
    assert e.value.status == B.PI_ERR_INVALID_ARG


@pytest.mark.parametrize("cap", [1e-7, 1e7, -INF])
def test_caps_out_of_range_are_refused(cap):
    with pytest.raises(B.PiError) as e:
        B.pi_attn_create(4, 2, 64, softcap=cap)
    assert e.value.status == B.PI_ERR_INVALID_ARG
