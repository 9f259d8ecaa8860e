"""The attention half of a decode layer (pi_int4_matvec, pi_kv_append, pi_kv_read,
pi_paged_attention) against plain 64-bit definitions (attn_ref.py), at the sizes,
types and masks where it can go wrong."""
import math

import pytest
import torch

import attn_ref as R
from activation_sparse_decode_threshold_b200 import binding as B

pytestmark = pytest.mark.gpu
NAN, INF = math.nan, math.inf


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check(got, want, bound, what=""):
    got, off = got.cpu().double(), None
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine), what
    off = (got - want).abs()[fine]
    over = off > bound.expand_as(want)[fine]
    assert not over.any(), f"{what}: off by {off[over].max():.3e}, bound {bound.expand_as(want)[fine][over].min():.3e}"


@pytest.fixture
def made():
    """Handles to release at the end of a test."""
    got = []
    yield got
    torch.cuda.synchronize()
    for release, h in got:
        release(h)


def matrix(made, q, s):
    m = B.pi_int4_create(q.cuda(), s.cuda())
    made.append((B.pi_int4_destroy, m))
    return m


def layer(made, heads, kv_heads, dim, **kw):
    a = B.pi_attn_create(heads, kv_heads, dim, **kw)
    made.append((B.pi_attn_destroy, a))
    return a


def cache_of(c):
    return B.pi_kv_cache(c.k, c.v, c.k_scale, c.v_scale)


# ---------------------------------------------------------------------------
# pi_int4_matvec
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,k,tokens,x,y,eps,add", [
    (1, 32, 1, "f32", "f32", 0.0, False),            # the least matrix
    (16, 64, 1, "f16", "f16", 1e-6, False),
    (17, 96, 2, "bf16", "bf16", 0.0, True),          # a row and half a unit over
    (250, 1056, 3, "f32", "f32", 1e-5, True),
    (33, 4128, 1, "f32", "f32", 1e-6, False),
    (1024, 4096, 1, "f16", "f32", 0.0, False),
    (100, 512, 8, "bf16", "f32", 1e-6, True),
    (64, 544, 9, "f16", "f16", 0.0, False),
    (48, 2080, 13, "f32", "bf16", 0.0, True),
    (31, 14336, 5, "bf16", "bf16", 0.0, False),
    (130, 8192, 32, "f32", "f32", 1e-6, False),
    (65, 1600, 32, "f16", "f16", 0.0, True),
    (8, 131072, 1, "f32", "f32", 0.0, False),        # the longest row
    (19, 32768, 32, "bf16", "f32", 1e-6, False),
    (2500, 320, 1, "bf16", "bf16", 0.0, False),
])
def test_matvec(made, n, k, tokens, x, y, eps, add):
    g = gen(n + k)
    q, s = R.encode_int4(torch.randn(n, k, generator=g) * 0.05)
    xv = (torch.randn(tokens, k, generator=g) * torch.exp(torch.randn(tokens, 1, generator=g))).to(R.DT[x])
    av = torch.randn(tokens, n, generator=g).to(R.DT[y]) if add else None
    m = matrix(made, q, s)
    out = torch.full((tokens, n), 7.0, dtype=R.DT[y], device="cuda")
    B.pi_int4_matvec(m, xv.cuda(), out, add=av.cuda() if add else None, norm_eps=eps)
    want, bound = R.matvec(q, s, xv, R.DT[y], av, eps)
    check(out, want, bound)


def test_matvec_in_place_with_row_distances(made):
    g = gen(3)
    n, k, t = 40, 160, 6
    q, s = R.encode_int4(torch.randn(n, k, generator=g))
    x = torch.randn(t, k + 24, generator=g)
    y = torch.randn(t, n + 3, generator=g)
    m = matrix(made, q, s)
    xd, yd = x.cuda(), y.cuda()
    B.pi_int4_matvec(m, xd[:, 8:8 + k], yd[:, 1:1 + n], add=yd[:, 1:1 + n])
    want, bound = R.matvec(q, s, x[:, 8:8 + k], torch.float32, y[:, 1:1 + n])
    check(yd[:, 1:1 + n], want, bound)
    assert torch.equal(yd[:, 0].cpu(), y[:, 0]) and torch.equal(yd[:, n + 1:].cpu(), y[:, n + 1:])   # nothing beside


def test_matvec_tokens_do_not_touch_each_other(made):
    """A token's bits are the same alone and in a batch with NaN, infinities and the largest numbers beside it."""
    g = gen(4)
    n, k = 70, 416
    q, s = R.encode_int4(torch.randn(n, k, generator=g))
    m = matrix(made, q, s)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        x = torch.randn(5, k, generator=g).to(dt).cuda()
        x[0, 3], x[1, 5], x[3, :] = NAN, INF, torch.finfo(dt).max
        both, alone = torch.zeros(5, n, device="cuda"), torch.zeros(1, n, device="cuda")
        B.pi_int4_matvec(m, x, both)
        assert both[0].isnan().all()
        for t in (2, 4):
            B.pi_int4_matvec(m, x[t:t + 1], alone)
            assert torch.equal(both[t], alone[0])
        # an infinity times a positive, a negative and a zero weight
        w5 = R.decode(q, s, "int4g32")[:, 5]
        assert torch.equal(both[1].cpu() == INF, w5 > 0) and torch.equal(both[1].cpu() == -INF, w5 < 0)
        assert torch.equal(both[1].cpu().isnan(), w5 == 0)


def test_matvec_small_numbers_keep_their_digits(made):
    q, s = R.encode_int4(torch.randn(20, 64, generator=gen(6)))
    m = matrix(made, q, s)
    x = torch.randn(1, 64, generator=gen(7)) * 1e-30
    y = torch.zeros(1, 20, device="cuda")
    B.pi_int4_matvec(m, x.cuda(), y)
    want, bound = R.matvec(q, s, x, torch.float32)
    check(y, want, bound)


def test_matvec_streams_graph_and_repeat(made):
    """The same bits on a stream of its own, twice at once, and replayed from a graph with new inputs."""
    g = gen(8)
    q, s = R.encode_int4(torch.randn(500, 2048, generator=g))
    m = matrix(made, q, s)
    xs = [torch.randn(1, 2048, generator=g).cuda() for _ in range(4)]
    want = []
    for x in xs:
        y = torch.zeros(1, 500, device="cuda")
        B.pi_int4_matvec(m, x, y, norm_eps=1e-6)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    ys = [torch.zeros(1, 500, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, x, y in zip(streams, xs, ys):
            B.pi_int4_matvec(m, x, y, norm_eps=1e-6, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, ys))
    x, y = xs[0].clone(), torch.zeros(1, 500, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.pi_int4_matvec(m, x, y, norm_eps=1e-6)
    for i in (2, 0, 3):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(y, want[i])


# ---------------------------------------------------------------------------
# pi_kv_append
# ---------------------------------------------------------------------------
def append_case(made, io, cache, heads, kv_heads, dim, page, rotary, pairs, eps, layout, pos, seq=None, weights=True,
                theta=10000.0, seed=1):
    g = gen(seed)
    t = len(pos)
    n_seqs = t if seq is None else max(seq) + 1
    lens = [1 + max([p for i, p in enumerate(pos) if (i if seq is None else seq[i]) == s] + [0]) for s in range(n_seqs)]
    c = R.Cache(g, lens, kv_heads, dim, cache, page, layout, fill=True).cuda()
    before = {n: None if getattr(c, n) is None else getattr(c, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    total = (heads + 2 * kv_heads) * dim
    qkv = torch.randn(t, total + 64, generator=g).to(R.DT[io])
    qw, kw = (1 + 0.3 * torch.randn(dim, generator=g) for _ in range(2)) if eps and weights else (None, None)
    a = layer(made, heads, kv_heads, dim, cache_dtype=cache, page_size=page, layout=layout, rotary_dim=rotary,
              rotary_pairs=pairs, rope_theta=theta, norm_eps=eps)
    d = qkv.cuda()
    cut = lambda x, i, n: x[:, i * dim:(i + n) * dim].unflatten(1, (n, dim))  # noqa: E731
    out = torch.full((t, heads, dim), 9.0, dtype=R.DT[io], device="cuda")
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    B.pi_kv_append(a, cache_of(c), c.table_dev, torch.tensor(pos, dtype=torch.int32).cuda(), cut(d, 0, heads),
                   cut(d, heads, kv_heads), cut(d, heads + kv_heads, kv_heads), out,
                   seq=None if seq is None else torch.tensor(seq, dtype=torch.int32).cuda(), q_norm=dev(qw), k_norm=dev(kw))
    assert B.pi_attn_sync(a) == B.PI_OK
    # the queries
    written = {}
    for i, p in enumerate(pos):
        if p < 0:
            assert (out[i] == 9.0).all()
            continue
        q, mag = R.norm_rotate(cut(qkv, 0, heads)[i], p, rotary, pairs, theta, eps, qw)
        # norm: a sum of dim squares, a root, a quotient, two products; rotation: two products and a sum, angles in 64 bits
        check(out[i], q, mag * (dim / 32 + 5 + 8 + 6) * R.U + R.half_step(q, R.DT[io]), f"q {i}")
        k, _ = R.norm_rotate(cut(qkv, heads, kv_heads)[i], p, rotary, pairs, theta, eps, kw)
        s = i if seq is None else seq[i]
        written[(int(c.table[s, p // page]), p % page)] = (k, cut(qkv, heads + kv_heads, kv_heads)[i].double())
    # the cache: the rows written, and every other row as it was
    for name, j in (("k", 0), ("v", 1)):
        codes, scale = getattr(c, name).cpu(), getattr(c, name + "_scale")
        want, wscale = before[name].cpu(), before[name + "_scale"]
        for (pg, slot), kv in written.items():
            at = (pg, slice(None), slot) if layout == "hnd" else (pg, slot)
            e, es = R.encode(kv[j], cache)
            if cache in ("f16", "bf16") and j == 0:
                # 64 bits rounded by way of fp32: half a step, and 2^-24
                check(codes[at], kv[j], R.half_step(kv[j], R.DT[cache]) + kv[j].abs() * R.U, "k")
                e = codes[at]
            want[at] = e
            if es is not None:
                wscale[at] = es.to(wscale.device)
        assert torch.equal(codes, want), f"{name}: {(codes != want).sum()} codes differ"
        assert scale is None or torch.equal(scale, wscale)
    return c, a


@pytest.mark.parametrize("cache", ["f16", "bf16", "i8", "int4g32"])
@pytest.mark.parametrize("dim,rotary,pairs,eps", [(128, 128, False, 1e-6), (64, 64, True, 0.0), (128, 34, False, 0.0),
                                                  (64, 0, False, 1e-5), (128, 96, True, 1e-6), (64, 2, False, 0.0)])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_append_formats(made, cache, dim, rotary, pairs, eps, layout):
    append_case(made, "bf16" if cache == "bf16" else "f16", cache, 6, 2, dim, 8, rotary, pairs, eps, layout, [0, 13, -1, 7])


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["f16", "bf16", "i8", "int4g32"])
def test_append_types(made, io, cache):
    append_case(made, io, cache, 4, 4, 128, 16, 128, False, 1e-6, "hnd", [5, 0, 31], weights=False)


def test_append_prompt_of_two_sequences_with_pads(made):
    """Tokens of two sequences in turn over page borders, empty places between them and behind."""
    pos = [i for i in range(3, 45) for _ in range(2)]
    seq = [s for _ in range(3, 45) for s in (1, 0)]
    for i in (5, 18, 80, 81, 83):
        pos[i] = -1
    append_case(made, "bf16", "int4g32", 8, 2, 64, 16, 64, False, 1e-6, "hnd", pos, seq)


def test_append_far_positions(made):
    """The angle of a far position: 64 bits hold it, 32 would be off by a hundredth of a turn."""
    append_case(made, "f32", "f16", 2, 1, 64, 256, 64, False, 0.0, "hnd", [1000003], theta=500000.0)


def test_append_one_head_and_many(made):
    append_case(made, "f16", "i8", 1, 1, 64, 8, 64, False, 0.0, "nhd", [2])
    append_case(made, "f16", "f16", 96, 8, 128, 32, 128, False, 1e-6, "hnd", [40])


def test_append_in_place(made):
    g = gen(5)
    a = layer(made, 4, 2, 64, cache_dtype="f16", page_size=8, rotary_dim=64)
    c = R.Cache(g, [8, 8], 2, 64, "f16", 8, fill=False).cuda()
    qkv = torch.randn(2, 8 * 64, generator=g).half().cuda()
    cut = lambda x, i, n: x[:, i * 64:(i + n) * 64].unflatten(1, (n, 64))  # noqa: E731
    pos = torch.tensor([3, 7], dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    rest = qkv[:, 4 * 64:].clone()
    B.pi_kv_append(a, cache_of(c), c.table_dev, pos, cut(qkv, 0, 4), cut(qkv, 4, 2), cut(qkv, 6, 2), out)
    B.pi_kv_append(a, cache_of(c), c.table_dev, pos, cut(qkv, 0, 4), cut(qkv, 4, 2), cut(qkv, 6, 2), cut(qkv, 0, 4))
    assert torch.equal(cut(qkv, 0, 4), out) and torch.equal(qkv[:, 4 * 64:], rest)


@pytest.mark.parametrize("cache", ["i8", "int4g32"])
def test_append_zero_tiny_and_not_finite(made, cache):
    """Rows of zeros, rows whose scale rounds to zero, infinities, NaN and rows too large for the scale."""
    g = gen(9)
    a = layer(made, 1, 1, 64, cache_dtype=cache, page_size=8)
    c = R.Cache(g, [8] * 6, 1, 64, cache, 8).cuda()
    v = torch.randn(6, 1, 64, generator=g)
    v[0], v[1] = 0.0, 1e-44 if cache == "i8" else 1e-8
    v[2, 0, 3], v[3, 0, 40], v[4] = INF, NAN, v[4] * (1e38 if cache == "i8" else 1e6)
    q = torch.zeros(6, 1, 64, device="cuda")
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    B.pi_kv_append(a, cache_of(c), c.table_dev, pos, q, v.cuda(), v.cuda(), torch.empty_like(q))
    ko, vo = torch.zeros_like(q), torch.zeros_like(q)
    B.pi_kv_read(a, cache_of(c), c.table_dev, pos, ko, vo)
    assert B.pi_attn_sync(a) == B.PI_OK
    codes, s = R.encode(v[[0, 1, 5]], cache)
    want = R.decode(codes, s, cache)
    for out in (ko.cpu(), vo.cpu()):
        assert torch.equal(out[[0, 1, 5]].double(), want.float().double())
        if cache == "i8":
            assert out[2:4].isnan().all() and out[4].isfinite().all()
        else:
            assert out[2, 0, :32].isnan().all() and out[2, 0, 32:].isfinite().all()
            assert out[3, 0, 32:].isnan().all() and out[3, 0, :32].isfinite().all()
            assert out[4].isnan().all()


def test_append_and_read_report_what_is_out_of_range(made):
    """Bad sequences, positions and pages: skipped and reported; the other tokens are done."""
    g = gen(10)
    a = layer(made, 2, 2, 64, cache_dtype="f16", page_size=8)
    c = R.Cache(g, [16, 16, 16], 2, 64, "f16", 8).cuda()
    c.table_dev[1, 1] = c.pages
    c.table_dev[2, 0] = -7
    seq = torch.tensor([0, 3, -1, 0, 1, 2, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([15, 0, 0, 16, 8, 3, 7], dtype=torch.int32, device="cuda")
    before = c.k.clone()
    x = torch.randn(7, 2, 64, generator=g).half().cuda()
    out = torch.full_like(x, 5.0)
    B.pi_kv_append(a, cache_of(c), c.table_dev, pos, x, x, x, out, seq=seq)
    assert B.pi_attn_sync(a) == B.PI_ERR_DEVICE_CHECK
    assert B.pi_attn_sync(a) == B.PI_OK
    for i, (s, p) in enumerate([(0, 15), None, None, None, None, None, (1, 7)][j] or (-1, -1) for j in range(7)):
        if s < 0:
            assert (out[i] == 5.0).all()
        else:
            assert torch.equal(out[i], x[i])
            before[int(c.table[s, p // 8]), :, p % 8] = x[i]
    assert torch.equal(c.k, before)
    ko, vo = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
    B.pi_kv_read(a, cache_of(c), c.table_dev, pos, ko, vo, seq=seq)
    assert B.pi_attn_sync(a) == B.PI_ERR_DEVICE_CHECK
    for i in range(7):
        assert torch.equal(ko[i], x[i]) if i in (0, 6) else (ko[i] == 3.0).all()


# ---------------------------------------------------------------------------
# pi_kv_read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["f16", "bf16", "i8", "int4g32"])
@pytest.mark.parametrize("dim,kv_heads,page,layout", [(64, 3, 8, "hnd"), (128, 1, 32, "nhd"), (128, 5, 16, "hnd")])
def test_read(made, io, cache, dim, kv_heads, page, layout):
    """The values that rows stand for, rounded once: the same bits as the plain product of code and scale."""
    g = gen(dim + kv_heads)
    c = R.Cache(g, [70, 1, 33], kv_heads, dim, cache, page, layout).cuda()
    a = layer(made, 2 * kv_heads, kv_heads, dim, cache_dtype=cache, page_size=page, layout=layout)
    seq = [0, 2, 1, 0, 0, 2, 0]
    pos = [69, 32, 0, 0, 8, -1, 69]     # one row twice
    ko = torch.full((7, kv_heads, dim), 4.0, dtype=R.DT[io], device="cuda")
    vo = ko.clone()
    B.pi_kv_read(a, cache_of(c), c.table_dev, torch.tensor(pos, dtype=torch.int32).cuda(), ko, vo,
                 seq=torch.tensor(seq, dtype=torch.int32).cuda())
    assert B.pi_attn_sync(a) == B.PI_OK
    for name, out in (("k", ko), ("v", vo)):
        for i, (s, p) in enumerate(zip(seq, pos)):
            if p < 0:
                assert (out[i] == 4.0).all()
            else:
                want = c.rows(name, s, p, p + 1)[0].float().to(R.DT[io])
                assert torch.equal(out[i].cpu(), want)


def test_read_many_rows(made):
    g = gen(2)
    c = R.Cache(g, [700, 333], 2, 64, "int4g32", 16).cuda()
    a = layer(made, 4, 2, 64, cache_dtype="int4g32", page_size=16)
    pos = torch.cat((torch.arange(700), torch.arange(333))).int()
    seq = torch.cat((torch.zeros(700), torch.ones(333))).int()
    ko = torch.zeros(1033, 2, 64, device="cuda")
    vo = torch.zeros_like(ko)
    B.pi_kv_read(a, cache_of(c), c.table_dev, pos.cuda(), ko, vo, seq=seq.cuda())
    for name, out in (("k", ko), ("v", vo)):
        want = torch.cat((c.rows(name, 0, 0, 700), c.rows(name, 1, 0, 333)))
        assert torch.equal(out.cpu(), want.float())


# ---------------------------------------------------------------------------
# pi_paged_attention
# ---------------------------------------------------------------------------
def attend(made, c, lens, heads, io, q=None, seed=0, **kw):
    g = gen(seed + 77)
    a = layer(made, heads, c.heads, c.dim, cache_dtype=c.kind, page_size=c.page, layout=c.layout, **kw)
    if q is None:
        q = (2 * torch.randn(len(lens), heads, c.dim, generator=g)).to(R.DT[io])
    out = torch.full((len(lens), heads, c.dim), 9.0, dtype=R.DT[io], device="cuda")
    lse = torch.full((len(lens), heads), 9.0, device="cuda")
    B.pi_paged_attention(a, cache_of(c), c.table_dev, torch.tensor(lens, dtype=torch.int32).cuda(), q.cuda(), out, lse=lse)
    return a, q, out, lse


def check_attention(c, lens, q, out, lse, **kw):
    dt = out.dtype
    for s, n in enumerate(lens):
        want, l, bound, lb = R.attention(c, s, n, q[s], window=kw.get("window", 0), scale=kw.get("scale", 0.0),
                                         cap=kw.get("softcap", 0.0))
        check(out[s], want, bound + R.half_step(want.abs() + bound, dt), f"out of sequence {s} ({n})")
        if n == 0:
            assert (lse[s] == -INF).all() and (out[s] == 0).all()
        else:
            check(lse[s], l, lb, f"lse of sequence {s} ({n})")


@pytest.mark.parametrize("cache,io", [("f16", "f16"), ("bf16", "bf16"), ("i8", "f16"), ("int4g32", "f16"), ("i8", "bf16"),
                                      ("int4g32", "f32"), ("f16", "f32"), ("bf16", "f32"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("dim,kv_heads,group", [(64, 2, 1), (128, 1, 4), (128, 2, 8), (64, 1, 16), (128, 1, 13), (64, 3, 7),
                                                (128, 1, 16), (64, 1, 24)])
def test_attention_formats_and_groups(made, cache, io, dim, kv_heads, group):
    lens = [100, 0, 1, 37, 16]
    c = R.Cache(gen(dim + group), lens, kv_heads, dim, cache, 8).cuda()
    a, q, out, lse = attend(made, c, lens, kv_heads * group, io)
    assert B.pi_attn_sync(a) == B.PI_OK
    check_attention(c, lens, q, out, lse)


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "i8", "int4g32"])
def test_attention_pages(made, cache, page, layout):
    """Lengths around every border of pages and of tiles of 16 and 32 positions."""
    lens = [7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 300]
    c = R.Cache(gen(page), lens, 2, 64, cache, page, layout).cuda()
    a, q, out, lse = attend(made, c, lens, 8, "bf16")
    assert B.pi_attn_sync(a) == B.PI_OK
    check_attention(c, lens, q, out, lse)


@pytest.mark.parametrize("window", [1, 2, 8, 16, 17, 63, 200, 100000])
@pytest.mark.parametrize("cache", ["f16", "i8", "int4g32"])
def test_attention_window_and_cap(made, cache, window):
    """Rows before the window are not read: their pages are taken out of the table, or hold NaN."""
    lens = [1, 2, 17, 64, 65, 200, 333, 0]
    c = R.Cache(gen(window), lens, 1, 128, cache, 16)
    full = R.Cache(gen(window), lens, 1, 128, cache, 16)
    for s, n in enumerate(lens):
        gone = max(0, n - window)
        for p in range(gone):
            page, slot = int(c.table[s, p // 16]), p % 16
            if cache == "f16":
                c.k[page, :, slot], c.v[page, :, slot] = NAN, NAN
            else:
                c.k_scale[page, :, slot], c.v_scale[page, :, slot] = NAN, NAN
        c.table[s, :gone // 16] = -1
    c.cuda()
    for cap in (0.0, 5.0):
        a, q, out, lse = attend(made, c, lens, 4, "f16", window=window, softcap=cap)
        assert B.pi_attn_sync(a) == B.PI_OK
        check_attention(full, lens, q, out, lse, window=window, softcap=cap)


def test_attention_rows_behind_the_end_do_not_count(made):
    """NaN and infinities in the rest of the last page, in other pages and behind the last sequence's table."""
    for cache in ("f16", "bf16", "i8", "int4g32"):
        lens = [5, 40, 0]
        c = R.Cache(gen(1), lens, 2, 128, cache, 32)
        for name in ("k", "v"):
            t = getattr(c, name) if cache in ("f16", "bf16") else getattr(c, name + "_scale")
            keep = t.clone()
            t[...] = NAN if name == "k" else INF
            for s, n in enumerate(lens):
                for p in range(n):
                    t[int(c.table[s, p // 32]), :, p % 32] = keep[int(c.table[s, p // 32]), :, p % 32]
        c.cuda()
        a, q, out, lse = attend(made, c, lens, 6, "f16")
        assert B.pi_attn_sync(a) == B.PI_OK
        check_attention(c, lens, q, out, lse)


def test_attention_values_that_are_not_finite_stay_in_their_head(made):
    for cache in ("f16", "bf16"):
        lens = [50, 50, 50, 50]
        c = R.Cache(gen(2), lens, 2, 64, cache, 16)
        at = lambda s, p: (int(c.table[s, p // 16]), 0, p % 16)  # noqa: E731
        c.v[at(0, 20)][7] = INF
        c.v[at(1, 33)][9] = NAN
        c.k[at(2, 1)][3] = NAN
        c.k[at(3, 49)] = 0.0
        c.cuda()
        q = torch.randn(4, 6, 64, generator=gen(3)).half()
        a, q, out, lse = attend(made, c, lens, 6, "f16", q=q)
        out, lse = out.cpu(), lse.cpu()
        assert out[:, 3:].isfinite().all() and lse[:, 3:].isfinite().all()       # the other head of the cache
        assert (out[0, :3, 7] == INF).all() and out[0, :3, :7].isfinite().all()
        assert out[1, :3, 9].isnan().all() and out[1, :3, :9].isfinite().all()
        assert out[2, :3].isnan().all() and lse[2, :3].isnan().all()
        assert out[3].isfinite().all()


@pytest.mark.parametrize("lens", [[4000], [1, 3000, 0, 5, 1700], [64] * 40, [1] * 300, [0] * 5, [2048, 2049] * 3, [0] * 300 + [900]])
@pytest.mark.parametrize("cache,heads,kv_heads,dim", [("bf16", 8, 8, 64), ("int4g32", 8, 2, 128), ("i8", 16, 1, 64)])
def test_attention_batches(made, lens, cache, heads, kv_heads, dim):
    """Long and short sequences shared out over the GPU, many sequences, none."""
    c = R.Cache(gen(len(lens)), lens, kv_heads, dim, cache, 16).cuda()
    a, q, out, lse = attend(made, c, lens, heads, "f16")
    assert B.pi_attn_sync(a) == B.PI_OK
    pick = [i for i in range(len(lens)) if i < 6 or i % 50 == 0 or i == len(lens) - 1]
    for s in pick:
        want, l, bound, lb = R.attention(c, s, lens[s], q[s])
        check(out[s], want, bound + R.half_step(want.abs() + bound, out.dtype), f"sequence {s}")
        check(lse[s], l, lb) if lens[s] else None
    # the same bits again, and each sequence's near what it is alone
    o1, l1 = out.clone(), lse.clone()
    B.pi_paged_attention(a, cache_of(c), c.table_dev, torch.tensor(lens, dtype=torch.int32).cuda(), q.cuda(), out, lse=lse)
    assert torch.equal(o1, out) and torch.equal(l1, lse)


def test_attention_extreme_scores(made):
    """Scores far apart (all weight on one position), all alike, and of the scale's other sign."""
    lens = [130]
    for cache in ("f16", "bf16", "i8", "int4g32"):
        c = R.Cache(gen(4), lens, 1, 64, cache, 16).cuda()
        for factor, kw in ((300.0, {}), (0.0, {}), (1.0, {"scale": -0.5}), (1e-4, {}), (40.0, {"softcap": 3.0})):
            q = (factor * torch.randn(1, 4, 64, generator=gen(5)))
            a, q, out, lse = attend(made, c, lens, 4, "f32", q=q, **kw)
            check_attention(c, lens, q, out, lse, **kw)


def test_attention_scales_of_all_sizes(made):
    """8-bit and 4-bit rows whose scales differ by many orders."""
    for cache, top in (("i8", 12.0), ("int4g32", 4.0)):
        lens = [150, 20]
        c = R.Cache(gen(6), lens, 2, 128, cache, 16)
        f = torch.exp(torch.randn(c.v_scale.shape, generator=gen(7)) * top / 3).clamp(math.exp(-top), math.exp(top))
        c.v_scale = (c.v_scale.float() * f).to(c.v_scale.dtype)
        c.cuda()
        a, q, out, lse = attend(made, c, lens, 4, "f32")
        check_attention(c, lens, q, out, lse)


def test_attention_reports_bad_lengths_and_pages(made):
    """A bad page's positions are left out and reported, as are lengths out of range; other sequences are right."""
    lens = [40, 40, 16, 40]
    c = R.Cache(gen(8), lens, 2, 64, "f16", 16).cuda()
    c.table_dev[1, 1] = c.pages + 3
    a, q, out, lse = attend(made, c, [40, 40, -3, 1000], 4, "f16")
    assert B.pi_attn_sync(a) == B.PI_ERR_DEVICE_CHECK
    assert B.pi_attn_sync(a) == B.PI_OK
    want, l, bound, lb = R.attention(c, 0, 40, q[0])
    check(out[0], want, bound + R.half_step(want.abs() + bound, out.dtype))
    assert (out[2] == 0).all() and (lse[2] == -INF).all()
    # sequence 1 without the positions 16 .. 31
    k, v = (torch.cat((c.rows(n, 1, 0, 16), c.rows(n, 1, 32, 40))).repeat_interleave(2, 1) for n in ("k", "v"))
    s = torch.einsum("hd,phd->hp", q[1].double(), k) / 8
    assert (out[1].cpu().double() - torch.einsum("hp,phd->hd", torch.softmax(s, -1), v)).abs().max() < 2e-3
    assert (lse[1].cpu().double() - torch.logsumexp(s, -1)).abs().max() < 1e-4
    # sequence 3: the 48 positions that its table has
    want, l, bound, lb = R.attention(c, 3, 48, q[3])
    check(out[3], want, bound + R.half_step(want.abs() + bound, out.dtype))


def test_attention_strides_and_no_lse(made):
    lens = [33, 70]
    c = R.Cache(gen(9), lens, 2, 64, "f16", 16).cuda()
    a = layer(made, 4, 2, 64, cache_dtype="f16", page_size=16)
    big = torch.full((2, 4 * 64 + 8), 3.0, dtype=torch.float16, device="cuda")
    q = torch.randn(2, 4 * 64 + 40, generator=gen(10)).half().cuda()
    wide = torch.full((2, c.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table.shape[1]] = c.table_dev
    out = big[:, 8:].unflatten(1, (4, 64))
    qv = q[:, 16:16 + 256].unflatten(1, (4, 64))
    B.pi_paged_attention(a, cache_of(c), wide[:, 2:2 + c.table.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(), qv, out)
    assert (big[:, :8] == 3.0).all()
    for s, n in enumerate(lens):
        want, _, bound, _ = R.attention(c, s, n, qv[s].cpu())
        check(out[s], want, bound + R.half_step(want.abs() + bound, out.dtype))


def test_attention_graphs_share_a_handle_and_lengths_grow(made):
    """Two captured graphs of one handle, replayed in turn on their stream with lengths that grow."""
    g = gen(11)
    top = 600
    c = R.Cache(g, [top, top], 2, 64, "bf16", 16).cuda()
    a = layer(made, 8, 2, 64, cache_dtype="bf16", page_size=16)
    q = torch.randn(2, 2, 8, 64, generator=g).bfloat16().cuda()
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    outs, graphs = [torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            B.pi_paged_attention(a, cache_of(c), c.table_dev, lens, q[i], outs[i])
        graphs.append(gr)
    for n in ([1, 17], [300, 0], [600, 599], [2, 600]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for _ in range(3):
            for gr in graphs:
                gr.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for s in range(2):
                want, _, bound, _ = R.attention(c, s, n[s], q[i][s].cpu())
                check(outs[i][s], want, bound + R.half_step(want.abs() + bound, torch.bfloat16))
    assert B.pi_attn_sync(a) == B.PI_OK


def test_cache_offsets_beyond_32_bits(made):
    """Rows more than 4 GiB into a cache: write, read and attend."""
    g = gen(12)
    pages, page, heads, dim = 70000, 64, 4, 128          # 4.6 GB for each of k and v
    k = torch.empty(pages, heads, page, dim, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    cache = B.pi_kv_cache(k, v)
    a = layer(made, 8, heads, dim, cache_dtype="f16", page_size=page)
    table = torch.tensor([[pages - 1, 3], [pages - 2, pages - 70]], dtype=torch.int32, device="cuda")
    n = 70
    pos = torch.arange(n, dtype=torch.int32).repeat(2).cuda()
    seq = torch.arange(2, dtype=torch.int32).repeat_interleave(n).cuda()
    x = torch.randn(3, 2 * n, heads, dim, generator=g).half().cuda()
    q = torch.randn(2 * n, 8, dim, generator=g).half().cuda()
    B.pi_kv_append(a, cache, table, pos, q, x[0], x[1], torch.empty_like(q), seq=seq)
    ko, vo = torch.empty_like(x[0]), torch.empty_like(x[0])
    B.pi_kv_read(a, cache, table, pos, ko, vo, seq=seq)
    assert torch.equal(ko, x[0]) and torch.equal(vo, x[1])
    out = torch.empty(2, 8, dim, dtype=torch.float16, device="cuda")
    B.pi_paged_attention(a, cache, table, torch.tensor([n, n], dtype=torch.int32, device="cuda"), q[:2], out)
    assert B.pi_attn_sync(a) == B.PI_OK
    for s in range(2):
        kk, vv = (x[i][s * n:(s + 1) * n].double().cpu().repeat_interleave(2, 1) for i in range(2))
        p = torch.softmax(torch.einsum("hd,phd->hp", q[s].double().cpu(), kk) / math.sqrt(dim), -1)
        assert (out[s].cpu().double() - torch.einsum("hp,phd->hd", p, vv)).abs().max() < 2e-3
    del k, v, cache
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# refusals that need a handle
# ---------------------------------------------------------------------------
def refused(call):
    with pytest.raises(B.PiError) as e:
        call()
    assert e.value.status == B.PI_ERR_INVALID_ARG


def test_matvec_refusals(made):
    q, s = R.encode_int4(torch.randn(32, 64, generator=gen(1)))
    m = matrix(made, q, s)
    x, y = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 32, device="cuda")
    refused(lambda: B.pi_int4_matvec(m, torch.zeros(33, 64, device="cuda"), torch.zeros(33, 32, device="cuda")))
    refused(lambda: B.pi_int4_matvec(m, x[:0], y[:0]))
    refused(lambda: B.pi_int4_matvec(m, x[:, :32], y))
    refused(lambda: B.pi_int4_matvec(m, x, y[:3]))
    refused(lambda: B.pi_int4_matvec(m, x.double(), y))
    refused(lambda: B.pi_int4_matvec(m, x, y, norm_eps=-1.0))
    refused(lambda: B.pi_int4_matvec(m, x, y, norm_eps=NAN))
    refused(lambda: B.pi_int4_matvec(m, x, y, add=y.half()))
    refused(lambda: B.pi_int4_matvec(m, x.cpu(), y))
    refused(lambda: B.pi_int4_matvec(m, torch.zeros(4 * 64 + 1, device="cuda")[1:].view(4, 64), y))
    refused(lambda: B.pi_int4_matvec(m, torch.zeros(4, 66, device="cuda")[:, :64], y))          # rows 264 bytes apart
    buf = torch.zeros(4, 64, device="cuda")
    refused(lambda: B.pi_int4_matvec(m, buf, buf[:, 16:48]))                                    # y inside x
    big = torch.zeros(9, 32, device="cuda")
    refused(lambda: B.pi_int4_matvec(m, x, big[1:5], add=big[:4]))                              # add one row before y
    side = torch.zeros(4, 96, device="cuda")
    B.pi_int4_matvec(m, side[:, :64], side[:, 64:])                                             # side by side is fine
    refused(lambda: B.pi_int4_matvec(12345, x, y))


def test_attention_refusals(made):
    c = R.Cache(gen(1), [20, 20], 2, 64, "i8", 16).cuda()
    a = layer(made, 4, 2, 64, cache_dtype="i8", page_size=16)
    b = layer(made, 4, 2, 64, cache_dtype="f16", page_size=16)
    cache, pos = cache_of(c), torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    q, k, o = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    ap = lambda **n: B.pi_kv_append(**{**dict(a=a, cache=cache, table=c.table_dev, pos=pos, q=q, k=k, v=k, q_out=o), **n})  # noqa: E731
    ap()
    refused(lambda: ap(a=b))                                   # another handle's format
    refused(lambda: ap(q_norm=w))                              # weights without a norm
    refused(lambda: ap(pos=pos.long()))
    refused(lambda: ap(pos=pos[:1]))
    refused(lambda: ap(pos=torch.zeros(3, dtype=torch.int32, device="cuda"), q=torch.zeros(3, 4, 64, device="cuda"),
                       k=torch.zeros(3, 2, 64, device="cuda"), v=torch.zeros(3, 2, 64, device="cuda"),
                       q_out=torch.zeros(3, 4, 64, device="cuda")))                            # no seq, more tokens than sequences
    refused(lambda: ap(q=q.half()))
    refused(lambda: ap(k=q))
    refused(lambda: ap(table=c.table_dev.long()))
    refused(lambda: ap(table=c.table_dev.cpu()))
    both = torch.zeros(2, 6, 64, device="cuda")
    refused(lambda: ap(q=both[:, :4], q_out=both[:, 1:5]))     # shifted onto itself
    refused(lambda: ap(q=both[:, :4], k=both[:, 4:], q_out=both[:, 2:]))
    rd = lambda **n: B.pi_kv_read(**{**dict(a=a, cache=cache, table=c.table_dev, pos=pos, k_out=k, v_out=k.clone()), **n})  # noqa: E731
    rd()
    refused(lambda: rd(k_out=k.half()))
    refused(lambda: rd(k_out=q))
    refused(lambda: rd(k_out=torch.zeros(2 * 2 * 64 + 1, device="cuda")[1:].view(2, 2, 64)))
    at = lambda **n: B.pi_paged_attention(**{**dict(a=a, cache=cache, table=c.table_dev, lens=pos, q=q, out=o), **n})  # noqa: E731
    at()
    refused(lambda: at(out=q))
    refused(lambda: at(lens=pos[:1]))
    refused(lambda: at(lse=torch.zeros(2, 3, device="cuda")))
    refused(lambda: at(q=torch.zeros(2, 4, 66, device="cuda")[..., :64]))
    refused(lambda: at(cache=B.pi_kv_cache(c.k, c.v)))
    refused(lambda: at(cache=B.pi_kv_cache(c.k[:, :1], c.v[:, :1], c.k_scale[:, :1], c.v_scale[:, :1])))
    torch.cuda.synchronize()
