"""The attention half of a decode layer at the limits of its numbers: the largest
values, few rounded steps, long exact sums; and what stands beside a call.  Definitions and roundings: attn_ref.py."""
import math

import pytest
import torch

import attn_ref as R
from activation_sparse_decode_threshold_b200 import binding as B
from test_gpu_attention import attend, cache_of, check, gen, layer, made, matrix, refused  # noqa: F401
from test_gpu_attention_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,tokens", [(40, 96, 1), (33, 416, 3), (70, 8192, 13)])
def test_matvec_largest_numbers(made, dt, n, k, tokens):
    """x up to the type's largest number: as long as the result is finite, so is every sum on the way to it."""
    g = gen(n + tokens)
    q, _ = R.encode_int4(torch.randn(n, k, generator=g))
    s = torch.full((n, k // 32), 2.0 ** -14, dtype=torch.float16)      # |y| <= 8 K 2^-14 max |x| / (random signs)
    top = torch.finfo(R.DT[dt]).max
    x = ((0.5 + 0.5 * torch.rand(tokens, k, generator=g)) * torch.where(torch.rand(tokens, k, generator=g) < 0.5, -1.0, 1.0)).double()
    x = (x * top).to(R.DT[dt]).clamp(-top, top)
    x[0] = x[0].abs()                                                  # (one token without the signs' help)
    x[0, ::2] = top
    y = torch.zeros(tokens, n, device="cuda")
    B.pi_int4_matvec(matrix(made, q, s), x.cuda(), y)
    want, bound = R.matvec(q, s, x, torch.float32)
    assert want.abs().max() < 0.9 * top
    check(y, want, bound)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,tokens", [(40, 96, 1), (33, 416, 7), (70, 8192, 13), (24, 8192, 32)])
def test_matvec_norm_of_large_and_small_numbers(made, dt, n, k, tokens):
    """Tokens whose squares leave fp32's range (above 1.8e19), beside ordinary ones, zeros and small ones."""
    g = gen(n + tokens)
    q, s = R.encode_int4(torch.randn(n, k, generator=g) * 0.05)
    sizes = torch.tensor([1e20, 1.0, 1e30, 0.0, 1e36, 1e19, 1e-20])[torch.arange(tokens) % 7]
    x = (torch.randn(tokens, k, generator=g) * sizes[:, None]).to(R.DT[dt])
    if tokens > 1:
        x[1, 5] = 1e22                                                 # one large element among ordinary ones
    y = torch.zeros(tokens, n, device="cuda")
    B.pi_int4_matvec(matrix(made, q, s), x.cuda(), y, norm_eps=1e-6)
    want, bound = R.matvec(q, s, x, torch.float32, eps=1e-6)
    check(y, want, bound)
    # without a norm the same numbers stay apart too: nothing of one token gets into another
    alone = torch.zeros(1, n, device="cuda")
    for t in (0, tokens - 1):
        B.pi_int4_matvec(matrix(made, q, s), x[t:t + 1].cuda(), alone, norm_eps=1e-6)
        want, bound = R.matvec(q, s, x[t:t + 1], torch.float32, eps=1e-6)
        check(alone, want, bound)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [3, 200])     # (4 and 8 elements to a lane)
def test_append_norm_of_large_queries(made, dt, dim, tokens):
    """Heads whose squares leave fp32's range are normed like all others, queries and keys."""
    g = gen(dim + tokens)
    heads, kv, eps = 6, 2, 1e-6
    c = R.Cache(g, [tokens], kv, dim, "bf16", 16, fill=False).cuda()
    a = layer(made, heads, kv, dim, cache_dtype="bf16", page_size=16, rotary_dim=dim, norm_eps=eps)
    sizes = torch.tensor([1e20, 1.0, 1e-3, 1e37, 1e19])
    mk = lambda h: torch.randn(tokens, h, dim, generator=g) * sizes[torch.arange(tokens * h) % 5].view(tokens, h, 1)  # noqa: E731
    q, k, v = mk(heads).to(R.DT[dt]), mk(kv).to(R.DT[dt]), torch.randn(tokens, kv, dim, generator=g).to(R.DT[dt])
    q[0, 0, 0] = torch.finfo(R.DT[dt]).max
    w = 1 + 0.3 * torch.randn(dim, generator=g)
    out = torch.zeros(tokens, heads, dim, dtype=R.DT[dt], device="cuda")
    pos, seq = torch.arange(tokens, dtype=torch.int32).cuda(), torch.zeros(tokens, dtype=torch.int32, device="cuda")
    B.pi_kv_append(a, cache_of(c), c.table_dev, pos, q.cuda(), k.cuda(), v.cuda(), out, seq=seq, q_norm=w.cuda(), k_norm=w.cuda())
    assert B.pi_attn_sync(a) == B.PI_OK
    rows = c.rows("k", 0, 0, tokens)
    for t in range(tokens):
        x, mag = R.norm_rotate(q[t], t, dim, False, 10000.0, eps, w)
        # (as in test_gpu_attention.py: the norm's sum, root and products, the rotation)
        check(out[t], x, mag * (dim / 32 + 5 + 8 + 6) * R.U + R.half_step(x, R.DT[dt]), f"q {t}")
        x, _ = R.norm_rotate(k[t], t, dim, False, 10000.0, eps, w)
        check(rows[t], x, R.half_step(x, torch.bfloat16) + x.abs() * R.U, f"k {t}")


def one_hot(cache, lens, kv_heads, dim, page, k_at, k_value, v_at, v_value):
    """A cache whose keys and values have one element each that is not zero: (position, head) -> element."""
    c = R.Cache(gen(0), lens, kv_heads, dim, cache, page, fill=False)
    ks, vs = (torch.zeros(c.pages, kv_heads, page, dim) for _ in range(2))
    for s, n in enumerate(lens):
        for p in range(n):
            at = int(c.table[s, p // page]), slice(None), p % page
            ks[at][:, k_at(p)] = k_value
            vs[at][:, v_at(p)] = v_value(p)
    c.k, c.k_scale = R.encode(ks, cache)
    c.v, c.v_scale = R.encode(vs, cache)
    return c.cuda()


@pytest.mark.parametrize("dim,kv_heads,group", [(64, 2, 1), (128, 1, 4), (64, 1, 8), (128, 2, 7), (64, 2, 16), (128, 1, 24)])
def test_scores_of_fp32_queries_over_bf16_keep_their_bits(made, dim, kv_heads, group):
    """One position with one product: the log of the sum is the score itself, q scale.  fp32 roundings on the way: scale
    log2 e (its constant and a product), the score's product, the log's two, and one to spare."""
    lens = [1] * 5
    c = one_hot("bf16", lens, kv_heads, dim, 16, lambda p: 7, 1.0, lambda p: 3, lambda p: 1.0)
    q = torch.randn(5, kv_heads * group, dim, generator=gen(dim + group)) * 8
    a, q, out, lse = attend(made, c, lens, kv_heads * group, "f32", q=q)
    want = q[:, :, 7].double() / math.sqrt(dim)
    check(lse, want, want.abs() * 6 * R.U + 2.0 ** -149)
    assert torch.equal(out[:, :, 3].cpu(), torch.ones(5, kv_heads * group))


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("dim,kv_heads,group", [(64, 2, 1), (128, 1, 4), (64, 1, 8), (128, 2, 7), (64, 2, 16), (128, 1, 24)])
def test_weights_of_fp32_callers_keep_their_bits(made, cache, dim, kv_heads, group):
    """Two positions of scores 0 and s in (-1, 0), values 0 and 1: out = w / (1 + w), w = e^s, the same w above and below.
    Roundings relative to out: the score 6 steps of s (test above), exp2 2^-22, the fp16 weight's two parts or the bf16
    one's three 2^-23 (x - m + 14 for fp16: half a step of 16, 2^-20 log 2 / 2), sums, quotient and products 12 steps."""
    n = 60
    lens = [2] * n
    c = one_hot(cache, lens, kv_heads, dim, 16, lambda p: p, 1.0, lambda p: 0, lambda p: float(p))
    q = torch.zeros(n, kv_heads * group, dim)
    q[:, :, 1] = -torch.rand(n, kv_heads * group, generator=gen(group)) * math.sqrt(dim)
    a, q, out, lse = attend(made, c, lens, kv_heads * group, "f32", q=q)
    s = q[:, :, 1].double() / math.sqrt(dim)
    want = torch.sigmoid(s)
    rel = 6 * R.U + 2.0 ** -22 + 2.0 ** -23 + 12 * R.U + (2.0 ** -21 * math.log(2) if cache == "f16" else 0)
    check(out[:, :, 0], want, want * rel)


@pytest.mark.parametrize("cap", [5.0, 30.0, 64.0, 65.0])
@pytest.mark.parametrize("cache,unit", [("bf16", 1.0), ("f16", 1.0), ("i8", 127.0), ("int4g32", 7.0)])
def test_capped_scores_of_fp32_callers(made, cache, unit, cap):
    """One position: the log of the sum is the capped score.  Relative roundings: the score 6 steps and its quotient by the
    cap 2 (2 log 2 of it is tanh's argument: 2 more), none of them larger in the tangent; tanh 2^-22; the products with the
    cap and log 2 and their constants 4."""
    lens = [1] * 40
    c = one_hot(cache, lens, 1, 64, 16, lambda p: 9, unit, lambda p: 0, lambda p: unit)
    q = torch.zeros(40, 4, 64)
    q[:, :, 9] = (torch.randn(40, 4, generator=gen(3)) * 4).bfloat16().float()
    a, q, out, lse = attend(made, c, lens, 4, "f32", q=q, scale=0.25 / unit, softcap=cap)
    # (scale is an fp32 number for the library)
    s = q[:, :, 9].double() * unit * float(torch.tensor(0.25 / unit, dtype=torch.float32))
    want = cap * torch.tanh(s / cap)
    check(lse, want, want.abs() * (6 + 2 + 2 + 4 + 4) * R.U + 2.0 ** -149)


def test_a_cache_s_tensors_are_taken_as_they_are_at_the_call(made):
    """A cache tensor that is given other memory or another shape after a call is used, or refused, as it then is."""
    c = R.Cache(gen(1), [20], 2, 64, "f16", 16, spare=1).cuda()
    other = R.Cache(gen(2), [20], 2, 64, "f16", 16, spare=1).cuda()
    a = layer(made, 4, 2, 64, cache_dtype="f16", page_size=16)
    pos, seq = torch.arange(20, dtype=torch.int32).cuda(), torch.zeros(20, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(20, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    cache, keep = cache_of(c), c.k.view(-1)
    table = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    read = lambda: B.pi_kv_read(a, cache, table, pos, k, v, seq=seq)  # noqa: E731
    flat = lambda t: torch.cat((t[0], t[2]), 1).transpose(0, 1)[:20]  # noqa: E731  (pages 0 and 2, [positions, heads, dim])
    read()
    assert torch.equal(k, flat(c.k)) and torch.equal(v, flat(c.v))
    c.k.set_(other.k)
    read()
    assert torch.equal(k, flat(other.k)) and torch.equal(v, flat(c.v))
    with pytest.raises(AttributeError):
        cache.k = c.v
    c.k.resize_(2, 2, 16, 64)          # K of two pages, V of three
    refused(read)
    c.v.resize_(2, 2, 16, 64)
    read()
    assert B.pi_attn_sync(a) == B.PI_ERR_DEVICE_CHECK      # page 2 is none of the cache's any more
    assert keep.numel() == 3 * 2 * 16 * 64


def test_read_into_overlapping_buffers_is_refused(made):
    """K's and V's rows must not share memory, with each other or with the cache."""
    for kind in ("f16", "i8", "int4g32"):
        c = R.Cache(gen(3), [20, 20], 2, 64, kind, 16).cuda()
        a, cache = layer(made, 4, 2, 64, cache_dtype=kind, page_size=16), cache_of(c)
        pos = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
        read = lambda k, v: B.pi_kv_read(a, cache, c.table_dev, pos, k, v)  # noqa: E731
        both = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
        read(both[:2], both[2:])                                           # side by side is fine
        assert torch.equal(both[1, :, :8].cpu(), c.rows("k", 1, 2, 3)[0, :, :8].half())
        keep = both.clone()
        refused(lambda: read(both[:2], both[:2]))
        refused(lambda: read(both[:2], both[1:3]))
        refused(lambda: read(both[1:3], both[:2]))
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                into = t.view(-1).view(torch.float16)
                refused(lambda: read(both[:2], into[:256].view(2, 2, 64)))
                refused(lambda: read(into[-256:].view(2, 2, 64), both[:2]))
        assert torch.equal(both, keep) and B.pi_attn_sync(a) == B.PI_OK


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,tokens", [(8, 131072, 1), (16, 131072, 32), (19, 32768, 32), (300, 8192, 13), (2500, 320, 1),
                                        (33, 4128, 24), (50, 14336, 8)])
def test_matvec_sums_of_whole_numbers_are_exact(made, dt, n, k, tokens):
    """x in -3 .. 3, scales 1/2 and 1: every sum is a multiple of 1/2 below 2^23, which fp32 holds, so that a group lost,
    doubled or of another row shows at any length."""
    g = gen(n + k)
    q = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    s = torch.where(torch.rand(n, k // 32, generator=g) < 0.5, 0.5, 1.0).half()
    x = torch.randint(-3, 4, (tokens, k), generator=g).to(R.DT[dt])
    add = torch.randint(-100, 101, (tokens, n), generator=g).float()
    w = R.decode(q, s, "int4g32")
    want = x.double() @ w.t()
    assert (x.double().abs() @ w.abs().t()).max() + 100 < 2 ** 23
    m, xd, y = matrix(made, q, s), x.cuda(), torch.full((tokens, n), 0.25, device="cuda")
    B.pi_int4_matvec(m, xd, y)
    assert torch.equal(y.cpu().double(), want)
    B.pi_int4_matvec(m, xd, y, add=add.cuda())
    assert torch.equal(y.cpu().double(), want + add)


@pytest.mark.parametrize("lens", [[1, 3000, 0, 5, 1700], [2048, 2049] * 3, [1] * 40 + [900]])
@pytest.mark.parametrize("cache,heads,kv_heads,dim", [("bf16", 8, 8, 64), ("int4g32", 8, 2, 128), ("i8", 16, 1, 64)])
def test_attention_of_a_batch_is_that_of_each_alone(made, lens, cache, heads, kv_heads, dim):
    """The same values, within both calls' bounds, whatever stands beside a sequence."""
    c = R.Cache(gen(len(lens)), lens, kv_heads, dim, cache, 16).cuda()
    a, q, out, lse = attend(made, c, lens, heads, "f16")
    for s in [i for i in range(len(lens)) if i < 6 or i > 38]:
        o1, l1 = torch.full_like(out[:1], 5.0), torch.full_like(lse[:1], 5.0)
        n1 = torch.tensor(lens[s:s + 1], dtype=torch.int32, device="cuda")
        B.pi_paged_attention(a, cache_of(c), c.table_dev[s:s + 1], n1, q[s:s + 1].cuda(), o1, lse=l1)
        want, l, bound, lb = R.attention(c, s, lens[s], q[s])
        if lens[s] == 0:
            assert torch.equal(o1[0], out[s]) and torch.equal(l1[0], lse[s])
            continue
        check(o1[0], out[s].cpu().double(), 2 * (bound + R.half_step(want.abs() + bound, out.dtype)), f"out of sequence {s}")
        check(l1[0], lse[s].cpu().double(), 2 * lb, f"lse of sequence {s}")


class LayerWithLse(Layer):
    """A layer whose attention gives the log of its sums too."""

    def step(self, a, r, pos, lens):
        h, k, d = self.heads, self.kv_heads, self.dim
        part = lambda i, n: self.qkv[:, i * d:(i + n) * d].unflatten(1, (n, d))  # noqa: E731
        self.logs = torch.full((r.shape[0], h), 3.0, device="cuda")
        B.pi_int4_matvec(self.m[0], r, self.qkv, norm_eps=1e-6)
        B.pi_kv_append(a, self.cache, self.c.table_dev, pos, part(0, h), part(h, k), part(h + k, k), self.q,
                       q_norm=self.norms[0], k_norm=self.norms[1])
        B.pi_paged_attention(a, self.cache, self.c.table_dev, lens, self.q, self.o.unflatten(1, (h, d)), lse=self.logs)
        B.pi_int4_matvec(self.m[1], self.o, r, add=r)

    def lse(self, lens, q):
        return self.logs


@pytest.mark.parametrize("cache,io,tokens", [("bf16", "bf16", 3), ("f16", "f16", 1), ("i8", "f16", 5), ("int4g32", "f16", 2),
                                             ("bf16", "f32", 2)])
def test_a_layer_s_steps_with_the_logs_of_the_sums(made, cache, io, tokens):
    """Steps of growing texts, every stage on the inputs that it really had, the logs of the sums among them."""
    g = gen(tokens)
    heads, kv_heads, dim, theta = 6, 2, 64, 10000.0
    lens = [29 + 7 * s for s in range(tokens)]
    a = layer(made, heads, kv_heads, dim, cache_dtype=cache, page_size=16, rotary_dim=dim, rope_theta=theta, norm_eps=1e-6)
    la = LayerWithLse(made, g, 512, heads, kv_heads, dim, cache, 16, [n + 4 for n in lens], tokens, io)
    r = torch.randn(tokens, 512, generator=g).cuda()
    for step in range(3):
        now = [n + step for n in lens]
        before = r.cpu()
        la.step(a, r, torch.tensor(now, dtype=torch.int32).cuda(), torch.tensor([n + 1 for n in now], dtype=torch.int32).cuda())
        assert B.pi_attn_sync(a) == B.PI_OK
        la.check(before, r, now, [n + 1 for n in now], theta)


@pytest.mark.parametrize("dim,kv_heads,group", [(64, 8, 1), (128, 4, 4), (64, 2, 8), (128, 1, 16), (64, 1, 16)])
@pytest.mark.parametrize("lens,window", [([4000], 0), ([1, 3000, 0, 5, 1700], 700), ([700, 2, 0, 130] * 10, 0)])
def test_attention_of_fp32_callers_over_bf16(made, lens, window, dim, kv_heads, group):
    """Texts that warps and CTAs share, empty ones and many, in the form that fp32 callers over a bf16 cache have."""
    c = R.Cache(gen(dim + group), lens, kv_heads, dim, "bf16", 16).cuda()
    a, q, out, lse = attend(made, c, lens, kv_heads * group, "f32", window=window)
    assert B.pi_attn_sync(a) == B.PI_OK
    for s in [i for i in range(len(lens)) if i < 6 or i == len(lens) - 1]:
        want, l, bound, lb = R.attention(c, s, lens[s], q[s], window=window)
        check(out[s], want, bound + R.half_step(want.abs() + bound, torch.float32), f"out of sequence {s}")
        if lens[s]:
            check(lse[s], l, lb, f"lse of sequence {s}")
        else:
            assert (lse[s] == -math.inf).all()
    o1, l1 = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    n, qd, cache = torch.tensor(lens, dtype=torch.int32).cuda(), q.cuda(), cache_of(c)
    with torch.cuda.graph(graph):
        B.pi_paged_attention(a, cache, c.table_dev, n, qd, out, lse=lse)
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        assert torch.equal(o1, out) and torch.equal(l1, lse)
