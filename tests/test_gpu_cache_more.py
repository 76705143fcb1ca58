"""The cache calls where they are used and at the ends of their ranges: with
the rotation in front, on streams of their own, in captured graphs, with many
rows and with caches that no level of cache holds."""
import math

import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B
from test_gpu_cache import BF16, F16, F32, FORMATS, U, U8, Batch, Cache, gpu, ints, np64  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def reference(q, k, v, lens, scale):
    """y and lse in fp64 on the GPU: q [rows, heads, d], k and v [rows, tokens,
    kv, d] (what the cache reads back as)."""
    rows, heads, d = q.shape
    kv = k.shape[2]
    y = torch.zeros((rows, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(rows):
        n = int(lens[r])
        if n == 0:
            continue
        for h in range(heads):
            g = h // (heads // kv)
            s = (k[r, :n, g].double() * q[r, h].double()).sum(1) * scale
            p = torch.exp(s - s.max())
            y[r, h] = (p[:, None] * v[r, :n, g].double()).sum(0) / p.sum()
            lse[r, h] = s.max() + torch.log(p.sum())
    return y, lse


class Decoder:
    """One layer's attention in decoding: queries and keys rotated by the same
    butterfly of n = d over their heads, keys and values into a paged cache."""

    def __init__(self, fmt, rows, heads, kv, d, most, page=16, seed=0, rotate=True):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.rows, self.heads, self.kv, self.d, self.most = fmt, rows, heads, kv, d, most
        self.width = -(-most // page)
        self.cache = Cache(fmt, rows * self.width + 1, kv, page, d)
        order = torch.randperm(rows * self.width + 1, generator=g)[: rows * self.width]
        self.tables = order.reshape(rows, self.width).to(torch.int32).cuda()
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.theta = ((torch.rand((int(math.log2(d)), d // 2), generator=g) * 2 - 1) * math.pi).cuda()
        self.table = torch.empty(B.bfly_coeff_bytes(d), dtype=U8, device="cuda")
        B.bfly_prepare(self.theta, d, self.table)
        self.rotate = rotate
        self.qkv = torch.empty((rows, heads + 2 * kv, d), dtype=BF16, device="cuda")
        self.rot = torch.empty_like(self.qkv)
        self.y = torch.empty((rows, heads, d), dtype=BF16, device="cuda")
        self.slots = torch.empty(rows, dtype=torch.int32, device="cuda")
        n = B.bfly_cache_attention_workspace_bytes(rows, heads, kv, d, most)
        self.ws = torch.empty(max(1, n), dtype=U8, device="cuda")

    def step(self, stream=None):
        """The tokens in qkv appended to every sequence, then looked at."""
        h, kv, c = self.heads, self.kv, self.cache
        src = self.qkv
        if self.rotate:
            B.bfly_forward(self.qkv.view(-1, self.d), self.rot.view(-1, self.d), coeffs=self.table,
                           stream=stream)
            src = self.rot
        at = self.lens.long()
        page = self.tables.gather(1, (at // c.page)[:, None])[:, 0]
        self.slots.copy_(page * c.page + at % c.page)
        self.lens += 1
        c.write(src[:, h:h + kv], self.qkv[:, h + kv:], self.slots, stream=stream)
        B.bfly_cache_attention(src[:, :h], c.k, c.v, self.tables, self.lens, self.y, max_len=self.most,
                               workspace=self.ws, stream=stream, **c.scales)
        return self.y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decoding_with_rotated_heads(fmt, d):
    """Forty decode steps of three sequences.  Every step against the formula in
    64 bits on what the cache reads back as and the rotated bf16 queries: the
    tolerance of one call, whose largest part is the result's own rounding (bf16
    2^-8) and a weight's (2^-11; its score's error stays below 2^-12 here: 300
    fp32 roundings of scores below 40).  And the last step against attention
    over the rows that were given: a row in the cache is off by half a code an
    element, dk in its 2-norm, and a rotated key and query by bf16's rounding,
    2^-8 of its norm each, so a score by at most ds = scale |q| (dk + 2^-7 |k|), a
    weight by the factor e^(2 ds), and y by that of sum p |v|, the values' own
    half codes dv, their bf16 roundings and the result's (2^-7 together)."""
    rows, heads, kv = 3, 6, 2
    dec = Decoder(fmt, rows, heads, kv, d, 64, seed=d)
    g = torch.Generator().manual_seed(1)
    ks, vs = [], []
    for i in range(40):
        x = torch.randn((rows, heads + 2 * kv, d), generator=g)
        x[:, heads:heads + kv, 3] *= 8.0                    # an outlier channel of the keys
        dec.qkv.copy_(x.to(BF16))
        y = dec.step()
        ks.append(dec.qkv[:, heads:heads + kv].clone())
        vs.append(dec.qkv[:, heads + kv:].clone())
        n = i + 1
        at = torch.arange(n, device="cuda")
        slots = (dec.tables[:, at // 16] * 16 + at % 16).reshape(-1).int()
        k, v = (torch.empty((rows * n, kv, d), device="cuda") for _ in "kv")
        dec.cache.read(slots, k, v)
        k, v = k.view(rows, n, kv, d), v.view(rows, n, kv, d)
        want, _ = reference(dec.rot[:, :heads], k, v, dec.lens, d ** -0.5)
        size, _ = reference(dec.rot[:, :heads], k, v.abs(), dec.lens, d ** -0.5)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -11) * size + 2.0 ** -20
        assert ((y.double() - want).abs() <= tol).all(), (i, float(((y.double() - want).abs() / tol).max()))
    if fmt not in ("bf16", "int8"):
        return                                              # too few bits for a bound by norms
    k0, v0 = torch.stack(ks, 1).float(), torch.stack(vs, 1).float()
    q0 = dec.qkv[:, :heads].float()
    want, _ = reference(q0, k0, v0, dec.lens, d ** -0.5)
    size, _ = reference(q0, k0, v0.abs(), dec.lens, d ** -0.5)
    half = {"bf16": 0.0, "int8": 0.5 / 127}[fmt]            # of a row's largest element, and 2^-11 of the scale
    knorm, qnorm = k0.norm(dim=3).max().item(), q0.norm(dim=2).max().item()
    dk = 1.2 * half * k.abs().max().item() * math.sqrt(d)
    ds = d ** -0.5 * qnorm * (dk + 2.0 ** -7 * knorm)
    dv = 1.2 * half * v0.abs().max().item()
    tol = (math.exp(2 * ds) - 1) * (size + dv) + dv + 2.0 ** -7 * size
    assert ((dec.y.double() - want).abs() <= tol).all()


def test_steps_on_another_stream_and_in_a_graph():
    """The same steps eagerly, on another stream with work in front of them, and
    captured once and replayed, with eager work between the replays; the
    sequence's length is on the device, so that replays go on appending."""
    def run(how):
        dec = Decoder("int8", 5, 8, 2, 128, 2000, seed=2)
        g = torch.Generator().manual_seed(3)
        xs = [torch.randn(dec.qkv.shape, generator=g).to(BF16).cuda() for _ in range(8)]
        dec.lens += torch.tensor([0, 1, 300, 1500, 1990], dtype=torch.int32, device="cuda")
        filler = torch.randn((2000, 2, 128), generator=g).cuda()
        for r in range(5):          # something to look at
            at = torch.arange(2000, device="cuda")
            dec.cache.write(filler, filler.flip(0), dec.tables[r, at // 16] * 16 + at.int() % 16)
        dec.qkv.copy_(xs[0])
        out = []
        if how == "graph":
            lens, pages = dec.lens.clone(), dec.cache.state()
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                dec.step()          # once before the capture
            torch.cuda.current_stream().wait_stream(s)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dec.step()
            dec.lens.copy_(lens)
            for t, was in zip((dec.cache.k, dec.cache.v, dec.cache.ks, dec.cache.vs), pages):
                t.view(U8).copy_(was)
        s = torch.cuda.Stream()
        for i, x in enumerate(xs):
            if how == "graph":
                dec.qkv.copy_(x)
                graph.replay()
                torch.cuda.synchronize() if i % 2 else None
                junk = torch.randn((512, 512), device="cuda") @ torch.randn((512, 512), device="cuda")
                del junk
            elif how == "stream":
                torch.cuda.synchronize()
                with torch.cuda.stream(s):
                    dec.qkv.zero_()
                    big = torch.randn((2048, 2048), device="cuda")
                    for _ in range(3):
                        big = big @ big * 1e-2
                    dec.qkv.copy_(x)
                    dec.step(stream=s if i % 2 else None)
                s.synchronize()
            else:
                dec.qkv.copy_(x)
                dec.step()
            out.append(dec.y.clone())
        return out + dec.cache.state()

    want = run("eager")
    for how in ("stream", "graph"):
        for a, b in zip(want, run(how)):
            assert torch.equal(a, b), how


def test_two_graphs_share_a_workspace():
    """Captured calls of different sizes over one workspace, replayed in turn."""
    a = Batch("int4", [3000, 40, 900], 8, 2, 64, 16, seed=20)
    b = Batch("bf16", [5000], 4, 4, 128, 32, y=F32, seed=21)
    size = [B.bfly_cache_attention_workspace_bytes(len(x.lens), x.heads, x.kv, x.d, x.width * x.page)
            for x in (a, b)]
    ws = torch.empty(max(size), dtype=U8, device="cuda")
    want, graphs, args = [], [], []
    for x in (a, b):
        want.append([t.clone() for t in x.run()])
        args.append((ints(x.tables), ints(x.lens)))
    for x, (t, n) in zip((a, b), args):
        x.run(tables=t, lens=n, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(tables=t, lens=n, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        x = (a, b)[i]
        x.y.fill_(7.0), x.lse.fill_(7.0)
        ws.fill_(0xFF)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(x.y, want[i][0]) and torch.equal(x.lse, want[i][1])


def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    xs = [Batch("int8", [4000, 100], 8, 2, 64, 16, seed=22 + i) for i in range(2)]
    want = [x.run()[0].clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    args = [(ints(x.tables), ints(x.lens)) for x in xs]
    for _ in range(5):
        for x in xs:
            x.y.fill_(7.0)
        torch.cuda.synchronize()
        for x, s, (t, n) in zip(xs, streams, args):
            for _ in range(4):
                x.run(tables=t, lens=n, stream=s)           # a fresh workspace each
        torch.cuda.synchronize()
        for x, y in zip(xs, want):
            assert torch.equal(x.y, y)


def test_joined_by_their_log_sums():
    """Attention over two parts of the tokens, joined with lse, is attention over
    all: p / sum = sum over parts of e^(lse_part - lse) y_part.  Both sides are
    off by a call's own tolerance: fp32 scores of d = 64 (2^-18), weights of 22
    bits, sums of 900 terms (2^-14)."""
    b = Batch("int8", [900], 4, 2, 64, 32, F32, F32, seed=24)
    y, l = (t.clone().double() for t in b.run())
    parts = []
    for first, n in ((0, 512), (16, 900 - 512)):
        t = b.tables[:, first:]
        parts.append([x.clone().double() for x in b.run(tables=ints(t), lens=ints([n]), max_len=n)])
    lse = torch.logaddexp(parts[0][1], parts[1][1])
    got = sum(torch.exp(p[1] - lse)[..., None] * p[0] for p in parts)
    assert (lse - l).abs().max() <= 2.0 ** -13
    assert (got - y).abs().max() <= 2.0 ** -12 * float(y.abs().max())


@pytest.mark.parametrize("rows,most", [(300, 1500), (257, 3000), (256, 1100), (70000, 20)])
def test_many_rows(rows, most):
    """More rows than a workgroup looks through, than a grid's second axis has."""
    d, kv, heads, page = 64, 1, 2, 16
    g = torch.Generator().manual_seed(rows)
    pages = 40
    c = Cache("int8", pages, kv, page, d, junk=False)
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((pages * page, kv, d), generator=g).cuda() for _ in "kv")
    c.write(k, v, slots)
    width = -(-most // page)
    tables = torch.randint(0, pages, (rows, width), generator=g).to(torch.int32).cuda()
    lens = torch.randint(0, most + 1, (rows,), generator=g).to(torch.int32)
    lens[0], lens[-1] = most, most
    q = torch.randn((rows, heads, d), generator=g).cuda()
    y, lse = torch.empty_like(q), torch.empty((rows, heads), device="cuda")
    B.bfly_cache_attention(q, c.k, c.v, tables, lens.cuda(), y, lse=lse, max_len=most, **c.scales)
    kr, vr = (torch.empty_like(k) for _ in "kv")
    c.read(slots, kr, vr)
    some = sorted({0, 1, rows // 2, rows - 2, rows - 1} | set(range(250, min(rows, 262))))
    at = torch.arange(most, device="cuda")
    for r in some:
        s = (tables[r, at // page] * page + at % page).long()
        want, wl = reference(q[r:r + 1], kr[s][None], vr[s][None], lens[r:r + 1], d ** -0.5)
        size, _ = reference(q[r:r + 1], kr[s][None], vr[s][None].abs(), lens[r:r + 1], d ** -0.5)
        # scores below 2^4 of 64 products, their shift and scales: 2^-16; sums of
        # up to 3000 terms in chains of at most 600: 2^-14
        assert ((y[r:r + 1].double() - want).abs() <= 2.0 ** -13 * size + 2.0 ** -40).all(), r
        if int(lens[r]):
            assert (lse[r:r + 1].double() - wl).abs().max() <= 2.0 ** -13
        else:
            assert (lse[r] == -math.inf).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_more_than_the_last_level_cache_holds(fmt):
    """One sequence of 2^28 bytes of keys and values and more, and ragged rows
    of 2^29: the loads that go past the caches."""
    d, kv, heads, page = 128, 4, 8, 256
    n = (1 << 28) // (2 * kv * {"bf16": 256, "int8": 128, "e4m3": 128, "int4": 64}[fmt]) + 77
    width = -(-n // page)
    c = Cache(fmt, width, kv, page, d, junk=False)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randperm(width, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(n, device="cuda")
    slots = (ids[at // page] * page + at % page).to(torch.int32)
    for part in slots.split(100000):
        k, v = (torch.randn((len(part), kv, d), generator=g, device="cuda") for _ in "kv")
        c.write(k, v, part)
    k, v = (torch.empty((n, kv, d), device="cuda") for _ in "kv")
    c.read(slots, k, v)
    q = 2.0 * torch.randn((4, heads, d), generator=g, device="cuda")
    for rows, lens in ((1, [n]), (4, [n, 5, n // 3, 0])):
        y, lse = torch.empty((rows, heads, d), device="cuda"), torch.empty((rows, heads), device="cuda")
        B.bfly_cache_attention(q[:rows], c.k, c.v, ids[None].expand(rows, -1).contiguous(), ints(lens), y,
                               lse=lse, **c.scales)
        kk, vv = k[None].expand(rows, -1, -1, -1), v[None].expand(rows, -1, -1, -1)
        want, wl = reference(q[:rows], kk, vv, lens, d ** -0.5)
        size, _ = reference(q[:rows], kk, vv.abs(), lens, d ** -0.5)
        # scores below 2^5 of 128 products: 2^-15 each way; a chunk's lane sums up
        # to 1000 terms, the join up to 512: 2^-13
        assert ((y.double() - want).abs() <= 2.0 ** -12 * size + 2.0 ** -40).all()
        ok = torch.tensor(lens, device="cuda") > 0
        assert (lse.double() - wl)[ok].abs().max() <= 2.0 ** -13 and (lse[~ok] == -math.inf).all()


def test_the_library_allocates_nothing():
    b = Batch("int4", [5000, 300], 8, 2, 128, 16, seed=30)
    t, n = ints(b.tables), ints(b.lens)
    ws = torch.empty(B.bfly_cache_attention_workspace_bytes(2, 8, 2, 128, b.width * 16), dtype=U8,
                     device="cuda")
    slots = ints(b.slots[:7])
    k, v = (torch.randn((7, 2, 128), device="cuda") for _ in "kv")
    b.run(tables=t, lens=n, workspace=ws)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        b.cache.write(k, v, slots)
        b.cache.read(slots, k, v)
        b.run(tables=t, lens=n, workspace=ws)
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]) == before


def test_as_many_rows_as_there_may_be():
    """2^24 - 1 rows of one head and one token or none: y is the token's value."""
    rows, d, page, pages = (1 << 24) - 1, 64, 16, 10
    c = Cache("int8", pages, 1, page, d, junk=False)
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((pages * page, 1, d), device="cuda") for _ in "kv")
    c.write(k, v, slots)
    c.read(slots, k, v)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    tables, lens = (at % pages)[:, None].contiguous(), at // 3 % 2
    q = torch.zeros((rows, 1, d), dtype=BF16, device="cuda")
    y = torch.full_like(q, 7.0)
    B.bfly_cache_attention(q, c.k, c.v, tables, lens, y, **c.scales)
    first = v[::page].to(BF16)                       # of every page
    for part in torch.arange(rows, device="cuda").split(1 << 22):
        want = torch.where((lens[part] > 0)[:, None, None], first[tables[part, 0].long()], 0.0)
        # 448 codes and one weight of 1 over itself: the result's rounding only
        assert ((y[part] - want).abs() <= 2.0 ** -7 * want.abs()).all()


@pytest.mark.parametrize("rows,heads", [(512, 32), (1, 1024)])
def test_tables_as_wide_as_they_may_be(rows, heads):
    """Tables of 2^30 tokens, whose product with rows and heads passes 2^44, and
    short sequences: no bound of their lengths is given."""
    d, page, most = 64, 65536, 100
    c = Cache("int4", 1, heads, page, d, junk=False)
    g = torch.Generator(device="cuda").manual_seed(rows)
    slots = torch.arange(most, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((most, heads, d), generator=g, device="cuda") for _ in "kv")
    c.write(k, v, slots)
    c.read(slots, k, v)
    tables = torch.full((rows, 16384), -1, dtype=torch.int32, device="cuda")
    tables[:, 0] = 0
    lens = torch.arange(rows, dtype=torch.int32) * 37 % (most + 1)
    lens[0] = most
    q = torch.randn((rows, heads, d), generator=g, device="cuda")
    y, lse = torch.full_like(q, 7.0), torch.empty((rows, heads), device="cuda")
    B.bfly_cache_attention(q, c.k, c.v, tables, lens.cuda(), y, lse=lse, **c.scales)
    for r in sorted({0, 1, rows // 2, rows - 1} & set(range(rows))):
        want, wl = reference(q[r:r + 1], k[None], v[None], lens[r:r + 1], d ** -0.5)
        size, _ = reference(q[r:r + 1], k[None], v[None].abs(), lens[r:r + 1], d ** -0.5)
        # as for many rows: scores 2^-16, sums of 100 terms 2^-17
        assert ((y[r:r + 1].double() - want).abs() <= 2.0 ** -13 * size + 2.0 ** -40).all(), r
        assert (lse[r:r + 1].double() - wl).abs().max() <= 2.0 ** -13
