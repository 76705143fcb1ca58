"""bfly_cache_write, bfly_cache_read and bfly_cache_attention against their
formulas in 64 bits, written in numpy from the bytes of a cache."""
import math

import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8
FORMATS = ("bf16", "int8", "e4m3", "int4")
TOP = {"int8": 127.0, "e4m3": 448.0, "int4": 7.0}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------
# a cache on the host: what its bytes stand for
# ---------------------------------------------------------------------------

def e4m3_value(byte):
    """The number that a byte stands for: 1 sign, 4 exponent, 3 mantissa bits."""
    b = byte.astype(np.int64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(b & 128, -v, v)


def e4m3_round(v):
    """To the nearest of those numbers, ties to even, at most 448."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), v)


def numbers(cache, fmt):
    """[pages, kv, page, d] of a cache tensor's bytes, before the scales."""
    if fmt == "bf16":
        return np64(cache)
    b = cache.view(U8).cpu().numpy()
    if fmt == "int8":
        return b.view(np.int8).astype(np.float64)
    if fmt == "e4m3":
        return e4m3_value(b)
    both = np.stack([b & 15, b >> 4], axis=-1).reshape(*b.shape[:-1], -1).astype(np.int64)
    return np.where(both > 7, both - 16, both).astype(np.float64)


def definition(x, fmt):
    """(numbers, fp16 scales) of rows in 64 bits."""
    if fmt == "bf16":
        return np64(torch.from_numpy(x).to(BF16)) if x.dtype == np.float32 else x, None
    x = x.astype(np.float64)
    top = np.abs(x).max(-1)
    with np.errstate(all="ignore"):
        s = np.minimum(top / TOP[fmt], 65504.0).astype(np.float16)
        d = s.astype(np.float64)[..., None]
        q = np.where(d > 0, x / np.where(d > 0, d, 1.0), 0.0)
        q = np.clip(q, -TOP[fmt], TOP[fmt])
        q = e4m3_round(q) if fmt == "e4m3" else np.rint(q)
    bad = np.isnan(x).any(-1)
    s[bad], q[bad] = np.nan, 0.0
    return q, s


class Cache:
    """Pages of a cache, filled with what no call may read: NaN where the
    format has one, its largest code else, and NaN scales."""

    def __init__(self, fmt, pages, kv, page, d, junk=True):
        self.fmt, self.pages, self.kv, self.page, self.d = fmt, pages, kv, page, d
        new = lambda *s: torch.full(s, 0x7F if junk else 0, dtype=U8, device="cuda")
        if fmt == "bf16":
            self.k, self.v = (torch.full((pages, kv, page, d), math.nan if junk else 0.0, dtype=BF16,
                                         device="cuda") for _ in "kv")
            self.ks = self.vs = None
        else:
            w = d // 2 if fmt == "int4" else d
            t = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "int4": U8}[fmt]
            self.k, self.v = (new(pages, kv, page, w).view(t) for _ in "kv")
            self.ks, self.vs = (torch.full((pages, kv, page), math.nan if junk else 0.0, dtype=F16,
                                           device="cuda") for _ in "kv")

    @property
    def scales(self):
        return {"k_scales": self.ks, "v_scales": self.vs}

    def write(self, k, v, slots, stream=None):
        B.bfly_cache_write(k, v, slots, self.k, self.v, stream=stream, **self.scales)

    def read(self, slots, k, v, stream=None):
        B.bfly_cache_read(self.k, self.v, slots, k, v, stream=stream, **self.scales)

    def rows(self):
        """[slots, kv, d] keys and values, scales applied, in 64 bits."""
        out = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            x = numbers(c, self.fmt)
            if s is not None:
                with np.errstate(all="ignore"):
                    x = x * np64(s)[..., None]
            out.append(x.transpose(0, 2, 1, 3).reshape(-1, self.kv, self.d))
        return out

    def state(self):
        return [t.view(U8).clone() for t in (self.k, self.v, self.ks, self.vs) if t is not None]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# written and read back
# ---------------------------------------------------------------------------

def special_rows(x):
    """Rows where a quantizer can go wrong, in the first tokens of x."""
    n, kv, d = x.shape
    for t, row in enumerate((
            lambda: np.zeros(d), lambda: np.full(d, -0.0),
            lambda: np.full(d, 3.0e-8),                        # scale below fp16's smallest
            lambda: np.linspace(-1, 1, d) * 2.0 ** -20,        # a subnormal scale
            lambda: np.linspace(-1, 1, d) * 1e-42,
            lambda: np.linspace(-1, 1, d) * 3.0e38,            # a saturated scale
            lambda: np.where(np.arange(d) == 5, 7.0, (np.arange(d) % 15 - 7) / 2.0),   # int4 ties
            lambda: np.where(np.arange(d) == 6, -127.0, (np.arange(d) % 250 - 125) / 2.0),
            lambda: np.where(np.arange(d) == 7, 448.0, 2.0 ** -9 * (np.arange(d) % 9 - 4) / 2.0),
            lambda: np.where(np.arange(d) == d - 1, np.inf, 1.0),
            lambda: np.where(np.arange(d) == d - 1, -np.inf, 1e5),
            lambda: np.where(np.arange(d) == 0, np.nan, 1.0),
            lambda: np.where(np.arange(d) == d - 1, np.nan, np.inf))):
        if t < n:
            x[t, t % kv] = row()
    return x


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("tokens,kv,page", [(1, 1, 16), (33, 3, 16), (300, 8, 64), (7, 40, 32)])
def test_write_and_read(fmt, d, dt, tokens, kv, page):
    rng = np.random.default_rng(tokens + kv)
    pages = -(-tokens // page) + 4
    x = [special_rows(rng.standard_normal((tokens, kv, d)) *
                      np.exp(2 * rng.standard_normal((tokens, kv, 1)))) for _ in "kv"]
    with np.errstate(over="ignore"):
        k, v = (torch.from_numpy(a.astype(np.float32)).to(dt) for a in x)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    out = rng.random(tokens) < 0.2
    slots[out] = rng.choice([-1, -2 ** 31, pages * page, pages * page + 5, 2 ** 31 - 1], out.sum())
    c = Cache(fmt, pages, kv, page, d)
    before = c.state()
    c.write(k.cuda(), v.cuda(), ints(slots))
    at = slots[~out]
    where = (at // page, slice(None), at % page)
    for t, s, src, was in ((c.k, c.ks, k, before[0]), (c.v, c.vs, v, before[1])):
        q, scale = definition(src.float().numpy()[~out], fmt)
        got = numbers(t, fmt)[where]
        assert np.array_equal(got, q, equal_nan=True)
        if s is not None:
            assert np.array_equal(s.cpu().numpy()[where], scale, equal_nan=True)
        # the other slots as they were
        rest = np.ones((pages, page), bool)
        rest[at // page, at % page] = False
        here = t.view(U8).cpu().numpy().transpose(0, 2, 1, 3)[rest]
        assert np.array_equal(here, was.cpu().numpy().transpose(0, 2, 1, 3)[rest])
        if s is not None:
            assert np.isnan(s.cpu().numpy().transpose(0, 2, 1)[rest]).all()
    # read back, some slots twice, the excluded ones as zeros; code * scale has
    # at most 19 bits, so that fp32 is exact and bf16 its rounding
    twice = np.concatenate([slots, at[::2]])
    rows = c.rows()
    for to in (F32, BF16):
        wide = torch.full((len(twice), kv + 2, d), 7.0, dtype=to, device="cuda")
        other = torch.full((len(twice), kv, d), 7.0, dtype=to, device="cuda")
        c.read(ints(twice), wide[:, 1:kv + 1], other)
        gone = (twice < 0) | (twice >= pages * page)
        for got, src in ((wide[:, 1:kv + 1], rows[0]), (other, rows[1])):
            want = np.where(gone[:, None, None], 0.0, src[np.where(gone, 0, twice)])
            want = torch.from_numpy(want).float().to(to)
            assert torch.equal(got.cpu().nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))
        assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()


def test_rows_of_a_projection_and_no_tokens():
    """k and v as views into the projection's output; zero tokens."""
    kv, d, heads = 4, 128, 12
    c, e = (Cache("int4", 6, kv, 16, d) for _ in "ab")
    qkv = torch.randn((37, heads + 2 * kv, d), device="cuda").to(BF16)
    k, v = qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    slots = ints(np.random.default_rng(0).permutation(96)[:37])
    c.write(k, v, slots)
    e.write(k.contiguous(), v.contiguous(), slots)
    assert all(torch.equal(a, b) for a, b in zip(c.state(), e.state()))
    c.write(k[:0], v[:0], slots[:0])
    c.read(slots[:0], k[:0].clone(), v[:0].clone())
    assert all(torch.equal(a, b) for a, b in zip(c.state(), e.state()))
    one = Cache("int4", 6, kv, 16, d)
    one.write(k[5:6], v[5:6], slots[5:6])
    s = int(slots[5])
    assert torch.equal(one.k[s // 16, :, s % 16], c.k[s // 16, :, s % 16])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Batch:
    """Sequences of the given lengths in a cache whose other slots hold junk,
    their pages anywhere, the tables' rest beyond every page."""

    def __init__(self, fmt, lens, heads, kv, d, page, q=BF16, y=BF16, seed=0, width=None,
                 peaked=1.5, spread=0.5, k=None, v=None):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv, self.d, self.page, self.fmt = lens, heads, kv, d, page, fmt
        need = [-(-n // page) for n in lens]
        self.width = width or max(1, *need)
        pages = sum(need) + 2
        order, self.tables, at = rng.permutation(pages), np.full((len(lens), self.width), pages), 0
        for r, n in enumerate(need):
            self.tables[r, :n], at = order[at:at + n], at + n
        self.tables[:, :] = np.where(self.tables == pages, rng.choice(
            [-1, pages, 2 ** 31 - 1, -2 ** 31], self.tables.shape), self.tables)
        self.cache = Cache(fmt, pages, kv, page, d)
        tokens = sum(lens)
        new = lambda: rng.standard_normal((tokens, kv, d)).astype(np.float32)
        k = new() if k is None else k
        v = new() * np.exp(spread * rng.standard_normal((tokens, kv, 1))).astype(np.float32) \
            if v is None else v
        self.slots = np.concatenate([self.tables[r, np.arange(n) // page] * page + np.arange(n) % page
                                     for r, n in enumerate(lens)] + [np.zeros(0)]).astype(np.int64)
        if tokens:
            self.cache.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), ints(self.slots))
        self.q = (torch.from_numpy(rng.standard_normal((len(lens), heads, d))) * peaked).to(q).cuda()
        self.ydt = y
        self.out()

    def out(self):
        n = len(self.lens)
        self.y = torch.full((n, self.heads, self.d), 7.0, dtype=self.ydt, device="cuda")
        self.lse = torch.full((n, self.heads), 7.0, device="cuda")

    def run(self, q=None, tables=None, lens=None, **more):
        c = self.cache
        given = dict(lse=self.lse, **c.scales)
        given.update(more)
        B.bfly_cache_attention(self.q if q is None else q, c.k, c.v,
                               ints(self.tables) if tables is None else tables,
                               ints(self.lens) if lens is None else lens, self.y, **given)
        return self.y, self.lse

    def check(self, window=0, scale=None, tables=None, lens=None, q=None):
        """y and lse against the formula.  A score is a sum of d exact products
        held in fp32, times two factors (the scale of a key, `scale`), and is
        compared and shifted in units of log 2: e = (d + 8) u A for
        A = scale sum_i |q_i k_i|, plus 4 u (|s| + |log vs| + 32); fp32 queries
        enter with 22 bits (2^-22 A; 24 over a bf16 cache).  A weight then is
        off by 2 e (its own score and the shift's), the exponential's and the
        scales' roundings (16 u) and its own: 2^-11 with bf16 q and y (2^-15
        over bf16 caches), 2^-22 else.  y is off by as much of sum p |v|, for
        the weights and, less their own rounding, for their sum, by the fp32
        sums, (tokens + 64) u of them, and by its own rounding.  Over a
        quantized cache a weight is e^(s - m) times the value's scale in fp16,
        the largest at 2^8 or above: what is below 2^-14 there is held to half
        of fp16's smallest step, 2^-25, which is 2^-33 of the largest, and
        multiplies the value's codes."""
        c = self.cache
        keys, values = c.rows()
        if c.vs is not None:
            scales = np64(c.vs).transpose(0, 2, 1).reshape(-1, c.kv)
        tables = self.tables if tables is None else tables
        lens = self.lens if lens is None else lens
        scale = self.d ** -0.5 if scale is None else scale
        exact = self.q.dtype == F32 or self.ydt == F32
        own = 2.0 ** -22 if exact else 2.0 ** -15 if self.fmt == "bf16" else 2.0 ** -11
        q64 = np64(self.q if q is None else q)
        got, lse = np64(self.y), np64(self.lse)
        half = 2.0 ** -8 if self.ydt == BF16 else U
        share, worst = self.heads // self.kv, 0.0
        for r, n in enumerate(lens):
            at = np.arange(max(0, n - window) if window else 0, max(0, n))
            page = tables[r, at // self.page]
            ok = (page >= 0) & (page < c.pages)
            slot = page[ok] * self.page + at[ok] % self.page
            if len(slot) == 0:
                assert (got[r] == 0).all() and (lse[r] == -np.inf).all()
                continue
            for h in range(self.heads):
                k, v = keys[slot, h // share], values[slot, h // share]
                s = scale * (k @ q64[r, h])
                m = s.max()
                p = np.exp(s - m)
                total = p.sum()
                p /= total
                a = abs(scale) * (np.abs(k) @ np.abs(q64[r, h])).max()
                vs = np.abs(v).max(1)
                logs = np.abs(np.log2(np.where(vs > 0, vs, 1.0))).max() + 9
                e = (self.d + 8) * U * a + 4 * U * (np.abs(s).max() + logs + 32)
                e += 2.0 ** -22 * a if self.q.dtype == F32 else 0.0
                weight = 1.01 * (2 * e + 16 * U)
                sums = (len(slot) + 64) * U
                tol = (2 * weight + own + 2 * sums) * (p @ np.abs(v))
                want = p @ v
                if self.fmt != "bf16":
                    sc = scales[slot, h // share]
                    codes = np.abs(v) / np.where(sc > 0, sc, 1.0)[:, None]
                    tol += 1.01 * 2.0 ** -33 * (p * sc).max() * codes.sum(0)
                tol += half * (np.abs(want) + tol) + 1e-37
                err = np.abs(got[r, h] - want)
                assert (err <= tol).all(), (r, h, n, float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
                want = m + math.log(total)
                assert abs(lse[r, h] - want) <= weight + sums + 2 * U * abs(want) + 64 * U, (r, h)
        return worst


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 255, 257]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q,y", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_attention(fmt, d, q, y):
    b = Batch(fmt, LENS, 6, 2, d, 16, q, y, seed=d)
    b.run()
    b.check()


@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (8, 4), (7, 1), (16, 1), (17, 1), (40, 2),
                                      (33, 1), (64, 1)])
def test_heads(heads, kv):
    for fmt in ("int4", "bf16"):
        b = Batch(fmt, [50, 0, 300], heads, kv, 64, 32, seed=heads)
        b.run()
        b.check()


@pytest.mark.parametrize("page", [16, 32, 64, 256, 65536])
def test_pages(page):
    for fmt in ("int8", "bf16"):
        b = Batch(fmt, [700, 1, 33, 257, 256], 4, 2, 128, page, seed=page)
        b.run()
        b.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 7, 16, 31, 32, 33, 100, 255, 1000, 1 << 30])
def test_window(fmt, window):
    lens = [0, 1, 7, 16, 40, 100, 131, 300, 1200]
    b = Batch(fmt, lens, 4, 2, 64, 16, seed=window % 97)
    b.run(window=window, max_len=1200)
    b.check(window=window)
    # the pages in front of the window are given back: their entries say nothing
    t = b.tables.copy()
    for r, n in enumerate(lens):
        t[r, :max(0, n - window) // 16] = -1
    b.out()
    b.run(window=window, max_len=1200, tables=ints(t))
    b.check(window=window, tables=t)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,kv,n", [(8, 2, 20011), (4, 4, 5000), (3, 1, 70000)])
def test_long(fmt, heads, kv, n):
    b = Batch(fmt, [n, 0, 300, n // 2], heads, kv, 64, 64, y=F32, seed=3)
    b.run()
    b.check()


def test_scale_and_bounds():
    b = Batch("int8", [100, 40, 7, 64], 4, 2, 128, 16, y=F32, seed=4, width=20)
    for scale in (0.0, -0.3, 2.0, 1e-30):
        b.run(scale=scale)
        b.check(scale=scale)
    # any bound that holds gives the formula; a length below 0 is 0, one above
    # the bound is the bound
    for most in (100, 128, 320, None):
        b.out()
        b.run(lens=ints([100, -5, 7, 64]), max_len=most)
        b.check(lens=[100, -5, 7, 64])
    first = b.run(max_len=64, lens=ints([64, 40, 7, 64]))[0].clone()
    again = b.run(max_len=64, lens=ints([100, 40, 7, 2 ** 31 - 1]))[0]
    assert torch.equal(first, again)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_that_are_not_there(fmt):
    """Tokens of table entries outside the cache are out of reach."""
    b = Batch(fmt, [200, 90, 48, 33], 6, 2, 64, 16, y=F32, seed=5)
    t = b.tables.copy()
    t[0, 3], t[0, 12], t[1, 0] = -1, 2 ** 31 - 1, b.cache.pages
    t[2, :] = -7                                       # nothing in reach
    b.run(tables=ints(t))
    b.check(tables=t)
    # also where the length is split
    c = Batch(fmt, [5000, 600], 2, 1, 64, 16, y=F32, seed=6)
    t = c.tables.copy()
    t[0, 40:200] = -1
    t[1, :] = c.cache.pages + 3
    c.run(tables=ints(t))
    c.check(tables=t)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q", [BF16, F32])
def test_extremes(fmt, q):
    """One token far above the rest; values of sizes far apart; large and small
    queries; rows of zeros."""
    d, n = 64, 400
    rng = np.random.default_rng(7)
    base = lambda: rng.standard_normal((n, 2, d)).astype(np.float32)
    far = np.exp(np.where(rng.random((n, 2, 1)) < 0.5, -9.0, 8.0)).astype(np.float32)
    zeros = base()
    zeros[::3] = 0.0
    for k, v, peaked in ((base(), base() * far, 1.0), (zeros, zeros[::-1].copy(), 1.0),
                         (base(), base(), 40.0), (base() * 1e-4, base() * far, 1e4),
                         (base(), base(), 1e-9), (base() * 1e4, base() * 1e4, 1e-3)):
        b = Batch(fmt, [n], 4, 2, d, 16, q, F32, seed=8, peaked=peaked, k=k, v=v)
        b.run()
        b.check()
    # a token that the small values hang on: all others' weights times values vanish
    k, v = base(), base() * 1e3
    b = Batch(fmt, [n], 4, 2, d, 16, q, F32, seed=9, k=k, v=v)
    best = torch.from_numpy(np64(b.q)[0].reshape(2, 2, d).mean(1) * 6).float()
    k[37], v[37] = best.numpy(), 1e-2 * v[37]
    b = Batch(fmt, [n], 4, 2, d, 16, q, F32, seed=9, k=k, v=v)
    b.run()
    b.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_nan_stays_where_it_is(fmt):
    lens = [70, 300, 40]
    make = lambda: Batch(fmt, lens, 4, 2, 64, 16, seed=10)
    a, b = make(), make()
    a.run()
    # a key of the second sequence's first head, a value of its last token's second
    nan = torch.full((1, 2, 64), 1.0, device="cuda")
    nan[0, 0, 3] = math.nan
    fine = torch.ones_like(nan)
    slot = b.slots[lens[0] + 5]
    b.cache.write(nan, fine, ints([slot]))
    b.run()
    y, l = b.y.clone(), b.lse.clone()
    assert torch.isnan(y[1, :2]).all() and torch.isnan(l[1, :2]).all()
    assert torch.isfinite(y[1, 2:].float()).all() and torch.isfinite(l[1, 2:]).all()
    assert torch.equal(y[[0, 2]], a.y[[0, 2]]) and torch.equal(l[[0, 2]], a.lse[[0, 2]])
    # out of the window it is not seen
    b.run(window=100, max_len=300)
    assert torch.isfinite(b.y.float()).all()
    # a query's NaN or infinity: its own head only, and not where nothing is in reach
    for bad in (math.nan, math.inf, -math.inf):
        q = a.q.clone()
        q[1, 3, 17] = bad
        c = make()
        c.run(q=q)
        assert torch.isnan(c.y[1, 3]).all() and torch.isnan(c.lse[1, 3])
        keep = torch.ones((3, 4), dtype=torch.bool, device="cuda")
        keep[1, 3] = False
        assert torch.equal(c.y[keep], a.y[keep]) and torch.equal(c.lse[keep], a.lse[keep])
        c.run(q=q, lens=ints([70, 0, 40]))
        assert (c.y[1] == 0).all() and (c.lse[1] == -math.inf).all()
        c.run(q=q, tables=ints(np.where(np.arange(3)[:, None] == 1, -1, c.tables)))
        assert (c.y[1] == 0).all() and (c.lse[1] == -math.inf).all()


def test_infinite_values_of_a_bf16_cache():
    """A value's infinity is the result's, by its sign, in fp32 and bf16."""
    for y in (F32, BF16):
        b = Batch("bf16", [50], 2, 1, 64, 16, y=y, seed=11)
        v = torch.randn((1, 1, 64), device="cuda")
        v[0, 0, 5], v[0, 0, 6] = math.inf, -math.inf
        b.cache.write(torch.zeros_like(v), v, ints([b.slots[20]]))
        b.run()
        got = b.y.float().cpu()
        assert (got[0, :, 5] == math.inf).all() and (got[0, :, 6] == -math.inf).all()
        rest = [i for i in range(64) if i not in (5, 6)]
        assert torch.isfinite(got[0][:, rest]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_row_depends_on_itself_only(fmt):
    """Same bits from run to run, and whatever the other rows of a call are."""
    lens = [700, 0, 33, 1025, 4000, 128]
    b = Batch(fmt, lens, 8, 2, 64, 16, seed=12)
    y, l = (t.clone() for t in b.run(max_len=4096, tables=ints(np.pad(b.tables, ((0, 0), (0, 6)), constant_values=-1))))
    order = [4, 2, 0, 5, 1, 3]
    t = np.pad(b.tables, ((0, 0), (0, 6)), constant_values=-1)
    b.out()
    b.run(q=b.q[order].contiguous(), tables=ints(t[order]), lens=ints([lens[i] for i in order]),
          max_len=4096)
    assert torch.equal(b.y, y[order]) and torch.equal(b.lse, l[order])
    some = [0 if i != 3 else lens[3] for i in range(6)]
    b.run(tables=ints(t), lens=ints(some), max_len=4096)
    assert torch.equal(b.y[3], y[3]) and (b.y[[0, 1, 2, 4, 5]] == 0).all()


def test_views_and_shared_pages():
    """q as a view into the projection's output; sequences over the same pages."""
    b = Batch("int4", [300, 40], 6, 2, 128, 32, y=F32, seed=13)
    wide = torch.randn((2, 10, 128), device="cuda").to(BF16)
    wide[:, :6] = b.q
    b.run(q=wide[:, :6])
    b.check()
    t = b.tables.copy()
    t[1] = t[0]
    b.run(tables=ints(t), lens=ints([300, 299]))
    b.check(tables=t, lens=[300, 299])


def test_without_a_workspace_and_with_one_that_holds_anything():
    b = Batch("int8", [3000, 100], 4, 2, 64, 16, seed=14)
    y = b.run()[0].clone()
    need = B.bfly_cache_attention_workspace_bytes(2, 4, 2, 64, b.width * 16)
    assert need > 0
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need + 64,), fill, dtype=U8, device="cuda")
        b.out()
        b.run(workspace=ws[:need])
        assert torch.equal(b.y, y) and (ws[need:] == fill).all()
    b.run(lse=None)
    assert torch.equal(b.y, y)


def test_no_rows():
    b = Batch("int8", [30], 4, 2, 64, 16)
    B.bfly_cache_attention(b.q[:0], b.cache.k, b.cache.v, ints(b.tables)[:0], ints(b.lens)[:0],
                           b.y[:0], **b.cache.scales)
    assert (b.y == 7).all()


def test_past_32_bit_offsets():
    """A cache of 5 GB a side: the last pages, and pages above 2^32 bytes."""
    kv, page, d, pages = 8, 64, 256, 20000
    assert pages * kv * page * d * 2 > 1 << 32
    c = Cache.__new__(Cache)
    c.fmt, c.pages, c.kv, c.page, c.d, c.ks, c.vs = "bf16", pages, kv, page, d, None, None
    c.k, c.v = (torch.empty((pages, kv, page, d), dtype=BF16, device="cuda") for _ in "kv")
    ids = [19999, 3, 16500, 17001, 19998]
    n = 5 * page - 9
    slots = np.array([ids[t // page] * page + t % page for t in range(n)])
    k, v = (torch.randn((n, kv, d), device="cuda").to(BF16) for _ in "kv")
    c.write(k, v, ints(slots))
    back = [torch.empty_like(k) for _ in "kv"]
    c.read(ints(slots), *back)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    q = torch.randn((1, 2 * kv, d), device="cuda").to(BF16)
    y = torch.empty((1, 2 * kv, d), device="cuda")
    B.bfly_cache_attention(q, c.k, c.v, ints([ids]), ints([n]), y)
    small = Batch("bf16", [n], 2 * kv, kv, d, page, y=F32, k=k.float().cpu().numpy(),
                  v=v.float().cpu().numpy())
    small.q = q
    small.run()
    small.check()
    assert torch.equal(y, small.y)
