"""bfly_cache_attention where a value's scale or a score lies at an end of its
range."""
import math

import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B
from test_gpu_cache import BF16, F32, TOP, U, Batch, gpu, ints, np64  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def ahead(b, token, score):
    """Keys of standard normals, but those of `token`, whose score with the
    queries of `b` (one to a key-value head) is `score`."""
    rng = np.random.default_rng(50 + token)
    k = rng.standard_normal((sum(b.lens), b.kv, b.d)).astype(np.float32)
    q = np64(b.q)[0]
    k[token] = q * (score * b.d ** 0.5 / (q * q).sum(1, keepdims=True))
    return k


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "int4"])
@pytest.mark.parametrize("q,y", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n", [400, 3000])
def test_a_row_of_zeros_takes_no_bits_from_the_others(fmt, q, y, n):
    """A token whose value is zero (scale 0) at the others' score and far above
    them, in one chunk and in several: the others' weights have the bits that
    they have without it.  The tolerance is the formula's, where a zero row
    counts as nothing in the products with the codes; its part of the exponent,
    60 at most, is within the 4 u (|s| + 41) that a score may be off by."""
    for scale, gap in ((1e-6, 0), (1e-4, 0), (1e-3, 10), (1e-3, 16), (1e-4, 20), (1e-2, 30)):
        v = np.random.default_rng(n).standard_normal((n, 2, 64)).astype(np.float32)
        v *= np.float32(scale * TOP[fmt] / 3)
        v[37] = 0.0
        same = dict(heads=2, kv=2, d=64, page=16, q=q, y=y, seed=40)
        k = np.zeros_like(v)
        k = ahead(Batch(fmt, [n], k=k, v=v, **same), 37, gap)
        b = Batch(fmt, [n], k=k, v=v, **same)
        b.run()
        b.check()
        assert (b.y != 0).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "int4"])
def test_rows_of_zeros_only(fmt):
    """y = 0, and the log-sum counts them."""
    for n in (1, 50, 3000):
        v = np.zeros((n, 2, 64), np.float32)
        b = Batch(fmt, [n], 4, 2, 64, 16, y=F32, seed=41, v=v,
                  k=np.random.default_rng(n).standard_normal((n, 2, 64)).astype(np.float32))
        b.run()
        b.check()
        assert (b.y == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "int4"])
@pytest.mark.parametrize("q,y", [(BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("n", [50, 3000])
def test_scores_as_large_as_fp32_holds(fmt, q, y, n):
    """Scores of 1e36 from queries of 1e38 and keys of 1e-3: the largest, five
    times the others' standard deviations and more ahead of them, has all the
    weight.  y is its value to the roundings of the scale's inverse and the
    division (4 u) and its own, lse its score to those of 64 products of up to 24
    bits and three factors (72 u of sum |q k|, 2^-22 of it for an fp32 query's)."""
    rng = np.random.default_rng(n)
    k = (1e-3 * rng.standard_normal((n, 2, 64))).astype(np.float32)
    b = Batch(fmt, [n], 2, 2, 64, 16, q, y, seed=42)
    b.q = (b.q.float() * 5e37).clamp(-2e38, 2e38).to(q)
    aim = np64(b.q)[0]
    k[7] = 2e-3 * aim / np.sqrt((aim * aim).mean(1, keepdims=True))
    v = rng.standard_normal(k.shape).astype(np.float32)
    b.cache.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), ints(b.slots))
    b.run()
    keys, values = b.cache.rows()
    half = 2.0 ** -8 if y == BF16 else U
    for h in range(2):
        s = keys[b.slots, h] @ aim[h] / 8
        a = (np.abs(keys[b.slots, h]) @ np.abs(aim[h])).max() / 8
        off = (72 * U + (2.0 ** -22 if q == F32 else 0.0)) * a
        assert np.argmax(s) == 7 and s[7] > 1e35 and s[7] - np.delete(s, 7).max() > 100 * off
        want = values[b.slots[7], h]
        assert (np.abs(np64(b.y)[0, h] - want) <= (4 * U + half) * np.abs(want)).all()
        assert abs(np64(b.lse)[0, h] - s[7]) <= off + 4 * U * s[7]


@pytest.mark.parametrize("y", [BF16, F32])
@pytest.mark.parametrize("n", [300, 5000])
def test_an_infinite_value_of_a_small_weight(y, n):
    """A weight of 2^-90 of the largest and above makes an infinity the result's,
    in the largest's wave and chunk and in others, before it and behind it."""
    for token, score in ((5, 0.0), (38, 0.0), (n - 1, 0.0), (5, -4.0), (n - 2, -4.0)):
        v = np.random.default_rng(n).standard_normal((n, 2, 64)).astype(np.float32)
        v[token, :, 3], v[token, :, 4] = np.inf, -np.inf
        same = dict(heads=2, kv=2, d=64, page=16, q=F32, y=y, seed=43)
        b = Batch("bf16", [n], k=np.zeros_like(v), v=v, **same)
        k = ahead(b, 37, 58.0)
        k[token] = k[37] * np.float32(score / 58.0)
        b = Batch("bf16", [n], k=k, v=v, **same)
        b.run()
        got = np64(b.y)[0]
        assert (got[:, 3] == np.inf).all() and (got[:, 4] == -np.inf).all()
        assert np.isfinite(np.delete(got, (3, 4), 1)).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "int4"])
@pytest.mark.parametrize("n", [300, 2000])
def test_scores_whose_last_bit_is_more_than_one(fmt, n):
    """Scores of up to 2^40, where fp32 has steps of 1, 2, 4 ... in the exponent of
    a weight.  All alike, they give the values' mean: n weights of 1 exactly, their
    sum and the values' scales (n + 64 u in all).  Over a quantized cache the
    exponent is u = s + log2 vs, rounded once, by half a step of s: 2^(E - 25) for
    |u| < 2^E, whatever the size of log2 vs.  Weights that should be 1 then lie
    between 1 / f and f = 2^(2^(E - 25)), each over their sum between 1 / (n f^2)
    and f^2 / n, so that y is off by up to f^2 - 1 of the largest value.  Apart by a
    few steps, the larger ones later, they have no weights to compare with, but a
    result between the values' least and largest, to the sums' roundings."""
    d, kv, heads = 64, 2, 4
    rng = np.random.default_rng(n)
    v = rng.standard_normal((n, kv, d)).astype(np.float32)
    alike = np.zeros((n, kv, d), np.float32)
    alike[:, :, 0] = 7.0
    apart = alike.copy()
    apart[:, :, 1] = (np.arange(n) * 8 // n)[:, None]            # codes 0 ... 7 of int4 too
    tol = (n + 64) * U
    for k in (alike, apart):
        b = Batch(fmt, [n], heads, kv, d, 16, F32, F32, seed=44, k=k, v=v)
        values = b.cache.rows()[1][b.slots]
        for power in range(18, 41):
            for sign in (1.0, -1.0):
                b.q.zero_()
                b.q[:, :, 0], b.q[:, :, 1] = sign * 2.0 ** power, 8.0
                for scale in (0.1, 0.125, 0.13):
                    b.out()
                    b.run(scale=scale)
                    got = np64(b.y)[0].reshape(kv, heads // kv, d)
                    size = np.abs(values).max(0)[:, None]
                    assert (got >= values.min(0)[:, None] - tol * size).all(), (power, sign, scale)
                    assert (got <= values.max(0)[:, None] + tol * size).all(), (power, sign, scale)
                    if k is alike:
                        e = math.ceil(math.log2(7 * 2.0 ** power * scale / math.log(2) + 32))
                        more = 0.0 if fmt == "bf16" else 4.0 ** (2.0 ** min(e - 25, 3)) - 1
                        off = np.abs(got - values.mean(0)[:, None])
                        assert (off <= (tol + more) * size).all(), (power, sign, scale)
