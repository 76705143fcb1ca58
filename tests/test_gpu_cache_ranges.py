"""bfly_cache_attention where a value's scale or a score lies at an end of its
range."""
import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B
from test_gpu_cache import BF16, F32, TOP, Batch, gpu, np64  # noqa: F401

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
