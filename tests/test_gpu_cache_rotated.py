"""Attention over a cache of rotated keys by rotated queries is attention over
the keys and queries that were rotated."""
import pytest

from test_gpu_cache import BF16, TOP, gpu  # noqa: F401
from test_gpu_cache_more import Decoder

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt,size", [("bf16", 1.0), ("int8", 1.0), ("e4m3", 0.5), ("int4", 0.5)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rotated_heads_have_the_products_they_had(fmt, size, d):
    """Twenty decode steps of three sequences, the keys with an outlier channel.

    The scores, element by element: with q', k' the rotated rows in bf16 and c
    what the cache holds of k', and R orthogonal,
      q' c - q k = q' (c - k') + q' (k' - R k) + (q' - R q) R k,
    where a rounding to bf16 is 2^-8 of its result (1.01 for the next order),
    the rotation's own fp32 errors are below 2^-18 |q| |k|, and a code is off by
    half a step: scale / 2 (int8, int4), 2^-4 of it or 2^-10 scale (e4m3), and by
    top 2^-11 scale more where the scale's rounding cuts the largest.

    The results: weights p' from the scores as the cache has them differ from p,
    from the scores of the given rows, by what they differ; y is off by sum
    |p' - p| |v| and a call's own tolerance (bf16 result 2^-8, weight 2^-11,
    score and sums 2^-12 here).  Against the same tolerance no y, its negative
    and the values' mean are wrong in most elements."""
    rows, heads, kv, steps = 3, 6, 2, 20
    dec = Decoder(fmt, rows, heads, kv, d, 64, seed=d + 1)
    g = torch.Generator().manual_seed(2)
    given, rotated = [], []
    for _ in range(steps):
        x = torch.randn((rows, heads + 2 * kv, d), generator=g)
        x[:, :heads] *= size
        x[:, heads:heads + kv, 3] *= 8.0
        dec.qkv.copy_(x.to(BF16))
        dec.step()
        given.append(dec.qkv[:, heads:heads + kv].double())
        rotated.append(dec.rot[:, heads:heads + kv].double())
    at = torch.arange(steps, device="cuda")
    slots = (dec.tables[:, at // 16] * 16 + at % 16).reshape(-1).int()
    c, v = (torch.empty((rows * steps, kv, d), device="cuda") for _ in "kv")
    dec.cache.read(slots, c, v)

    def per_head(t):                                    # [rows, heads, tokens, d]
        return t.view(rows, steps, kv, d).repeat_interleave(heads // kv, 2).transpose(1, 2).double()

    c, v = per_head(c), per_head(v)
    k, k2 = (per_head(torch.stack(t, 1)) for t in (given, rotated))
    q, q2 = (t[:, :heads].double()[:, :, None] for t in (dec.qkv, dec.rot))
    s, s2 = ((q * k).sum(3) * d ** -0.5, (q2 * c).sum(3) * d ** -0.5)
    if fmt == "bf16":
        code = torch.zeros_like(k2)
    else:
        step = 1.001 * k2.abs().amax(3, keepdim=True) / TOP[fmt]
        half = torch.maximum(2.0 ** -4 * k2.abs(), 2.0 ** -10 * step) if fmt == "e4m3" else step / 2
        code = half + TOP[fmt] * 2.0 ** -11 * step
    off = (q2.abs() * (code + 2 * 1.01 * 2.0 ** -8 * k2.abs())).sum(3)
    off += 2.0 ** -18 * q.norm(dim=3) * k.norm(dim=3)
    assert ((s2 - s).abs() <= d ** -0.5 * off).all()

    p, p2 = torch.softmax(s, 2)[..., None], torch.softmax(s2, 2)[..., None]
    want, all_of = (p * v).sum(2), (p * v.abs()).sum(2)
    tol = ((p2 - p).abs() * v.abs()).sum(2) + 2.0 ** -8 * want.abs() + 2.0 ** -9 * all_of + 2.0 ** -20
    assert ((dec.y.double() - want).abs() <= tol).all()
    for wrong in (torch.zeros_like(want), -want, v.mean(2)):
        assert ((wrong - want).abs() > tol).double().mean() > 0.5
