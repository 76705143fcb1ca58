"""bfly_grad_clip on the GPU.  The sum of squares is held in fp64 (2^-52 a
rounding, at most a few thousand of them), so the norm and the factor are the
fp64 values rounded to fp32: 2^-24 relative, and one part in 10^6 of that for
the sum.  A scaled gradient is one fp32 product and one rounding to its type:
with the kernel's factor numpy reproduces its bits."""
import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16
TOL = 2.0 ** -24 * (1 + 1e-6)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def workspace(count):
    return torch.full((B.bfly_grad_clip_workspace_bytes(count),), 0x7F, dtype=torch.uint8,
                      device="cuda")


def tensors(seed, sizes, dtypes, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def check(grads, max_norm, in_place, on_gpu=None):
    dev = on_gpu or [g.cuda() for g in grads]
    before = [g.cpu() for g in dev]
    outs = None if in_place else [torch.full_like(g, 7.0) for g in dev]
    norm, ws = torch.full((2,), 7.0, device="cuda"), workspace(len(dev))
    B.bfly_grad_clip(dev, max_norm, norm, ws, outs=outs)
    torch.cuda.synchronize()
    want = float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in before)))
    got, factor = (float(v) for v in norm.cpu())
    assert abs(got - want) <= TOL * want
    # the call takes max_norm as fp32: 0.01 is 0.00999999977..., 2.2e-8 below, and
    # that value is what the formula divides
    most = float(np.float32(max_norm))
    f64 = most / want if want > most else 1.0
    assert abs(factor - f64) <= TOL * f64
    for g, o in zip(before, dev if in_place else outs):
        assert torch.equal(o.cpu(), (g.float() * np.float32(factor)).to(g.dtype))
    if not in_place:
        for g, d in zip(before, dev):
            assert torch.equal(g, d.cpu())


SIZES = [[1], [4096], [4097], [1, 1, 1], [3, 4095, 4096, 4097, 8192, 1], [24576] * 40, [5] * 500,
         [0, 7, 0, 0, 20000, 0], [5000000], [100003] * 70, [1 << 20, 3, 1 << 20]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_sizes(sizes, dtypes, in_place):
    check(tensors(len(sizes), sizes, dtypes), 0.01, in_place)


@pytest.mark.parametrize("count", [111, 112, 113, 159, 160, 161, 320, 321, 500])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_counts(count, in_place):
    # lengths of all kinds, every ninth tensor empty
    sizes = [0 if i % 9 == 4 else 1 + i * 977 % 9001 for i in range(count + (count + 4) // 8)]
    check(tensors(len(sizes), sizes, (F32, BF16), 1.0), 0.7, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("count", [3, 300])
def test_clip_many_elements(count, in_place):
    # beyond 56 MiB the norm has a launch of its own; the sizes are odd and the
    # tensors views that start anywhere
    g = torch.Generator().manual_seed(count)
    each = (70 << 20) // count
    sizes = [each - 7 * i for i in range(count)]
    flat = torch.randn(sum(sizes), generator=g).cuda()
    for dtype, grads in ((F32, flat), (BF16, flat.to(BF16))):
        check(None, 0.5, in_place, on_gpu=list(grads.split(sizes)))
        check(None, 1e9, in_place, on_gpu=list(grads.split(sizes)))


@pytest.mark.parametrize("in_place", [False, True])
def test_clip_below_the_limit(in_place):
    check(tensors(1, [4096, 100, 9999], (F32, BF16)), 1e4, in_place)


@pytest.mark.parametrize("skip", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clip_views_of_one_buffer(skip, dtype):
    # tensors that start anywhere in a flat buffer; what lies between stays
    flat = (torch.randn(60000, generator=torch.Generator().manual_seed(skip)) * 0.1).to(dtype).cuda()
    cuts = [(skip, 4096), (5001 + skip, 9000), (15000 + skip, 1), (15001 + skip, 30001)]
    views = [flat[a:a + n] for a, n in cuts]
    keep = torch.ones(60000, dtype=torch.bool, device="cuda")
    for a, n in cuts:
        keep[a:a + n] = False
    before = flat.clone()
    check(None, 0.5, True, on_gpu=views)
    assert torch.equal(before[keep], flat[keep])


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 1e30])
def test_clip_magnitudes(scale):
    # squares below and above fp32's range
    check(tensors(2, [5000, 300], (F32,), scale), 1.0, False)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_clip_not_finite(bad):
    grads = [g.cuda() for g in tensors(3, [5000, 300], (F32, BF16), 10.0)]
    grads[1][7] = bad
    before = [g.clone() for g in grads]
    norm = torch.zeros(2, device="cuda")
    B.bfly_grad_clip(grads, 1.0, norm, workspace(2))
    assert not torch.isfinite(norm[0]) and norm[1] == 1.0
    for a, b in zip(before, grads):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_clip_nothing_and_zeros():
    norm = torch.full((2,), 7.0, device="cuda")
    B.bfly_grad_clip([], 1.0, norm, workspace(0))
    assert norm.tolist() == [0.0, 1.0]
    g = torch.zeros(100, device="cuda")
    B.bfly_grad_clip([g], 1.0, norm, workspace(1))
    assert norm.tolist() == [0.0, 1.0] and (g == 0).all()
    B.bfly_grad_clip([g + 3], float("inf"), norm, workspace(1))
    assert norm.tolist() == [30.0, 1.0]


def test_clip_same_bits_every_time():
    grads = [g.cuda() for g in tensors(5, [100003] * 30, (F32,))]
    norm, ws = torch.empty(2, device="cuda"), workspace(30)
    outs = [torch.empty_like(g) for g in grads]
    first = None
    for _ in range(5):
        B.bfly_grad_clip(grads, 0.1, norm, ws, outs=outs)
        v = norm.tolist()
        first = first or v
        assert v == first


def test_clip_tensors_that_overlap():
    flat, norm = torch.ones(1000, device="cuda"), torch.empty(2, device="cuda")
    for views in ([flat, flat], [flat[:10], flat[5:20]], [flat[500:], flat[:501]],
                  [flat[:1], flat[3:9], flat[0:0], flat[8:9]]):
        with pytest.raises(ValueError):
            B.bfly_grad_clip(views, 1.0, norm, workspace(len(views)))
        with pytest.raises(ValueError):
            B.bfly_grad_clip([torch.ones_like(v) for v in views], 1.0, norm,
                             workspace(len(views)), outs=views)
    assert (flat == 1).all()
    # read twice, written to different places; and neighbours in any order
    B.bfly_grad_clip([flat, flat], 1.0, norm, workspace(2),
                     outs=[torch.empty_like(flat) for _ in range(2)])
    assert abs(float(norm[0]) - 2000 ** 0.5) <= TOL * 2000 ** 0.5
    B.bfly_grad_clip([flat[500:], flat[:0], flat[:500]], 1.0, norm, workspace(3))
    assert abs(float(norm[0]) - 1000 ** 0.5) <= TOL * 1000 ** 0.5


def test_clip_outputs_that_overlap_other_gradients():
    a, b, norm = torch.ones(300, device="cuda"), torch.ones(300, device="cuda"), \
        torch.empty(2, device="cuda")
    for grads, outs in (([a, b], [b, a]), ([a, b], [torch.empty_like(a), a]),
                        ([a[:200]], [a[1:201]]), ([a, a], [a, b])):
        with pytest.raises(ValueError):
            B.bfly_grad_clip(grads, 1.0, norm, workspace(len(grads)), outs=outs)
    assert (a == 1).all() and (b == 1).all()
    out = torch.empty_like(b)
    B.bfly_grad_clip([a, b], 1.0, norm, workspace(2), outs=[a, out])
    assert torch.equal(a, out) and (b == 1).all()
    assert abs(float(a[7]) - 600 ** -0.5) <= 4 * TOL


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1, 1], [5000, 3, 70001], [9000] * 200, [16 << 20, 16 << 20]],
                         ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_clip_norm_beyond_fp32(sizes, dtype):
    # finite gradients whose norm is not: it is reported as an infinity, with
    # factor 1, and the gradients stay as they are
    total = sum(sizes)
    flat = torch.full((total,), 3e38, device="cuda").to(dtype)
    flat[1::2] *= -1
    keep = flat.clone()
    norm, ws = torch.zeros(2, device="cuda"), workspace(len(sizes))
    out = torch.zeros_like(flat)
    for outs in (list(out.split(sizes)), None):
        norm.zero_()
        B.bfly_grad_clip(list(flat.split(sizes)), 1.0, norm, ws, outs=outs)
        assert norm.tolist() == [float("inf"), 1.0]
        assert torch.equal(flat, keep)
    assert torch.equal(out, keep)


def test_clip_norm_at_the_largest_fp32():
    # the largest finite norm still scales: the factor 1 / 3.4e38 is a subnormal,
    # off by 2^-150 at most, 2^-22 of it, and the product by 2^-24
    g = torch.full((1,), torch.finfo(F32).max, device="cuda")
    norm = torch.zeros(2, device="cuda")
    B.bfly_grad_clip([g], 1.0, norm, workspace(1))
    assert float(norm[0]) == torch.finfo(F32).max and 0 < float(norm[1]) < 3e-39
    assert abs(float(g[0]) - 1.0) <= (2.0 ** -22 + 2.0 ** -24) * (1 + 1e-3)


@pytest.mark.parametrize("count,each", [(5000, 11), (65536, 3), (5000, 5000)])
def test_clip_thousands_of_tensors(count, each):
    # 5000 of up to 5000 elements are beyond 56 MiB
    g = torch.Generator().manual_seed(count)
    sizes = [each - i % 3 for i in range(count)]
    flat = torch.randn(sum(sizes), generator=g).cuda()
    out, norm, ws = torch.zeros_like(flat), torch.zeros(2, device="cuda"), workspace(count)
    B.bfly_grad_clip(list(flat.split(sizes)), 0.5, norm, ws, outs=list(out.split(sizes)))
    want = float(flat.double().square().sum().sqrt())
    assert abs(float(norm[0]) - want) <= TOL * want
    assert abs(float(norm[1]) - 0.5 / want) <= TOL * 0.5 / want
    assert torch.equal(out, flat * norm[1])
    B.bfly_grad_clip(list(flat.split(sizes)), 0.5, norm, ws)
    assert torch.equal(out, flat)
