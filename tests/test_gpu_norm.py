"""bfly_rmsnorm and bfly_rmsnorm_backward on the GPU against the formulas in
64 bits.

Tolerances (u = 2^-24, half a step of fp32):
* h is one fp32 addition and one rounding: equal bits.
* rstd is the fp64 value rounded once: u relative.
* y in fp32 has three roundings (rstd, two products): 3 u |y|; a bf16 y half
  a step (eps / 2) more.
* scales and codes follow from the fp32 y, whose bits numpy reproduces from
  the kernel's own rstd: equal.
* dx: xhat 1, g 1, the mean's terms 3 and its sum at most D = 8 V + 6 + T / 64
  <= 38 roundings, 1 / n and the product with it 2, the last two fused
  multiply-adds 2.
* dweight: terms 2, a thread's sum over its rows, four waves, the slots.
"""
import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rows_of(seed, rows, n, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, n), generator=g) * scale
    if n >= 64:
        x[:, 5] *= 50.0
    return x.to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def quantized(y32, group, e4m3):
    """The quantizer of the fp32 rows, in numpy's (and torch's CPU) arithmetic."""
    rows, n = y32.shape
    top = np.float32(448.0 if e4m3 else 127.0)
    v = y32.reshape(rows, n // group, group)
    # the quotient by top is a product with its fp32 reciprocal
    s = np.minimum(np.abs(v).max(2) * (np.float32(1) / top), np.float32(65504)).astype(np.float16)
    d = s.astype(np.float32)[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        q = np.where(d > 0, v / d, np.float32(0))
    q = np.clip(q, -top, top).reshape(rows, n)
    if e4m3:
        return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), s
    return np.rint(q).astype(np.int8).view(np.uint8), s


def check_norm(x, res, w, y_dt, fmt, group, h_out=True):
    rows, n = x.shape
    xd = x.cuda()
    rd = None if res is None else res.cuda()
    wd = None if w is None else w.cuda()
    # two rows more than the call is given, which it must leave alone
    h = torch.full((rows + 2, n), 7.0, dtype=x.dtype, device="cuda") if rd is not None and h_out \
        else None
    y = torch.full((rows + 2, n), 7.0, dtype=y_dt, device="cuda") if y_dt else None
    rstd = torch.full((rows + 2,), 7.0, device="cuda")
    codes = scales = None
    if fmt is not None:
        codes = torch.full((rows + 2, n), 77, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows + 2, n // group), 7.0, dtype=torch.float16, device="cuda")
    cut = lambda t: None if t is None else t[:rows]
    B.bfly_rmsnorm(xd, wd, EPS, y=cut(y), codes=cut(codes), scales=cut(scales), residual=rd,
                   h=cut(h), rstd=rstd[:rows], format=fmt or 0, group=group)
    torch.cuda.synchronize()
    for t, v in ((h, 7.0), (y, 7.0), (rstd, 7.0), (codes, 77), (scales, 7.0)):
        if t is not None:
            assert (t[rows:].float() == v).all()
    hx = x if res is None else (x.float() + res.float()).to(x.dtype)
    if h is not None:
        assert torch.equal(h[:rows].cpu(), hx)
    h64 = np64(hx)
    r64 = 1.0 / np.sqrt((h64 * h64).sum(1) / n + float(np.float32(EPS)))
    r32 = rstd[:rows].cpu().numpy()
    assert (np.abs(r32.astype(np.float64) - r64) <= U * (1 + 1e-6) * r64).all()
    w32 = np.ones(n, np.float32) if w is None else w.float().numpy()
    y64 = h64 * r64[:, None] * w32.astype(np.float64)
    y32 = (hx.float().numpy() * r32[:, None]) * w32
    if y is not None:
        tol = 3.01 * U * np.abs(y64)
        if y_dt == BF16:
            tol += half(BF16) * (1 + 4 * U) * np.abs(y64)
        assert (np.abs(np64(y[:rows]) - y64) <= tol).all()
    if fmt is not None:
        c, s = quantized(y32, group, fmt == B.BFLY_Q8_E4M3)
        assert np.array_equal(scales[:rows].cpu().numpy().view(np.uint16), s.view(np.uint16))
        assert np.array_equal(codes[:rows].cpu().numpy(), c)


WIDTHS = [1, 2, 7, 8, 63, 64, 72, 127, 128, 129, 136, 200, 256, 511, 512, 520, 1000, 1023, 1024, 1025, 1032, 2047, 2048,
          2056, 4095, 4096, 4104, 5120, 8191, 8192, 8200, 11008, 16383, 16384]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("x_dt", [F32, BF16])
def test_norm_widths(n, x_dt):
    rows = 5 if n > 512 else 9
    x, res = rows_of(n, rows, n, x_dt), rows_of(n + 1, rows, n, x_dt)
    g = torch.Generator().manual_seed(n + 2)
    w = 1 + 0.1 * torch.randn(n, generator=g)
    check_norm(x, res, w, F32, B.BFLY_Q8_INT8, n)
    check_norm(x, None, w.to(BF16), BF16, B.BFLY_Q8_E4M3, n)
    check_norm(x, res, None, BF16, None, None, h_out=False)


@pytest.mark.parametrize("rows", [256, 257])
@pytest.mark.parametrize("n", [2049, 2056, 4096, 4100, 5120, 6152, 8191, 8192, 8200])
@pytest.mark.parametrize("x_dt", [F32, BF16])
def test_norm_widths_of_few_and_more_rows(rows, n, x_dt):
    x, res = rows_of(n, rows, n, x_dt), rows_of(n + 1, rows, n, x_dt)
    w = 1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(n + 2))
    group = 8 if n % 8 == 0 else n
    check_norm(x, res, w, F32, B.BFLY_Q8_INT8, group)
    check_norm(x, None, w.to(BF16), BF16, B.BFLY_Q8_E4M3, n)
    check_norm(x, res, None, BF16, None, None, h_out=False)


@pytest.mark.parametrize("group,n", [(g, n) for g in (8, 16, 32, 64, 128, 256, 512) for n in
                                     (64, 128, 512, 1024, 2048, 1536, 4096, 5120, 11776, 16384)
                                     if g <= n])
def test_norm_groups(group, n):
    x, res = rows_of(n + group, 6, n, BF16), rows_of(n + group + 1, 6, n, BF16)
    w = 1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(n))
    check_norm(x, res, w, None, B.BFLY_Q8_INT8, group)
    check_norm(x.float(), None, w, BF16, B.BFLY_Q8_E4M3, group)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 2047, 2048, 2049, 8191, 8195])
@pytest.mark.parametrize("n", [64, 100, 128, 256, 1031, 4096])
def test_norm_rows(rows, n):
    x, res = rows_of(rows, rows, n, BF16), rows_of(rows + 1, rows, n, BF16)
    check_norm(x, res, None, BF16, B.BFLY_Q8_INT8, n)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e-3, 1e4, 1e18, 1e30])
@pytest.mark.parametrize("fmt", [B.BFLY_Q8_INT8, B.BFLY_Q8_E4M3])
def test_norm_magnitudes(scale, fmt):
    # squares far beyond fp32, and rows that eps dominates (tiny scales, some
    # of them subnormal or zero in fp16)
    x = rows_of(3, 4, 1024, F32, scale)
    w = torch.logspace(-8, 3, 1024)
    check_norm(x, None, w, F32, fmt, 128)


def test_norm_zero_rows_and_codes_of_zero():
    x = torch.zeros((3, 256))
    x[1, 7] = 2.0
    check_norm(x, None, None, F32, B.BFLY_Q8_INT8, 8)


def test_norm_rows_that_are_not_finite():
    x = rows_of(11, 6, 4096, F32)
    x[1, 17] = float("inf")
    x[3, 4095] = float("nan")
    clean = x.clone()
    clean[1, 17] = clean[3, 4095] = 0.0
    y, r = torch.empty_like(x).cuda(), torch.empty(6).cuda()
    B.bfly_rmsnorm(x.cuda(), None, EPS, y=y, rstd=r)
    y0, r0 = torch.empty_like(y), torch.empty_like(r)
    B.bfly_rmsnorm(clean.cuda(), None, EPS, y=y0, rstd=r0)
    for i in (0, 2, 4, 5):
        assert torch.equal(y[i], y0[i]) and r[i] == r0[i]
    assert r[1] == 0 and (y[1, :17] == 0).all() and torch.isnan(y[1, 17])
    assert torch.isnan(r[3]) and torch.isnan(y[3]).all()


@pytest.mark.parametrize("into", ["x", "residual"])
def test_norm_in_place(into):
    x, res = rows_of(5, 33, 4096, BF16).cuda(), rows_of(6, 33, 4096, BF16).cuda()
    h, y = torch.empty_like(x), torch.empty_like(x)
    B.bfly_rmsnorm(x, None, EPS, y=y, residual=res, h=h)
    a, b = x.clone(), res.clone()
    y2 = torch.empty_like(x)
    B.bfly_rmsnorm(a, None, EPS, y=y2, residual=b, h=a if into == "x" else b)
    assert torch.equal(a if into == "x" else b, h) and torch.equal(y, y2)
    a, b = x.clone(), res.clone()
    B.bfly_rmsnorm(a, None, EPS, y=a if into == "x" else b, residual=b)
    assert torch.equal(a if into == "x" else b, y)


def test_norm_no_rows():
    x = torch.empty((0, 4096), device="cuda")
    B.bfly_rmsnorm(x, None, EPS, y=torch.empty_like(x))
    dw = torch.full((4096,), 3.0, device="cuda")
    B.bfly_rmsnorm_backward(x, None, torch.empty(0, device="cuda"), x, torch.empty_like(x),
                            dweight=dw, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert (dw == 0).all()


def check_backward(h, w, dy, dh, in_place=False):
    rows, n = h.shape
    h64, dy64 = np64(h), np64(dy)
    r32 = (1.0 / np.sqrt((h64 * h64).mean(1) + EPS)).astype(np.float32)
    r64 = r32.astype(np.float64)[:, None]
    w64 = np.ones(n) if w is None else np64(w)
    dev = lambda t: None if t is None else t.cuda()
    dyd = dev(dy)
    dx = dyd if in_place else torch.full((rows + 1, n), 7.0, dtype=dy.dtype, device="cuda")
    dw = torch.empty(n, device="cuda")
    ws = torch.full((B.bfly_rmsnorm_backward_workspace_bytes(rows, n),), 0x7F, dtype=torch.uint8,
                    device="cuda")
    args = (dev(h), dev(w), torch.from_numpy(r32).cuda(), dyd, dx[:rows])
    B.bfly_rmsnorm_backward(*args, dweight=dw, dh=dev(dh), workspace=ws)
    torch.cuda.synchronize()
    if not in_place:
        assert (dx[rows:] == 7.0).all()
        # without dweight and its workspace: the same dx; with them: the same bits again
        dx2, dw2 = torch.empty_like(dx[:rows]), torch.empty_like(dw)
        B.bfly_rmsnorm_backward(*args[:4], dx2, dh=dev(dh))
        assert torch.equal(dx2, dx[:rows])
        B.bfly_rmsnorm_backward(*args[:4], dx2, dweight=dw2, dh=dev(dh), workspace=ws)
        assert torch.equal(dx2, dx[:rows]) and torch.equal(dw2, dw)
    g, xhat = dy64 * w64, h64 * r64
    c, cabs = (g * xhat).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    d64 = 0.0 if dh is None else np64(dh)
    want = (g - xhat * c) * r64 + d64
    tol = r64 * (4 * U * (np.abs(g) + np.abs(xhat * c)) + np.abs(xhat) * (38 + 5) * U * cabs)
    tol = 1.01 * tol + (U if dy.dtype == F32 else half(BF16)) * (np.abs(want) + tol) + U * np.abs(want)
    assert (np.abs(np64(dx[:rows]) - want) <= tol).all()
    together = 16 if n <= 128 else 4 if n <= 1024 else 1  # rows of a workgroup
    slots = -(-rows // together)
    most = 1024 if n <= 1024 else 256 if n >= 4096 else (1 << 20) // n
    groups, slots = slots, min(slots, max(most, min(2048, slots // 128)))
    depth = -(-groups // slots) + together - 1 + -(-slots // 16) + 15 + 2
    term = dy64 * xhat
    tol = 1.01 * depth * U * np.abs(term).sum(0)
    assert (np.abs(np64(dw) - term.sum(0)) <= tol).all()


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("h_dt,g_dt", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
def test_backward_widths(n, h_dt, g_dt):
    rows = 9
    h, dy, dh = rows_of(n, rows, n, h_dt), rows_of(n + 1, rows, n, g_dt), rows_of(n + 2, rows, n, g_dt)
    w = 1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(n))
    check_backward(h, w, dy, dh)
    check_backward(h, w.to(BF16), dy, None)


@pytest.mark.parametrize("rows", [1, 3, 4, 1023, 1025, 4097, 5000])
@pytest.mark.parametrize("n", [64, 101, 256, 1023, 2048])
def test_backward_rows(rows, n):
    check_backward(rows_of(rows, rows, n, BF16), None, rows_of(rows + 1, rows, n, BF16),
                   rows_of(rows + 2, rows, n, BF16))


@pytest.mark.parametrize("rows,n", [(70000, 1500), (40000, 4096), (500000, 16)])
def test_backward_many_rows(rows, n):
    # beyond 128 rows to a thread's sum there are more partial sums
    g = torch.Generator(device="cuda").manual_seed(rows)
    h, dy = (torch.randn((rows, n), generator=g, device="cuda") for _ in range(2))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = torch.empty_like(h), torch.empty(n, device="cuda")
    ws = torch.empty(B.bfly_rmsnorm_backward_workspace_bytes(rows, n), dtype=torch.uint8,
                     device="cuda")
    B.bfly_rmsnorm_backward(h, None, rstd, dy, dx, dweight=dw, workspace=ws)
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(0, rows, 10000):
        t = dy[i:i + 10000].double() * h[i:i + 10000].double() * rstd[i:i + 10000, None].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    # two roundings of a term; 200 of a thread, its workgroup's and the slots'
    # sums (at most 16 + 128 + 16) at the very most
    assert ((dw.double() - want).abs() <= 1.01 * (2 + 200 + 160) * U * size).all()
    # and as random roundings add up, far closer: 2^-24 sqrt(362) of the 2-norm
    # of the terms' partial sums, which the sum's own size (~ sqrt(rows)) bounds
    err = float((dw.double() - want).norm() / want.norm())
    assert err <= 362 ** 0.5 * U


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 12, 13, 48, 49])
@pytest.mark.parametrize("n", [64, 100, 520, 4096, 11008])
def test_backward_weight_gradient_at_any_address(rows, n):
    g = torch.Generator().manual_seed(rows * n)
    h, dy = (torch.randn((rows, n), generator=g).cuda() for _ in range(2))
    r = torch.rand(rows, generator=g).cuda() + 0.5
    ws = torch.full((B.bfly_rmsnorm_backward_workspace_bytes(rows, n),), 0x7F, dtype=torch.uint8,
                    device="cuda")
    buf, got = torch.full((n + 9,), 7.0, device="cuda"), []
    for at in (4, 1, 2, 3):
        B.bfly_rmsnorm_backward(h, None, r, dy, torch.empty_like(h), dweight=buf[at:at + n],
                                workspace=ws)
        got.append(buf[at:at + n].clone())
        assert (buf[:at] == 7.0).all() and (buf[at + n:] == 7.0).all()
        buf.fill_(7.0)
    for v in got[1:]:
        assert torch.equal(v, got[0])
    exact = (dy.double() * h.double() * r.double()[:, None])
    # at most rows + 40 additions, and the two products' roundings
    tol = 1.01 * (rows + 42) * U * exact.abs().sum(0)
    assert ((got[0].double() - exact.sum(0)).abs() <= tol).all()


def test_backward_in_place():
    check_backward(rows_of(1, 40, 4096, F32), None, rows_of(2, 40, 4096, F32), None, in_place=True)


def test_backward_against_differences():
    # d/dt of sum(dy * y(h + t v)) and of the weight's, in fp64 around the point
    n, rows = 96, 3
    h, dy = rows_of(1, rows, n, F32), rows_of(2, rows, n, F32)
    w = 1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(3))
    rstd, y = torch.empty(rows, device="cuda"), torch.empty((rows, n), device="cuda")
    B.bfly_rmsnorm(h.cuda(), w.cuda(), EPS, y=y, rstd=rstd)
    dx, dw = torch.empty((rows, n), device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(B.bfly_rmsnorm_backward_workspace_bytes(rows, n), dtype=torch.uint8,
                     device="cuda")
    B.bfly_rmsnorm_backward(h.cuda(), w.cuda(), rstd, dy.cuda(), dx, dweight=dw, workspace=ws)

    def loss(h64, w64):
        r = 1.0 / np.sqrt((h64 * h64).mean(1, keepdims=True) + float(np.float32(EPS)))
        return float((np64(dy) * h64 * r * w64).sum())

    rng = np.random.default_rng(4)
    for _ in range(8):
        v, u = rng.standard_normal((rows, n)), rng.standard_normal(n)
        t = 1e-5
        num = (loss(np64(h) + t * v, np64(w)) - loss(np64(h) - t * v, np64(w))) / (2 * t)
        # the differences are off by t^2 times a third derivative, about 1e-8
        # of the gradient's size, and by the cancellation in fp64, about 1e-9
        assert abs(num - float((np64(dx) * v).sum())) <= 1e-5 * np.abs(np64(dx) * v).sum() + 1e-6
        num = (loss(np64(h), np64(w) + t * u) - loss(np64(h), np64(w) - t * u)) / (2 * t)
        assert abs(num - float((np64(dw) * u).sum())) <= 1e-5 * np.abs(np64(dw) * u).sum() + 1e-6


@pytest.mark.parametrize("n,group", [(100, 100), (128, 16), (520, 520), (1023, 1023), (1024, 64),
                                     (4096, 4096), (4096, 128), (5120, 512), (11008, 11008),
                                     (16384, 8), (16383, 16383)])
@pytest.mark.parametrize("fmt", [B.BFLY_Q8_INT8, B.BFLY_Q8_E4M3])
@pytest.mark.parametrize("x_dt", [F32, BF16])
def test_norm_codes_of_a_y_beyond_fp32(n, group, fmt, x_dt):
    # finite rows and weights whose product is an infinity: its code is +-top
    # and its group's scale 65504
    x = rows_of(n + group, 5, n, x_dt)
    w = 1 + 0.1 * torch.randn(n, generator=torch.Generator().manual_seed(n))
    w[n // 3::7] = 3e38
    w[n // 2::11] = -3.4e38
    with np.errstate(over="ignore"):
        check_norm(x, None, w, None, fmt, group)
        r = (x.double().square().mean(1) + EPS) ** -0.5
        # short rows of a large element stay just below: 2.5e38
        assert n < 1000 or (x.double() * r[:, None] * w.double()).abs().max() > 3.5e38


@pytest.mark.parametrize("rows,n", [(131073, 64), (131090, 100), (32769, 520), (32771, 1023),
                                    (8200, 5120), (8200, 6150), (8200, 11008), (8193, 16384)])
def test_norm_rows_beyond_the_grid(rows, n):
    # a workgroup's second turn
    x, res = rows_of(rows, rows, n, BF16), rows_of(rows + 1, rows, n, BF16)
    check_norm(x, res, None, BF16, B.BFLY_Q8_INT8, n)


@pytest.mark.parametrize("rows", [600, 1025])
@pytest.mark.parametrize("n", [5120, 8191, 11008, 16384])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_rows_beyond_the_slots(rows, n, with_dh):
    check_backward(rows_of(1, rows, n, BF16), None, rows_of(2, rows, n, F32),
                   rows_of(3, rows, n, F32) if with_dh else None)


@pytest.mark.parametrize("into", ["dy", "dh", "h"])
@pytest.mark.parametrize("rows,n", [(9, 100), (9, 1031), (40, 4096), (600, 5120), (600, 16384)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_into_its_inputs(into, rows, n, dtype):
    h, dy, dh = (rows_of(k, rows, n, dtype).cuda() for k in (1, 2, 3))
    rstd = torch.rand(rows, generator=torch.Generator().manual_seed(4)).cuda() + 0.5
    ws = torch.empty(B.bfly_rmsnorm_backward_workspace_bytes(rows, n), dtype=torch.uint8,
                     device="cuda")
    dx, dw, dw2 = torch.empty_like(h), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    B.bfly_rmsnorm_backward(h, None, rstd, dy, dx, dweight=dw, dh=dh, workspace=ws)
    to = {"dy": dy, "dh": dh, "h": h}[into]
    B.bfly_rmsnorm_backward(h, None, rstd, dy, to, dweight=dw2, dh=dh, workspace=ws)
    assert torch.equal(to, dx) and torch.equal(dw, dw2)
