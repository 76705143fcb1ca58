"""The norm, the adapters and the clipping together with the rotation and the
quantized product, as a program uses them: one layer's serving path, one
training step of its angles and norm weight, on streams of their own and in
captured graphs."""
import numpy as np
import pytest

import oracle
import learnable_butterfly_rotation_amd as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.detach().cpu().double().numpy()


def scratch(nbytes):
    return torch.full((max(1, nbytes),), 0x7F, dtype=U8, device="cuda")


class Layer:
    """A rotated, quantized projection of n = 1024 to 256 with its norm in
    front and 4 adapters of rank 16 beside it, and the buffers of `rows` rows."""

    def __init__(self, rows, seed=0):
        g = torch.Generator().manual_seed(seed)
        n, out, num, rank = 1024, 256, 4, 16
        self.rows, self.n, self.out = rows, n, out
        rand = lambda *s: torch.randn(s, generator=g)
        self.x, self.res = rand(rows, n).to(BF16).cuda(), rand(rows, n).to(BF16).cuda()
        self.weight = (1 + 0.1 * rand(n)).cuda()
        self.theta = ((torch.rand((10, n // 2), generator=g) * 2 - 1) * np.pi).cuda()
        self.ids = torch.randint(-1, num, (rows,), generator=g, dtype=torch.int32).cuda()
        self.a = (rand(num, rank, n) / 32).to(BF16).cuda()
        self.b = (0.1 * rand(num, out, rank)).to(BF16).cuda()
        self.s = torch.ones(num).cuda()
        w = (0.02 * rand(out, n)).to(BF16).cuda()
        self.codes = torch.empty((out, n // 2), dtype=U8, device="cuda")
        self.scales = torch.empty((out, n // 128), dtype=F16, device="cuda")
        self.table = scratch(B.bfly_coeff_bytes(n))
        B.bfly_prepare(self.theta, n, self.table)
        B.bfly_forward_quant(w, None, self.codes, self.scales, coeffs=self.table, bits=4)
        new = lambda dt, *s: torch.empty(s, dtype=dt, device="cuda")
        self.h, self.y, self.rot = (new(BF16, rows, n) for _ in range(3))
        self.codes8, self.scales8, self.rstd = new(torch.int8, rows, n), new(F16, rows, 1), new(F32, rows)
        self.base, self.z = new(F32, rows, out), new(BF16, rows, out)
        self.ws = scratch(B.bfly_lora_matmul_workspace_bytes(rows, out, n, rank))

    def serve(self, stream=None):
        B.bfly_rmsnorm(self.x, self.weight, EPS, y=self.y, codes=self.codes8, scales=self.scales8,
                       residual=self.res, h=self.h, rstd=self.rstd, stream=stream)
        B.bfly_forward(self.y, self.rot, coeffs=self.table, stream=stream)
        B.bfly_quant_matmul(self.rot, self.codes, self.scales, None, self.base, bits=4,
                            mode=B.BFLY_SYM_ABSMAX, stream=stream)
        B.bfly_lora_matmul(self.y, self.ids, self.a, self.b, self.s, self.z, self.ws,
                           base=self.base, stream=stream)
        return self.outputs() if stream is None else None

    def outputs(self):
        return [t.clone() for t in (self.h, self.codes8, self.scales8, self.rstd, self.z)]


@pytest.mark.parametrize("rows", [1, 7, 300])
def test_serving_path(rows):
    """Against the formulas in 64 bits from the layer's inputs to its output.
    The rotation keeps norms, so the bf16 roundings of y and of Q y (half a
    step, 2^-8 relative, each) move an output by at most their 2-norm times the
    weight row's: 2 * 2^-8 |y| |w|; the fp32 sums by (n + 64) u |y| |w|, the
    fp32 y and rotation by (3 + 4 * 10) u |y| |w|; an adapter's output likewise,
    with one bf16 rounding, the rows of A and 2^-16 of t; z half a step."""
    L = Layer(rows)
    L.serve()
    h = np64((L.x.float() + L.res.float()).to(BF16))
    assert np.array_equal(np64(L.h), h)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * np64(L.weight)
    q = oracle.forward(y.astype(np.float32), L.theta.cpu().numpy())
    w = dequantized(L)
    want = q @ w.T
    ynorm = np.sqrt((y * y).sum(1, keepdims=True))
    wnorm = np.sqrt((w * w).sum(1))[None, :]
    tol = (2 * 2.0 ** -8 * 1.01 + (L.n + 64 + 43 + 2) * U) * ynorm * wnorm
    ids = L.ids.cpu().numpy()
    for i in range(4):
        at = ids == i
        a, b = np64(L.a[i]), np64(L.b[i])
        t = y[at] @ a.T
        anorm = np.sqrt((a * a).sum(1))[None, :]
        et = (2.0 ** -8 * 1.01 + (L.n + 64 + 3) * U) * ynorm[at] * anorm + 2.0 ** -16 * np.abs(t)
        want[at] += t @ b.T
        tol[at] += 1.01 * et @ np.abs(b).T + 40 * U * (np.abs(t) @ np.abs(b).T)
    tol += 2.0 ** -8 * (np.abs(want) + tol)
    got = np64(L.z)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    # the 8-bit rows stand for y: half a step of the code, 2^-11 of the scale
    # (127 codes), and the fp32 roundings of y
    v = np64(L.codes8) * np64(L.scales8)
    step = np64(L.scales8)
    assert (np.abs(v - y) <= 0.5 * step + 127 * 2.0 ** -11 * step + 4 * U * np.abs(y)).all()


def dequantized(L):
    c = L.codes.cpu().numpy()
    q = np.stack([c & 15, c >> 4], axis=2).reshape(L.out, L.n).astype(np.int64)
    q = np.where(q > 7, q - 16, q)
    return q * np.repeat(np64(L.scales), 128, axis=1)


def test_training_step():
    """Norm, rotation, their gradients and the clipping, each from the values
    before it; the gradients also against differences of the loss
    sum(G * Q(theta) norm(h)) in 64 bits."""
    rows, n = 64, 256
    g = torch.Generator().manual_seed(5)
    h = torch.randn((rows, n), generator=g).cuda()
    w = (1 + 0.1 * torch.randn(n, generator=g)).cuda()
    theta = ((torch.rand((8, n // 2), generator=g) * 2 - 1) * np.pi).cuda()
    G = torch.randn((rows, n), generator=g).cuda()
    y, dy, dx = (torch.empty_like(h) for _ in range(3))
    rstd, dw = torch.empty(rows, device="cuda"), torch.empty(n, device="cuda")
    dtheta, norm = torch.empty_like(theta), torch.empty(2, device="cuda")
    B.bfly_rmsnorm(h, w, EPS, y=y, rstd=rstd)
    B.bfly_backward(y, G, None, dy, dtheta, scratch(B.bfly_backward_workspace_bytes(rows, n)),
                    theta=theta)
    B.bfly_rmsnorm_backward(h, w, rstd, dy, dx, dweight=dw,
                            workspace=scratch(B.bfly_rmsnorm_backward_workspace_bytes(rows, n)))
    raw = [np64(dtheta), np64(dw)]
    B.bfly_grad_clip([dtheta, dw], 1.0, norm, scratch(B.bfly_grad_clip_workspace_bytes(2)))
    size = np.sqrt(sum((t * t).sum() for t in raw))
    assert size > 1.0 and abs(float(norm[0]) - size) <= 1.01 * U * size
    for t, r in ((dtheta, raw[0]), (dw, raw[1])):
        assert (np.abs(np64(t) - r / size) <= 2.02 * U * np.abs(r / size)).all()

    def loss(h64, w64, th64):
        r = 1.0 / np.sqrt((h64 * h64).mean(1, keepdims=True) + float(np.float32(EPS)))
        v = h64 * r * w64
        for s in range(8):
            i = np.arange(n)
            lo = i[(i >> s) & 1 == 0]
            p = (lo >> (s + 1) << s) | (lo & ((1 << s) - 1))
            c, sn = np.cos(th64[s][p]), np.sin(th64[s][p])
            a, b = v[:, lo].copy(), v[:, lo + (1 << s)].copy()
            v[:, lo], v[:, lo + (1 << s)] = c * a - sn * b, sn * a + c * b
        return float((np64(G) * v).sum())

    # central differences: the truncation is t^2 of third derivatives (10^-10
    # relative), the cancellation 2^-52 / t (10^-11); the kernels' fp32 sums
    # over 64 rows and 8 stages stay below 10^-5 of the sum of |terms|
    rng = np.random.default_rng(6)
    t = 1e-5
    for k, grad in ((0, np64(dx)), (1, raw[1]), (2, raw[0])):
        at = [np64(h), np64(w), np64(theta)]
        for _ in range(4):
            v = rng.standard_normal(at[k].shape)
            up, down = list(at), list(at)
            up[k], down[k] = at[k] + t * v, at[k] - t * v
            num = (loss(*up) - loss(*down)) / (2 * t)
            assert abs(num - (grad * v).sum()) <= 1e-5 * np.abs(grad * v).sum() + 1e-4


def test_on_another_stream_with_work_before_it():
    L = Layer(300, seed=1)
    want = L.serve()
    x = L.x.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        L.x.zero_()
        big = torch.randn((4096, 4096), device="cuda")
        for _ in range(4):
            big = big @ big * 1e-2
        L.x.copy_(x)        # the calls have to wait for this one
        L.serve(stream=s)
        got = L.outputs()
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # the current stream is the default
    with torch.cuda.stream(s):
        L.x.zero_()
        L.x.copy_(x)
        got = L.serve()
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    layers = [Layer(300, seed=k) for k in (2, 3)]
    want = [L.serve() for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for L, s in zip(layers, streams):
            L.serve(stream=s)
    torch.cuda.synchronize()
    for L, w in zip(layers, want):
        for a, b in zip(w, L.outputs()):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    L = Layer(300, seed=4)
    n = L.n
    dy, dx = torch.randn((300, n), device="cuda").to(BF16), torch.empty((300, n), dtype=BF16, device="cuda")
    dw, norm = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    bws = scratch(B.bfly_rmsnorm_backward_workspace_bytes(300, n))
    grads = [torch.empty(k, device="cuda") for k in (5000, 3, 70001)] + [dw]
    cws = scratch(B.bfly_grad_clip_workspace_bytes(len(grads)))
    src = [torch.randn_like(t) for t in grads[:-1]]

    def step():
        L.serve(stream=torch.cuda.current_stream())
        B.bfly_rmsnorm_backward(L.h, L.weight, L.rstd, dy, dx, dweight=dw, workspace=bws)
        for t, v in zip(grads, src):
            t.copy_(v)
        B.bfly_grad_clip(grads, 0.5, norm, cws)

    def outputs():
        return L.outputs() + [t.clone() for t in (dx, norm, *grads)]

    xs = [torch.randn_like(L.x.float()).to(BF16) for _ in range(3)]
    ids = [torch.randint(-1, 4, (300,), dtype=torch.int32, device="cuda") for _ in range(3)]
    want = []
    for x, i in zip(xs, ids):
        L.x.copy_(x)
        L.ids.copy_(i)
        step()
        torch.cuda.synchronize()
        want.append(outputs())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in (0, 1, 2, 1, 0):
        L.x.copy_(xs[k])
        L.ids.copy_(ids[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want[k], outputs()):
            assert torch.equal(a, b)
        # eager work between the replays, in the same buffers
        L.x.copy_(xs[(k + 1) % 3])
        L.ids.copy_(ids[(k + 1) % 3])
        step()
        torch.cuda.synchronize()
        for a, b in zip(want[(k + 1) % 3], outputs()):
            assert torch.equal(a, b)


def test_what_the_binding_refuses():
    x = torch.zeros((4, 64), device="cuda")
    w = torch.zeros(64, device="cuda")
    v = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        B.bfly_rmsnorm(x.half(), w, EPS, y=x)
    with pytest.raises(TypeError):
        B.bfly_rmsnorm(x, w, EPS, y=x, residual=x.to(BF16))
    with pytest.raises(ValueError):
        B.bfly_rmsnorm(x, w[:32], EPS, y=x)
    with pytest.raises(ValueError):
        B.bfly_rmsnorm(x.T.contiguous().T, w, EPS, y=x)
    with pytest.raises(ValueError):
        B.bfly_rmsnorm(x, w, EPS, y=x[:3])
    with pytest.raises(ValueError):
        B.bfly_rmsnorm(x, w.cpu(), EPS, y=x)
    with pytest.raises(ValueError):  # scales of another group
        B.bfly_rmsnorm(x, w, EPS, codes=torch.zeros((4, 64), dtype=U8, device="cuda"),
                       scales=torch.zeros((4, 8), dtype=F16, device="cuda"), group=16)
    for kw in (dict(group=24), dict(format=2), dict(group=0), dict(group=-8)):
        with pytest.raises((B.BflyError, ValueError)):
            B.bfly_rmsnorm(x, w, EPS, codes=torch.zeros((4, 64), dtype=U8, device="cuda"),
                           scales=torch.zeros((4, 1), dtype=F16, device="cuda"), **kw)
    with pytest.raises(B.BflyError) as e:
        B.bfly_rmsnorm(x, w, 0.0, y=x)
    assert e.value.status == 2
    with pytest.raises(B.BflyError):  # no output
        B.bfly_rmsnorm(x, w, EPS)
    with pytest.raises(B.BflyError) as e:
        B.bfly_rmsnorm_backward(x, w, v, x, torch.empty_like(x), dweight=torch.empty_like(w))
    assert e.value.status == 1
    with pytest.raises(B.BflyError) as e:
        B.bfly_rmsnorm_backward(x, w, v, x, torch.empty_like(x), dweight=torch.empty_like(w),
                                workspace=torch.empty(16, dtype=U8, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(ValueError):
        B.bfly_rmsnorm_backward(x, w, v[:3], x, torch.empty_like(x))
    b = torch.zeros((4, 64), dtype=BF16, device="cuda")
    a, lb = torch.zeros((2, 8, 64), dtype=BF16, device="cuda"), torch.zeros((2, 16, 8), dtype=BF16, device="cuda")
    ids, s, y = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda"), \
        torch.zeros((4, 16), device="cuda")
    ws = scratch(B.bfly_lora_matmul_workspace_bytes(4, 16, 64, 8))
    B.bfly_lora_matmul(b, ids, a, lb, s, y, ws)
    with pytest.raises(TypeError):
        B.bfly_lora_matmul(x, ids, a, lb, s, y, ws)
    with pytest.raises(TypeError):
        B.bfly_lora_matmul(b, ids.long(), a, lb, s, y, ws)
    with pytest.raises(ValueError):
        B.bfly_lora_matmul(b, ids, a[:1], lb, s, y, ws)
    with pytest.raises(ValueError):
        B.bfly_lora_matmul(b, ids, a.transpose(1, 2).contiguous().transpose(1, 2), lb, s, y, ws)
    with pytest.raises(ValueError):
        B.bfly_lora_matmul(b, ids, a, lb, s, y, ws.cpu())
    with pytest.raises(B.BflyError) as e:
        B.bfly_lora_matmul(b, ids, a, lb, s, y, ws[:-1])
    assert e.value.status == 6
    n2, cws = torch.zeros(2, device="cuda"), scratch(B.bfly_grad_clip_workspace_bytes(2))
    with pytest.raises(ValueError):
        B.bfly_grad_clip([x, x.cpu()], 1.0, n2, cws)
    with pytest.raises(ValueError):
        B.bfly_grad_clip([x, x.T], 1.0, n2, cws)
    with pytest.raises(TypeError):
        B.bfly_grad_clip([x, x.half()], 1.0, n2, cws)
    with pytest.raises(ValueError):
        B.bfly_grad_clip([x, x], 1.0, n2, cws, outs=[x])
    with pytest.raises(ValueError):
        B.bfly_grad_clip([x, w], 1.0, n2, cws, outs=[x, b])
    with pytest.raises(B.BflyError) as e:
        B.bfly_grad_clip([x, w, v], 1.0, n2, cws)
    assert e.value.status == 6
    with pytest.raises(B.BflyError):
        B.bfly_grad_clip([x], float("nan"), n2, cws)


def test_norm_past_32_bit_offsets():
    # 4.4 GB of rows: a row's results are those of a call with few rows
    rows, n = 540000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((rows, n), dtype=BF16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn(n, device="cuda", generator=g)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    codes = torch.empty((rows, n), dtype=torch.int8, device="cuda")
    scales = torch.empty((rows, n // 128), dtype=F16, device="cuda")
    B.bfly_rmsnorm(x, w, EPS, y=y, codes=codes, scales=scales, rstd=rstd, group=128)
    few = [slice(0, 200), slice(524200, 524400), slice(rows - 200, rows)]
    small = []
    for at in few:
        part = x[at].clone()
        out = [torch.empty_like(t[at]) for t in (y, codes, scales, rstd)]
        B.bfly_rmsnorm(part, w, EPS, y=out[0], codes=out[1], scales=out[2], rstd=out[3], group=128)
        small.append((part, out[3]))
        for a, b in zip(out, (y, codes, scales, rstd)):
            assert torch.equal(a, b[at])
    # the gradient, in place of dy, which is zero but in those rows
    dy = y.zero_()
    ws = scratch(B.bfly_rmsnorm_backward_workspace_bytes(rows, n))
    ws2 = scratch(B.bfly_rmsnorm_backward_workspace_bytes(200, n))
    dw, want, total, size = (torch.zeros(n, device="cuda") for _ in range(4))
    for at, (part, r) in zip(few, small):
        d = torch.empty((200, n), dtype=BF16, device="cuda").normal_(generator=g)
        dy[at] = d
        total += (d.double() * part.double() * r.double()[:, None]).sum(0).float()
        size += (d.double() * part.double() * r.double()[:, None]).abs().sum(0).float()
        small[few.index(at)] = (part, r, d)
    B.bfly_rmsnorm_backward(x, w, rstd, dy, dy, dweight=dw, workspace=ws)
    for at, (part, r, d) in zip(few, small):
        B.bfly_rmsnorm_backward(part, w, r, d, d, dweight=want, workspace=ws2)
        assert torch.equal(dy[at], d)
    # 600 products (two roundings each) among zeros, and both references' roundings
    assert ((dw - total).abs() <= 1.01 * (600 + 8) * U * size).all()
    assert not dy[200:524200].any()


def test_adapters_past_32_bit_offsets():
    # 4.4 GB of x and of y: a block of rows, again and again
    blocks, k, out, num, rank = 1056, 8192, 8192, 5, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)
    x, base = rand(256, k).to(BF16), rand(256, out).to(BF16)
    ids = torch.randint(-1, num, (256,), device="cuda", generator=g, dtype=torch.int32)
    a, b, s = (rand(num, rank, k) / k ** 0.5).to(BF16), rand(num, out, rank).to(BF16), \
        0.5 + torch.rand(num, device="cuda", generator=g)
    rows = 256 * blocks
    y = base.repeat(blocks, 1)
    ws = scratch(B.bfly_lora_matmul_workspace_bytes(rows, out, k, rank))
    B.bfly_lora_matmul(x.repeat(blocks, 1), ids.repeat(blocks), a, b, s, y, ws, base=y)
    first = y[:256]
    assert (y.view(blocks, 256, out) == first).all()
    for i in range(num):
        at = ids == i
        t = x[at].double() @ a[i].double().T * s[i].double()
        tabs = x[at].double().abs() @ a[i].double().abs().T * s[i].double()
        add, b64 = t @ b[i].double().T, b[i].double().abs().T
        # t's sum over k and its 16 bits, the second sum, the base's addition, y
        err = (1.01 * (k + 64) * U * tabs + (2 * U + 2.0 ** -16) * t.abs()) @ b64 \
            + 1.01 * 2 * rank * U * (t.abs() @ b64)
        want = base[at].double() + add
        tol = err + U * (want.abs() + err) + 2.0 ** -8 * (want.abs() + 2 * err)
        assert ((first[at].double() - want).abs() <= tol).all()
    assert torch.equal(first[ids < 0], base[ids < 0])


def test_clipping_past_32_bit_offsets():
    n = 2 ** 32 + 37
    g = torch.full((n,), 2.0 ** -8, dtype=BF16, device="cuda")
    g[-1] = 96.0
    norm = torch.empty(2, device="cuda")
    ws = scratch(B.bfly_grad_clip_workspace_bytes(1))
    B.bfly_grad_clip([g], 1.0, norm, ws)
    exact = ((n - 1) * 2.0 ** -16 + 96.0 ** 2) ** 0.5
    # an fp64 sum, rounded once; the factor likewise
    assert abs(float(norm[0]) - exact) <= 1.01 * U * exact
    assert abs(float(norm[1]) - 1 / exact) <= 1.01 * U / exact
    assert (g[:-1] == (norm[1] * 2.0 ** -8).to(BF16)).all()
    assert g[-1] == (norm[1] * 96.0).to(BF16)
