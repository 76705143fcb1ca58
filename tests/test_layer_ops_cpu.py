"""What bfly_rmsnorm, bfly_rmsnorm_backward, bfly_lora_matmul and
bfly_grad_clip refuse, at the C ABI and in the binding: all before any HIP
call, so these run on a machine without a GPU."""
import ctypes
import os

import pytest

import learnable_butterfly_rotation_amd as B

torch = pytest.importorskip("torch")

OK, NULL, SIZE, DTYPE, ALIGN, QUANT, WORKSPACE, UNSUPPORTED, HIP = range(9)
# fake, well-aligned device addresses: validation never dereferences them
P = {v: 0x10000 * (i + 1) for i, v in enumerate("abcdefghij")}


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.library_path):
        pytest.skip("libbfly.so not built")
    return B.lib()


def norm(L, x=P["a"], xd=1, res=P["b"], h=P["c"], w=P["d"], wd=0, y=P["e"], yd=0, c=P["f"],
         s=P["g"], r=P["h"], rows=4, n=4096, eps=1e-5, fmt=0, group=128):
    # with rows = 4 a call that passed would reach the GPU: only refusals use it
    return L.bfly_rmsnorm(x, xd, res, h, w, wd, y, yd, c, s, r, rows, n, eps, fmt, group, None)


def test_rmsnorm_refusals(L):
    assert norm(L, rows=0) == OK
    assert norm(L, rows=0, x=None, res=None, h=None, y=None, c=None, s=None, r=None) == OK
    assert norm(L, x=None) == NULL
    assert norm(L, res=None) == NULL                     # h without a residual
    assert norm(L, c=None) == NULL and norm(L, s=None) == NULL
    assert norm(L, h=None, y=None, c=None, s=None, r=None) == NULL
    assert norm(L, xd=2) == DTYPE and norm(L, wd=-1) == DTYPE and norm(L, yd=7) == DTYPE
    assert norm(L, rows=0, w=None, wd=9, y=None, yd=9) == OK
    assert norm(L, rows=-1) == SIZE and norm(L, n=0) == SIZE and norm(L, n=-8) == SIZE
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert norm(L, eps=eps) == SIZE
    assert norm(L, n=16385, group=16385) == UNSUPPORTED
    assert norm(L, rows=(1 << 46) // 4096 + 1) == UNSUPPORTED
    assert norm(L, fmt=2) == QUANT and norm(L, fmt=-1) == QUANT
    for group in (0, -8, 4, 7, 96, 1024, 4095):
        assert norm(L, group=group) == QUANT
    assert norm(L, n=4104, group=16) == QUANT            # does not divide
    assert norm(L, rows=0, n=1023, group=1023) == OK
    assert norm(L, rows=0, c=None, s=None, group=-5, fmt=77) == OK
    for name in ("x", "res", "h", "w", "y", "c"):
        assert norm(L, **{name: 0x10008}) == ALIGN, name
    assert norm(L, s=0x10001) == ALIGN and norm(L, r=0x10002) == ALIGN


def bwd(L, h=P["a"], hd=1, w=P["b"], wd=0, r=P["c"], dy=P["d"], dh=P["e"], dx=P["f"], gd=1,
        dw=P["g"], rows=4, n=4096, ws=P["h"], wsb=None):
    if wsb is None:
        wsb = L.bfly_rmsnorm_backward_workspace_bytes(rows, n)
    return L.bfly_rmsnorm_backward(h, hd, w, wd, r, dy, dh, dx, gd, dw, rows, n, ws, wsb, None)


def test_rmsnorm_backward_refusals(L):
    assert bwd(L, rows=0, dw=None) == OK
    for name in ("h", "r", "dy", "dx", "ws"):
        assert bwd(L, **{name: None}) == NULL, name
    assert bwd(L, hd=2) == DTYPE and bwd(L, gd=-1) == DTYPE and bwd(L, wd=3) == DTYPE
    assert bwd(L, rows=-1) == SIZE and bwd(L, n=0) == SIZE
    assert bwd(L, n=16385) == UNSUPPORTED
    assert bwd(L, wsb=L.bfly_rmsnorm_backward_workspace_bytes(4, 4096) - 1) == WORKSPACE
    for name in ("h", "w", "dy", "dh", "dx", "ws"):
        assert bwd(L, **{name: 0x10008}) == ALIGN, name
    assert bwd(L, r=0x10002) == ALIGN and bwd(L, dw=0x10002) == ALIGN
    assert B.bfly_rmsnorm_backward_workspace_bytes(-1, 64) == 0
    assert B.bfly_rmsnorm_backward_workspace_bytes(4, 16385) == 0
    assert B.bfly_rmsnorm_backward_workspace_bytes(0, 64) == 0


def lora(L, x=P["a"], xd=1, ids=P["b"], a=P["c"], b=P["d"], s=P["e"], base=P["f"], bd=1, y=P["g"],
         yd=1, rows=4, n_out=256, k=512, num=3, rank=16, ws=P["h"], wsb=None):
    if wsb is None:
        wsb = 1 << 40
    return L.bfly_lora_matmul(x, xd, ids, a, b, s, base, bd, y, yd, rows, n_out, k, num, rank, ws,
                              wsb, None)


def test_lora_refusals(L):
    assert lora(L, rows=0) == OK
    assert lora(L, rows=0, x=None, ids=None, a=None, b=None, s=None, base=None, y=None, ws=None,
                wsb=0) == OK
    for name in ("x", "ids", "a", "b", "s", "y", "ws"):
        assert lora(L, **{name: None}) == NULL, name
    assert lora(L, xd=0) == DTYPE and lora(L, bd=2) == DTYPE and lora(L, yd=-1) == DTYPE
    assert lora(L, y=P["f"], yd=0) == DTYPE              # in place with another type
    for name in ("n_out", "k", "num", "rank"):
        assert lora(L, **{name: 0}) == SIZE, name
    assert lora(L, rows=-1) == SIZE
    for name, v in (("n_out", 12), ("k", 4), ("rank", 12), ("n_out", (1 << 20) + 8), ("k", 65544),
                    ("rank", 264), ("rows", (1 << 23) + 1), ("num", (1 << 22) + 1)):
        assert lora(L, **{name: v}) == UNSUPPORTED, (name, v)
    need = B.bfly_lora_matmul_workspace_bytes(4, 256, 512, 16)
    assert need > 0 and lora(L, wsb=need - 1) == WORKSPACE
    for name in ("x", "a", "b", "base", "y", "ws"):
        assert lora(L, **{name: 0x10008}) == ALIGN, name
    assert lora(L, ids=0x10002) == ALIGN and lora(L, s=0x10002) == ALIGN
    assert B.bfly_lora_matmul_workspace_bytes(-1, 256, 512, 16) == 0
    assert B.bfly_lora_matmul_workspace_bytes(4, 256, 512, 12) == 0
    assert B.bfly_lora_matmul_workspace_bytes(0, 256, 512, 16) == 0


def clip(L, count=2, grads=(P["a"], P["b"]), outs=None, numels=(100, 5), dtypes=(0, 1), most=1.0,
         norm=P["c"], ws=P["d"], wsb=1 << 30):
    arr = lambda t, v: None if v is None else (t * max(1, len(v)))(*v)
    return L.bfly_grad_clip(count, arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs),
                            arr(ctypes.c_int64, numels), arr(ctypes.c_int32, dtypes), most, norm,
                            ws, wsb, None)


def test_clip_refusals(L):
    assert clip(L, count=-1) == SIZE
    for most in (0.0, -1.0, float("nan")):
        assert clip(L, most=most) == SIZE
    for name in ("grads", "numels", "dtypes", "norm", "ws"):
        assert clip(L, **{name: None}) == NULL, name
    assert clip(L, grads=(P["a"], None)) == NULL
    assert clip(L, outs=(P["a"], None)) == NULL
    assert clip(L, numels=(100, -1)) == SIZE
    assert clip(L, dtypes=(0, 2)) == DTYPE
    assert clip(L, count=65537) == UNSUPPORTED
    assert clip(L, numels=(1 << 41, 1 << 41)) == UNSUPPORTED
    assert clip(L, wsb=B.bfly_grad_clip_workspace_bytes(2) - 1) == WORKSPACE
    assert clip(L, grads=(0x10002, P["b"])) == ALIGN     # fp32 at 2 bytes
    assert clip(L, grads=(P["a"], 0x10001)) == ALIGN
    assert clip(L, outs=(0x10002, P["b"])) == ALIGN
    assert clip(L, norm=0x10002) == ALIGN and clip(L, ws=0x10008) == ALIGN
    assert B.bfly_grad_clip_workspace_bytes(-1) == 0
    assert B.bfly_grad_clip_workspace_bytes(65537) == 0


def test_the_binding_refuses_tensors_of_the_host():
    x, w, v = torch.zeros((2, 64)), torch.zeros(64), torch.zeros(2)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.bfly_rmsnorm(x, w, 1e-5, y=torch.zeros_like(x))
    with pytest.raises(ValueError):
        B.bfly_rmsnorm_backward(x, w, v, x, torch.zeros_like(x))
    with pytest.raises(ValueError):
        b = torch.zeros((2, 64), dtype=torch.bfloat16)
        B.bfly_lora_matmul(b, torch.zeros(2, dtype=torch.int32), b.reshape(1, 2, 64)[:, :2],
                           torch.zeros((1, 8, 2), dtype=torch.bfloat16), torch.zeros(1),
                           torch.zeros((2, 8)), ws)
    with pytest.raises(ValueError):
        B.bfly_grad_clip([w], 1.0, v, ws)


def extension():
    if not os.path.exists(os.path.join(os.path.dirname(B.library_path), "_tensors.so")):
        pytest.skip("the extension is not built")
    return B._ext()


def refused(call, *args, error):
    for _ in range(3):
        with pytest.raises(error):
            call(0, 0, *args)


def test_the_lists_of_gradients_are_checked():
    ext, ok = extension(), torch.zeros(3)
    clip = lambda grads, error, outs=None: refused(ext.grad_clip, 1.0, None, None, grads, outs,
                                                   error=error)
    assert ext.grad_clip(0, 0, 1.0, None, None, [], None) == NULL      # the library's answer
    assert ext.grad_clip(0, 0, 1.0, None, None, (), []) == NULL
    assert ext.grad_clip(0, 0, 0.0, None, None, [], None) == SIZE
    for bad, error in ((3, TypeError), (None, TypeError), ([3], TypeError),
                       ([ok.double()], TypeError), ([torch.zeros(2, dtype=torch.int8), ok], TypeError),
                       ([None], TypeError), ([ok.to_sparse()], ValueError),
                       ([torch.zeros((3, 4)).T], ValueError), ([ok], ValueError)):
        clip(bad, error)
        if bad is not None:
            clip([], error, bad)
    refused(ext.grad_clip, "1", None, None, [], None, error=TypeError)
    refused(ext.grad_clip, 1.0, ok.half(), None, [], None, error=TypeError)
    refused(ext.grad_clip, 1.0, ok, None, [], None, error=ValueError)       # [3]
    refused(ext.grad_clip, 1.0, ok[:2], None, [], None, error=ValueError)   # not on a GPU
    refused(ext.grad_clip, 1.0, None, None, [], error=TypeError)


def test_overlapping_outputs_are_found():
    ext = extension()

    def apart(ins, outs, numels, types=None):
        return ext.overlaps(tuple(ins), None if outs is None else tuple(outs), tuple(numels),
                            tuple(types or [0] * len(ins))) is None

    assert apart([], [], []) and apart([], None, [])
    assert apart([64], [64], [4]) and apart([64], None, [4])      # in place
    assert not apart([64], [68], [4])                             # moved by an element
    assert not apart([64], [60], [4])
    assert apart([64], [80], [4]) and apart([64], [48], [4])
    assert apart([64], [72], [4], [1])                            # bf16: 8 bytes
    assert not apart([64, 128], [128, 64], [4, 4])                # swapped
    assert not apart([64, 128], [256, 64], [4, 4])
    assert apart([64, 128], [256, 64], [0, 4])                    # the first is empty
    assert not apart([64, 64], [64, 256], [4, 4])                 # read again after it is written
    assert apart([64, 64], [128, 256], [4, 4])
    assert not apart([64, 64], None, [4, 4]) and not apart([64, 64], [128, 140], [4, 4])
    assert not apart([64, 60], None, [4, 2]) and apart([64, 60], None, [4, 2], [0, 1])
    assert not apart([64, 64], [100, 72], [16, 1])                # an output inside an input
    assert not apart([72, 300], [500, 64], [1, 16])               # an input inside an output
    n = 50
    ins = [4096 + 64 * (i * 7 % n) for i in range(n)]
    assert apart(ins, ins, [16] * n) and apart(ins, None, [16] * n)
    assert not apart(ins, None, [17] * n)
    assert apart(ins, [1 << 20 | 64 * i for i in range(n)], [16] * n)
    assert not apart(ins, [a + 4 for a in ins], [15] * n)
    for bad in (((), (), ()), ((1,), (), (), ()), ((), (), (1,), ()), ((), (), (), [])):
        with pytest.raises((TypeError, ValueError)):
            ext.overlaps(*bad)


def test_the_tensors_of_a_norm_are_checked():
    ext, x = extension(), torch.zeros((3, 64))
    w, v, c = torch.zeros(64), torch.zeros(3), torch.zeros((3, 64), dtype=torch.int8)
    # eps, format, group, x, weight, y, codes, scales, residual, h, rstd: a call
    # whose tensors are as they have to be stops at the GPU they are not on
    good = [1e-5, 0, None, x, w, x, c, torch.zeros((3, 1), dtype=torch.float16), x, x, v]
    refused(ext.rmsnorm, *good, error=ValueError)
    for at, value, error in ((0, "1", TypeError), (0, None, TypeError), (1, 1.5, TypeError),
                             (1, 1 << 40, ValueError), (2, "n", TypeError), (2, 1 << 32, ValueError),
                             (3, None, TypeError), (3, 5, TypeError), (3, x.half(), TypeError),
                             (3, x[0], ValueError), (3, x.to_sparse(), ValueError),
                             (3, x[:, ::2], ValueError), (4, 5, TypeError),
                             (4, w.double(), TypeError), (4, w[1:], ValueError),
                             (5, x.half(), TypeError), (5, x[1:], ValueError), (6, x, TypeError),
                             (6, c[:, 1:], ValueError), (7, v, TypeError),
                             (7, x.half(), ValueError), (2, 32, ValueError), (2, 0, ValueError),
                             (8, x.bfloat16(), TypeError), (9, x.bfloat16(), TypeError),
                             (8, x.T, ValueError), (9, w, ValueError), (10, v.double(), TypeError),
                             (10, w, ValueError)):
        refused(ext.rmsnorm, *good[:at], value, *good[at + 1:], error=error)
    refused(ext.rmsnorm, *good[:-1], error=TypeError)
    # h, weight, rstd, dy, dx, dweight, dh, workspace
    good = [x, w, v, x, x, w, x, v]
    refused(ext.rmsnorm_backward, *good, error=ValueError)
    for at, value, error in ((0, None, TypeError), (0, x.long(), TypeError), (0, x[0], ValueError),
                             (1, v, ValueError), (2, w, ValueError), (3, x.half(), TypeError),
                             (3, x[:2], ValueError), (4, x.bfloat16(), TypeError),
                             (5, w.bfloat16(), TypeError), (6, x.bfloat16(), TypeError),
                             (6, x.T, ValueError), (7, 5, TypeError), (7, x.T, ValueError),
                             (7, x.to_sparse(), ValueError)):
        refused(ext.rmsnorm_backward, *good[:at], value, *good[at + 1:], error=error)
    refused(ext.rmsnorm_backward, *good, None, error=TypeError)


def test_the_tensors_of_adapters_are_checked():
    ext, b = extension(), torch.zeros((3, 64), dtype=torch.bfloat16)
    a, up = torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 8), dtype=torch.bfloat16)
    y, ids = torch.zeros((3, 16)), torch.zeros(3, dtype=torch.int32)
    # x, lora_a, y, ids, lora_b, scaling, base, workspace
    v2 = torch.zeros(2)
    good = [b, a, y, ids, up, v2, y, ids]
    refused(ext.lora_matmul, *good, error=ValueError)
    for at, value, error in ((0, None, TypeError), (0, b.float(), TypeError), (0, b[0], ValueError),
                             (0, b[:, ::2], ValueError), (1, a[0], ValueError),
                             (1, a.float(), TypeError), (1, a[:, :, :8], ValueError),
                             (2, None, TypeError), (2, y.half(), TypeError), (2, y[1:], ValueError),
                             (3, ids.long(), TypeError), (3, ids[1:], ValueError),
                             (4, a, ValueError), (4, up.float(), TypeError),
                             (5, v2.double(), TypeError), (5, ids, TypeError), (5, y[0], ValueError),
                             (6, y.T, ValueError), (6, y.half(), TypeError), (7, "w", TypeError)):
        refused(ext.lora_matmul, *good[:at], value, *good[at + 1:], error=error)
    with pytest.raises(TypeError):
        ext.lora_matmul(0, "0", *good)
    with pytest.raises(TypeError):
        ext.lora_matmul()
    with pytest.raises(ValueError):
        ext.bind(0, 1, 2, 3)


def test_a_workspace_for_the_most_rows_serves_fewer(L):
    size = B.bfly_lora_matmul_workspace_bytes
    steps = list(range(1, 4200)) + list(range(4200, 16500, 7)) + [1 << b for b in range(15, 24)]
    for k, rank in ((4096, 64), (65536, 8), (65536, 256), (8, 8), (1000, 16), (4096, 24),
                    (11008, 40), (4096, 72), (512, 128), (11008, 200)):
        sizes = [size(r, 4096, k, rank) for r in steps]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (k, rank)
        # and one for the longest rows or the highest rank
        assert all(size(r, 8, k, rank) <= size(r, 8, min(65536, 2 * k), rank) and
                   size(r, 8, k, rank) <= size(r, 8, k, min(256, rank + 8)) for r in steps[::17])
    # a call with the size for the most rows passes its check, one with a byte less does not
    need = size(4096, 256, 4096, 64)
    for rows in (1, 64, 300, 2048, 2700, 4096):
        assert lora(L, rows=rows, k=4096, rank=64, wsb=need, ids=0x10002) == ALIGN
    assert lora(L, rows=4096, k=4096, rank=64, wsb=need - 1, ids=0x10002) == WORKSPACE
    for n in (16, 128, 129, 1024, 1025, 4095, 4096, 16384):
        sizes = [B.bfly_rmsnorm_backward_workspace_bytes(r, n) for r in steps]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), n
    sizes = [B.bfly_grad_clip_workspace_bytes(c) for c in range(0, 65537, 13)]
    assert all(a < b for a, b in zip(sizes, sizes[1:]))


def test_the_adapters_workspace_holds_their_sums():
    # how a call is cut up, by itself: 1552 bytes of order to a block of 256 rows,
    # and the splits' fp32 sums of t in rows of a multiple of 16 ranks
    for rows in list(range(1, 700)) + list(range(700, 20000, 97)):
        blocks, tiles = -(-rows // 256), -(-rows // 64)
        for k in (8, 520, 4096, 11008, 65536):
            for rank in (8, 16, 24, 32, 40, 64, 72, 128, 136, 192, 200, 256):
                ways = -(-rank // (16 if rank <= 16 else 32 if rank <= 32 else 64))
                splits = max(1, min(256 // ((tiles + blocks) * ways), -(-k // 512)))
                run = -(-(-(-k // splits)) // 128) * 128
                need = 1552 * blocks + 4 * -(-k // run) * rows * -(-rank // 16) * 16
                assert B.bfly_lora_matmul_workspace_bytes(rows, 64, k, rank) >= need


def test_codes_of_a_type_that_names_another_format_are_refused():
    ext, x = extension(), torch.zeros((3, 64))
    v, i8 = torch.zeros(3), torch.zeros((3, 64), dtype=torch.int8)
    scales = torch.zeros((3, 1), dtype=torch.float16)
    call = lambda codes, fmt, error: refused(ext.rmsnorm, 1e-5, fmt, None, x, None, None, codes,
                                             scales, None, None, v, error=error)
    e4m3, u8 = i8.view(torch.float8_e4m3fn), i8.view(torch.uint8)
    call(e4m3, B.BFLY_Q8_INT8, TypeError)
    call(i8, B.BFLY_Q8_E4M3, TypeError)
    # what names the format, and bytes for either, stop at the GPU they are not on
    for codes, fmt in ((i8, B.BFLY_Q8_INT8), (e4m3, B.BFLY_Q8_E4M3), (u8, B.BFLY_Q8_INT8),
                       (u8, B.BFLY_Q8_E4M3)):
        call(codes, fmt, ValueError)
