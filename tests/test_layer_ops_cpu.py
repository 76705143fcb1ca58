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


def test_the_list_of_gradients_is_checked():
    ext, ok = extension(), torch.zeros(3)
    assert ext.describe([], 0, True) == (b"", b"", b"")
    for bad, error in ((3, TypeError), ([3], TypeError), ([ok.double()], TypeError),
                       ([torch.zeros(2, dtype=torch.int8), ok], TypeError), ([ok], ValueError),
                       ([None], TypeError)):
        for _ in range(3):
            with pytest.raises(error):
                ext.describe(bad, 0, False)
    with pytest.raises(TypeError):
        ext.describe([])


def test_outputs_and_other_gradients_are_told_apart():
    ext = extension()

    def apart(ins, outs, numels, types=None):
        n = len(ins)
        pack = lambda t, v: bytes((t * n)(*v))
        return ext.apart(pack(ctypes.c_uint64, ins), pack(ctypes.c_uint64, outs),
                         pack(ctypes.c_int64, numels), pack(ctypes.c_int32, types or [0] * n))

    assert apart([], [], []) is True
    assert apart([64], [64], [4]) is True                         # in place
    assert apart([64], [68], [4]) is False                        # moved by an element
    assert apart([64], [60], [4]) is False
    assert apart([64], [80], [4]) is True and apart([64], [48], [4]) is True
    assert apart([64], [72], [4], [1]) is True                    # bf16: 8 bytes
    assert apart([64, 128], [128, 64], [4, 4]) is False           # swapped
    assert apart([64, 128], [256, 64], [4, 4]) is False
    assert apart([64, 128], [256, 64], [0, 4]) is True            # the first is empty
    assert apart([64, 64], [64, 256], [4, 4]) is False            # read again after it is written
    assert apart([64, 64], [128, 256], [4, 4]) is True
    assert apart([64, 64], [100, 72], [16, 1]) is False           # an output inside an input
    assert apart([72, 300], [500, 64], [1, 16]) is False          # an input inside an output
    n = 50
    ins = [4096 + 64 * (i * 7 % n) for i in range(n)]
    assert apart(ins, ins, [16] * n) is True
    assert apart(ins, [1 << 20 | 64 * i for i in range(n)], [16] * n) is True
    assert apart(ins, [a + 4 for a in ins], [15] * n) is False
    for bad in ((b"", b"", b"", b"1"), (b"", b"", b"", b"1234"), (b"",), (b"", b"", b"", 3)):
        with pytest.raises((TypeError, ValueError)):
            ext.apart(*bad)


def test_a_tensor_is_checked():
    ext, x = extension(), torch.zeros((3, 4))
    assert ext.at("x", None, (3, 4), 1, 0) is None
    for args, error in ((("x", 5, (3, 4), 1, 0), TypeError), (("x", x, [3, 4], 1, 0), TypeError),
                        (("x", x, (3, 4), 2, 0), TypeError), (("x", x, (3, 4), "1", 0), TypeError),
                        (("x", x, (3, 5), 1, 0), ValueError), (("x", x, (3,), 1, 0), ValueError),
                        (("x", x, (3, 4, 1), 1, 0), ValueError),
                        (("x", x, (3, "4"), 1, 0), TypeError),
                        (("x", x.T, (4, 3), 1, 0), ValueError),
                        (("x", x.to_sparse(), (3, 4), 1, 0), ValueError),
                        (("x", x, (3, 4), 1, 0), ValueError),      # not on a GPU
                        (("x", x, (3, 4), 1, -1), ValueError), (("x", x), TypeError)):
        for _ in range(3):
            with pytest.raises(error):
                ext.at(*args)


def test_a_workspace_is_checked():
    ext, x = extension(), torch.zeros((3, 4))
    assert ext.scratch(None, 0) == (None, 0)
    for args, error in (((5, 0), TypeError), ((x, 0), ValueError), ((x, -1), ValueError),
                        ((x.to_sparse(), 0), ValueError), ((x, "0"), TypeError), ((x,), TypeError)):
        for _ in range(3):
            with pytest.raises(error):
                ext.scratch(*args)
