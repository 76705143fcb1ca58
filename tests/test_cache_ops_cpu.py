"""What bfly_cache_write, bfly_cache_read and bfly_cache_attention refuse, at
the C ABI and in the binding: all before any HIP call, so these run on a
machine without a GPU."""
import os

import pytest

import learnable_butterfly_rotation_amd as B

torch = pytest.importorskip("torch")

OK, NULL, SIZE, DTYPE, ALIGN, QUANT, WORKSPACE, UNSUPPORTED, HIP = range(9)
# fake, well-aligned device addresses: validation never dereferences them
P = {v: 0x10000 * (i + 1) for i, v in enumerate("abcdefghijkl")}
FORMATS = (B.BFLY_KV_BF16, B.BFLY_KV_INT8, B.BFLY_KV_E4M3, B.BFLY_KV_INT4)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.library_path):
        pytest.skip("libbfly.so not built")
    return B.lib()


def rows(L, write, k=P["a"], ks=1024, v=P["b"], vs=1024, dt=1, slots=P["c"], tokens=4, kc=P["d"],
         vc=P["e"], sk=P["f"], sv=P["g"], pages=10, kv=8, page=16, d=128, fmt=1):
    # with tokens = 4 a call that passed would reach the GPU: only refusals use it
    if write:
        return L.bfly_cache_write(k, ks, v, vs, dt, slots, tokens, kc, vc, sk, sv, pages, kv, page,
                                  d, fmt, None)
    return L.bfly_cache_read(kc, vc, sk, sv, slots, tokens, k, ks, v, vs, dt, pages, kv, page, d,
                             fmt, None)


@pytest.mark.parametrize("write", [True, False])
def test_cache_rows_refusals(L, write):
    call = lambda **a: rows(L, write, **a)
    assert call(tokens=0) == OK
    assert call(tokens=0, k=None, v=None, slots=None, kc=None, vc=None, sk=None, sv=None) == OK
    for name in ("k", "v", "slots", "kc", "vc", "sk", "sv"):
        assert call(**{name: None}) == NULL, name
    assert call(tokens=0, fmt=0, sk=None, sv=None) == OK
    assert call(fmt=0, sk=None, sv=None, ks=8) == SIZE          # bf16: no scales needed
    assert call(dt=2) == DTYPE and call(dt=-1) == DTYPE
    assert call(fmt=4) == QUANT and call(fmt=-1) == QUANT
    assert call(tokens=-1) == SIZE
    for name in ("pages", "kv", "page", "d"):
        assert call(**{name: 0}) == SIZE and call(**{name: -16}) == SIZE, name
    assert call(ks=1016) == SIZE and call(vs=1016) == SIZE and call(vs=-1024) == SIZE
    for name, value in (("d", 32), ("d", 96), ("d", 512), ("page", 8), ("page", 48),
                        ("page", 131072), ("kv", 4097), ("ks", 1 << 32), ("tokens", 1 << 40)):
        more = {"ks": 1 << 22, "vs": 1 << 22} if name == "kv" else {}
        assert call(**{name: value}, **more) == UNSUPPORTED, (name, value)
    assert call(pages=1 << 15, page=65536) == UNSUPPORTED       # 2^31 slots
    assert call(tokens=0, pages=(1 << 15) - 1, page=65536) == OK
    assert call(tokens=(1 << 24) + 1) == UNSUPPORTED            # 2^34 elements of 8 * 128
    for name in ("k", "v", "kc", "vc"):
        assert call(**{name: 0x10008}) == ALIGN, name
    assert call(ks=1028) == ALIGN and call(vs=1025) == ALIGN
    assert call(slots=0x10002) == ALIGN and call(sk=0x10001) == ALIGN and call(sv=0x10001) == ALIGN


def attend(L, q=P["a"], qs=4096, qd=1, kc=P["b"], vc=P["c"], sk=P["d"], sv=P["e"], tables=P["f"],
           width=8, lens=P["g"], y=P["h"], yd=1, lse=P["i"], rows=4, heads=32, pages=10, kv=8,
           page=16, d=128, fmt=1, scale=0.1, most=128, window=0, ws=P["j"], wsb=1 << 40):
    return L.bfly_cache_attention(q, qs, qd, kc, vc, sk, sv, tables, width, lens, y, yd, lse, rows,
                                  heads, pages, kv, page, d, fmt, scale, most, window, ws, wsb, None)


def test_cache_attention_refusals(L):
    call = lambda **a: attend(L, **a)
    assert call(rows=0) == OK
    assert call(rows=0, q=None, kc=None, vc=None, sk=None, sv=None, tables=None, lens=None, y=None,
                lse=None, ws=None, wsb=0) == OK
    for name in ("q", "kc", "vc", "sk", "sv", "tables", "lens", "y"):
        assert call(**{name: None}) == NULL, name
    assert call(fmt=0, sk=None, sv=None, qs=8) == SIZE          # bf16: no scales needed
    assert call(qd=2) == DTYPE and call(yd=-1) == DTYPE
    assert call(fmt=4) == QUANT and call(fmt=-1) == QUANT
    assert call(rows=-1) == SIZE
    for name in ("heads", "pages", "kv", "page", "d", "most", "width"):
        assert call(**{name: 0}) == SIZE and call(**{name: -16}) == SIZE, name
    assert call(heads=33, qs=8192) == SIZE and call(heads=4) == SIZE
    assert call(most=129) == SIZE and call(window=-1) == SIZE and call(qs=4088) == SIZE
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=scale) == SIZE
    for name, value in (("d", 32), ("d", 96), ("page", 48), ("kv", 4097), ("rows", (1 << 24) + 1),
                        ("heads", 1 << 17), ("rows", 1 << 19), ("qs", 1 << 32)):
        more = {"heads": 4097, "qs": 1 << 24} if name == "kv" else {}
        assert call(**{name: value}, **more) == UNSUPPORTED, (name, value)
    assert call(most=(1 << 30) + 1, width=1 << 27) == UNSUPPORTED
    for name in ("q", "kc", "vc", "y"):
        assert call(**{name: 0x10008}) == ALIGN, name
    assert call(qs=4100) == ALIGN and call(sk=0x10001) == ALIGN and call(sv=0x10001) == ALIGN
    for name in ("tables", "lens", "lse"):
        assert call(**{name: 0x10002}) == ALIGN, name


def test_cache_attention_workspace(L):
    size = B.bfly_cache_attention_workspace_bytes
    for bad in ((-1, 32, 8, 128, 99), (0, 32, 8, 128, 99), (1, 33, 8, 128, 9999),
                (1, 32, 8, 96, 9999), (1, 32, 8, 128, 0), (1, 0, 8, 128, 99),
                ((1 << 24) + 1, 1, 1, 64, 9999)):
        assert size(*bad) == 0, bad
    assert size(4, 32, 8, 128, 20) == 0                         # one workgroup to an item
    need = size(4, 32, 8, 128, 100000)
    long = dict(width=8192, most=100000)
    assert need > 0 and attend(L, **long, wsb=need - 1) == WORKSPACE
    assert attend(L, **long, ws=None) == NULL and attend(L, **long, ws=0x10008) == ALIGN
    assert attend(L, **long, wsb=need, lens=0x10002) == ALIGN   # past the workspace's checks
    assert attend(L, ws=None, wsb=0, most=20, lens=0x10002) == ALIGN
    # one for the largest call serves the others
    steps = list(range(1, 300)) + [1 << b for b in range(9, 18)]
    for heads, kv, d, most in ((32, 8, 128, 8192), (32, 32, 64, 1000), (1, 1, 256, 1 << 20),
                               (40, 8, 128, 300), (64, 1, 256, 131072)):
        for sizes in ([size(r, heads, kv, d, most) for r in steps],
                      [size(r, heads, kv, d, most) for r in steps],
                      [size(3, heads, kv, d, n) for n in range(1, 5000, 7)],
                      [size(3, heads * i, heads * i, d, most) for i in range(1, 40)],
                      [size(3, heads, kv, v, most) for v in (64, 128, 256)]):
            assert all(a <= b for a, b in zip(sizes, sizes[1:])), (heads, kv, d, most)


def extension():
    if not os.path.exists(os.path.join(os.path.dirname(B.library_path), "_tensors.so")):
        pytest.skip("the extension is not built")
    return B._ext()


def refused(call, *args, error):
    for _ in range(3):
        with pytest.raises(error):
            call(0, 0, *args)


def cache(fmt, pages=5, kv=2, page=16, d=64):
    t = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn,
         "int4": torch.uint8}[fmt]
    new = lambda: torch.zeros((pages, kv, page, d // 2 if fmt == "int4" else d), dtype=torch.uint8)
    if fmt == "bf16":
        return [torch.zeros((pages, kv, page, d), dtype=t), torch.zeros((pages, kv, page, d), dtype=t),
                None, None]
    scale = lambda: torch.zeros((pages, kv, page), dtype=torch.float16)
    return [new().view(t), new().view(t), scale(), scale()]


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "int4"])
def test_the_tensors_of_a_cache_are_checked(fmt):
    ext, c = extension(), cache(fmt)
    x, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int32)
    wide = torch.zeros((3, 8, 64))
    for f in (ext.cache_write, ext.cache_read):
        good = [*c, x, x, slots]
        # a call whose tensors are as they have to be stops at the GPU they are not on
        refused(f, *good, error=ValueError)
        refused(f, *c, wide[:, 2:4], wide[:, 6:], slots, error=ValueError)
        with pytest.raises(ValueError, match="on GPU"):
            f(0, 0, *c, wide[:, 2:4], wide[:, 6:], slots)
        half = c[0][..., :32] if fmt != "int4" else c[0][..., :16]
        for at, value, error in ((0, None, TypeError), (0, c[0].double() if fmt != "e4m3" else x,
                                                        (TypeError, ValueError)),
                                 (0, c[0][0], ValueError), (0, half, ValueError),
                                 (1, None, TypeError), (1, c[1][1:], ValueError),
                                 (1, x.half(), TypeError), (1, half, ValueError),
                                 (2, torch.zeros((5, 2, 16)), TypeError),
                                 (2, torch.zeros((5, 2, 15), dtype=torch.float16), ValueError),
                                 (3, torch.zeros((5, 16, 2), dtype=torch.float16), ValueError),
                                 (4, None, TypeError), (4, x[0], ValueError), (4, x.half(), TypeError),
                                 (4, x[:, :1], ValueError), (4, wide, ValueError),
                                 (4, x.transpose(1, 2).contiguous().transpose(1, 2), ValueError),
                                 (4, wide[:, ::4], ValueError), (4, torch.zeros((3, 2, 128)), ValueError),
                                 (4, torch.zeros((3, 2, 128))[:, :, ::2], ValueError),
                                 (5, x.bfloat16(), TypeError), (5, x[:2], ValueError),
                                 (5, None, TypeError), (6, slots.long(), TypeError),
                                 (6, slots[1:], ValueError)):
            refused(f, *good[:at], value, *good[at + 1:], error=error)
        refused(f, *good[:-1], error=TypeError)
    q, y = torch.zeros((3, 6, 64)), torch.zeros((3, 6, 64))
    tables, lse = torch.zeros((3, 7), dtype=torch.int32), torch.zeros((3, 6))
    good = [None, None, 0, *c, q, tables, slots, y, lse, slots]
    refused(ext.cache_attention, *good, error=ValueError)
    with pytest.raises(ValueError, match="on GPU"):
        ext.cache_attention(0, 0, *good)
    for at, value, error in ((0, "1", TypeError), (1, 1.5, TypeError), (1, 1 << 32, ValueError),
                             (2, None, TypeError), (2, 1 << 32, ValueError), (3, None, TypeError),
                             (7, None, TypeError), (7, q[0], ValueError), (7, q.half(), TypeError),
                             (7, q.transpose(0, 1), ValueError), (7, torch.zeros((3, 6, 128)), ValueError),
                             (8, tables.long(), TypeError), (8, tables[1:], ValueError),
                             (8, tables[0], ValueError), (8, torch.zeros((7, 3), dtype=torch.int32).T,
                                                          ValueError),
                             (9, slots[1:], ValueError), (9, lse, TypeError), (10, y[1:], ValueError),
                             (10, y.half(), TypeError), (10, y.transpose(0, 1), ValueError),
                             (11, lse.bfloat16(), TypeError), (11, lse[:, :5], ValueError),
                             (12, 5, TypeError), (12, x.transpose(0, 1), ValueError)):
        refused(ext.cache_attention, *good[:at], value, *good[at + 1:], error=error)
    refused(ext.cache_attention, *good[:-1], error=TypeError)


def test_the_binding_refuses_tensors_of_the_host():
    x, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int32)
    k, v, ks, vs = cache("int8")
    with pytest.raises(ValueError):
        B.bfly_cache_write(x, x, slots, k, v, ks, vs)
    with pytest.raises(ValueError):
        B.bfly_cache_read(k, v, slots, x, x, ks, vs)
    with pytest.raises(ValueError):
        B.bfly_cache_attention(x, k, v, torch.zeros((3, 2), dtype=torch.int32), slots, x, ks, vs)
    with pytest.raises(ValueError):
        extension().bind_cache(0, 1, 2)
    with pytest.raises(TypeError):
        extension().bind_cache(1, 2)


def test_the_attention_workspace_holds_its_chunks(L):
    # how a call's lengths are cut, by itself: head_dim + 4 fp32 to a chunk of a head
    def chunks(rows, heads, kv, d, reach):
        share = heads // kv
        items = rows * kv * -(-share // 16)
        if reach <= 512 or (reach <= 1024 and items >= 128):
            return 1
        chunk = 256 if min(share, 16) * d >= 2048 else 128
        if rows == 1:
            chunk = max(chunk, -(-(-(-items * reach // 512)) // 128) * 128)
        else:
            while chunk < 512 and items * -(-reach // chunk) > 2048:
                chunk *= 2
            if items * -(-reach // chunk) > 8192:
                chunk = max(chunk, -(-(-(-items * reach // 8192)) // 128) * 128)
        return -(-reach // chunk)

    for rows in (1, 2, 3, 7, 16, 33, 64, 100, 256, 257, 1000, 5000, 70000):
        for heads, kv in ((1, 1), (4, 1), (16, 1), (17, 1), (32, 8), (32, 32), (64, 4), (40, 40)):
            for d in (64, 256):
                for most in (1, 100, 512, 513, 1000, 1025, 3000, 8192, 50000, 131072, 1 << 22):
                    need = B.bfly_cache_attention_workspace_bytes(rows, heads, kv, d, most)
                    for reach in {most, min(most, 700), min(most, 2000), min(most, 30000)}:
                        n = chunks(rows, heads, kv, d, reach)
                        used = 0 if n == 1 else 4 * (d + 4) * rows * heads * n
                        assert used <= need, (rows, heads, kv, d, most, reach)
