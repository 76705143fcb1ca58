"""bfly_lora_matmul on the GPU against the formula in 64 bits.

Tolerance (u = 2^-24): t = A x is a sum of k exact products in fp32, at most
k + 64 roundings whatever the order; times scaling one more; what the bf16
terms of s t leave out is at most 2^-16 of it (two terms, bf16 y) or 2^-24
(three, fp32 y); the second product sums terms * rank exact products; the
base's addition one rounding; y half a step of its type."""
import numpy as np
import pytest

import learnable_butterfly_rotation_amd as B

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, rows, k, n_out, rank, num, ids="mixed", base=BF16, y=BF16, seed=0):
        g = torch.Generator().manual_seed(seed + rows + 7 * k + rank)
        self.x = torch.randn((rows, k), generator=g).to(BF16)
        self.a = (torch.randn((num, rank, k), generator=g) / k ** 0.5).to(BF16)
        self.b = torch.randn((num, n_out, rank), generator=g).to(BF16)
        self.s = 0.5 + torch.rand(num, generator=g)
        if isinstance(ids, str):
            if ids == "mixed":
                self.ids = torch.randint(-1, num, (rows,), generator=g, dtype=torch.int32)
            elif ids == "runs":
                self.ids = torch.sort(torch.randint(0, num, (rows,), generator=g,
                                                    dtype=torch.int32))[0]
            else:
                self.ids = torch.full((rows,), int(ids), dtype=torch.int32)
        else:
            self.ids = torch.tensor(ids, dtype=torch.int32)
        self.base = None if base is None else torch.randn((rows, n_out), generator=g).to(base)
        self.y_dt, self.num, self.rank = y, num, rank

    def run(self, in_place=False, stream=None):
        rows, k = self.x.shape
        n_out = self.b.shape[1]
        dev = [t.cuda() for t in (self.x, self.ids, self.a, self.b, self.s)]
        base = None if self.base is None else self.base.cuda()
        y = base if in_place else torch.full((rows + 1, n_out), 7.0, dtype=self.y_dt,
                                             device="cuda")
        ws = torch.full((max(1, B.bfly_lora_matmul_workspace_bytes(rows, n_out, k, self.rank)),),
                        0x7F, dtype=torch.uint8, device="cuda")
        B.bfly_lora_matmul(*dev, y[:rows], ws, base=base)
        torch.cuda.synchronize()
        if not in_place:
            assert (y[rows:] == 7.0).all()
        return y[:rows]

    def check(self, y):
        rows, k = self.x.shape
        x, base = np64(self.x), 0.0 if self.base is None else np64(self.base)
        add = np.zeros((rows, self.b.shape[1]))
        err = np.zeros_like(add)
        for i in range(self.num):
            at = np.nonzero(self.ids.numpy() == i)[0]
            if not len(at):
                continue
            a, b, s = np64(self.a[i]), np64(self.b[i]), float(self.s[i])
            t, tabs = x[at] @ a.T * s, np.abs(x[at]) @ np.abs(a).T * s
            terms, cut = (2, 2.0 ** -16) if self.y_dt == BF16 else (3, 2.0 ** -24)
            et = 1.01 * (k + 64) * U * tabs + (2 * U + cut) * np.abs(t)
            add[at] = t @ b.T
            err[at] = et @ np.abs(b).T + 1.01 * terms * self.rank * U * (np.abs(t) @ np.abs(b).T)
        want = base + add
        half = torch.finfo(self.y_dt).eps / 2
        tol = err + U * (np.abs(want) + err) + half * (np.abs(want) + 2 * err)
        got = np64(y)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
        none = (self.ids.numpy() < 0) | (self.ids.numpy() >= self.num)
        if none.any():
            b0 = torch.zeros_like(y.cpu()) if self.base is None else self.base.to(self.y_dt)
            assert torch.equal(y.cpu()[none], b0[none])


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 136, 200, 256])
@pytest.mark.parametrize("y", [F32, BF16])
def test_ranks(rank, y):
    c = Case(37, 520, 272, rank, 3, y=y)
    c.check(c.run())


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 300, 513, 1100])
@pytest.mark.parametrize("ids", ["mixed", "runs", "0", "-1", "5"])
def test_rows_and_orders(rows, ids):
    c = Case(rows, 264, 136, 16, 4, ids=ids)
    c.check(c.run())


@pytest.mark.parametrize("rank", [8, 40, 104, 176])
@pytest.mark.parametrize("base,y", [(None, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_many_rows(rank, base, y):
    for ids in ("mixed", "runs"):
        c = Case(2300, 136, 328, rank, 5, ids=ids, base=base, y=y)
        c.check(c.run())


@pytest.mark.parametrize("k", [8, 16, 120, 128, 136, 504, 512, 520, 1000, 4096, 11008])
def test_depths(k):
    for rows in (3, 70):
        c = Case(rows, k, 64, 8, 2, y=F32, base=F32)
        c.check(c.run())


@pytest.mark.parametrize("n_out", [8, 16, 24, 32, 40, 64, 248, 256, 264, 1000, 4096])
def test_widths(n_out):
    for rows in (3, 70):
        c = Case(rows, 128, n_out, 16, 2)
        c.check(c.run())


@pytest.mark.parametrize("base", [None, F32, BF16])
@pytest.mark.parametrize("y", [F32, BF16])
def test_types(base, y):
    for rows in (5, 260):
        c = Case(rows, 264, 136, 32, 5, base=base, y=y)
        c.check(c.run())


@pytest.mark.parametrize("y", [F32, BF16])
def test_in_place(y):
    for rows in (5, 260):
        c = Case(rows, 264, 136, 32, 5, base=y, y=y)
        c.check(c.run(in_place=True))


def test_every_row_its_own_adapter():
    rng = np.random.default_rng(0)
    c = Case(256, 128, 64, 8, 300, ids=rng.permutation(300)[:256])
    c.check(c.run())


@pytest.mark.parametrize("num", [1, 2, 255, 256, 257])
@pytest.mark.parametrize("rows", [64, 65, 128, 200, 256, 321])
def test_numbers_of_adapters(num, rows):
    rng = np.random.default_rng(num + rows)
    for ids in (rng.integers(-1, num, rows), num - 1 - np.arange(rows) % min(num, 7),
                np.where(np.arange(rows) % 3 == 0, num - 1, 0)):
        c = Case(rows, 128, 64, 8, num, ids=ids)
        c.check(c.run())


def test_ids_out_of_range():
    c = Case(7, 128, 64, 8, 3, ids=[0, 3, 2, -2147483648, 2147483647, -1, 1])
    c.check(c.run())


def test_a_row_does_not_depend_on_the_others():
    # the same rows alone, and among others in another order, in one block of
    # rows and so with the same split of the k axis
    c = Case(64, 1024, 128, 16, 6)
    y = c.run()
    perm = torch.randperm(64, generator=torch.Generator().manual_seed(1))
    d = Case(64, 1024, 128, 16, 6)
    d.x, d.ids, d.base = c.x[perm], c.ids[perm], c.base[perm]
    assert torch.equal(d.run(), y[perm.cuda()])


def test_unused_adapters_and_missing_ranks_are_not_read():
    # adapters that no row has hold NaN; so do the rows of x without one
    c = Case(40, 264, 136, 24, 6)
    c.ids[c.ids == 2] = 4
    c.a[2] = c.b[2] = c.s[2] = float("nan")
    y = c.run()
    c.x[c.ids < 0] = float("nan")
    assert torch.equal(c.run(), y)
    c.x[c.ids < 0] = 0.0
    c.a[2], c.b[2], c.s[2] = 0, 0, 1
    c.check(y)


@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_many_blocks_of_rows(ids):
    c = Case(4300 * 256 + 77, 16, 8, 8, 9, ids=ids, y=F32)
    c.check(c.run())


def test_no_rows():
    c = Case(0, 128, 64, 8, 2)
    c.run()


def test_same_bits_every_time():
    c = Case(300, 4096, 264, 64, 7, y=F32)
    y = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), y)


@pytest.mark.parametrize("rank", [8, 24, 64, 136, 256])
@pytest.mark.parametrize("y", [F32, BF16])
def test_rows_with_an_infinity(rank, y):
    # t is an infinity in every rank; a column of B of one sign passes it on,
    # one of both signs gives NaN; the other rows stay as they are
    c = Case(70, 264, 136, rank, 3, ids="mixed", y=y)
    c.a = c.a.abs() + 0.01
    c.b = c.b.abs() + 0.01
    c.b[:, 1::3] *= -1
    c.b[:, 2::3, 0] *= -1
    want = c.run()
    c.check(want)
    c.ids[5], c.ids[66] = 1, 2
    keep = torch.ones(70, dtype=torch.bool)
    for r, v in ((5, float("inf")), (66, -float("inf"))):
        c.x[r, 77] = v
        keep[r] = False
    got = c.run().cpu()
    assert torch.equal(got[keep], want.cpu()[keep])
    for r, sign in ((5, 1.0), (66, -1.0)):
        assert (got[r, 0::3] == sign * float("inf")).all()
        assert (got[r, 1::3] == -sign * float("inf")).all()
        assert torch.isnan(got[r, 2::3]).all()


@pytest.mark.parametrize("rank", [8, 24, 64, 136, 256])
@pytest.mark.parametrize("y", [F32, BF16])
@pytest.mark.parametrize("in_place", [False, True])
def test_adapters_with_infinities_in_b(rank, y, in_place):
    # what the formula gives, from 64 bits: an infinity of t's sign, its
    # opposite's, NaN where two of them meet and where t is zero; rows whose t
    # bf16 holds exactly (nothing is left for its second term) among them
    inf = float("inf")
    c = Case(70, 264, 136, rank, 3, ids="mixed", y=y, base=y)
    c.ids[:6] = torch.tensor([1, 1, 1, 0, 2, 1], dtype=torch.int32)
    c.s[1] = 1.0
    c.x[0] = 0.0                       # t is zero
    c.x[1:3] = 0.0
    c.x[1, 9] = c.x[2, 40] = 1.0       # t is a column of A
    c.x[5, 7] = inf                    # t is an infinity, of A's sign
    plain = c.b.clone()
    c.x[5, 7] = 1.0
    finite = c.run(in_place).cpu()
    c.x[5, 7] = inf
    put = {(0, 3): {0: inf}, (1, 3): {rank - 1: inf}, (1, 4): {5: -inf}, (1, 9): {2: inf, 6: inf},
           (1, 68): {0: -inf, rank - 1: inf}, (1, 77): {3: float("nan")}, (1, 135): {rank // 2: inf},
           (2, 0): {1: inf, 4: -inf, 7: 1.0}}
    hit = torch.zeros((3, 136), dtype=torch.bool)
    for (i, o), at in put.items():
        hit[i, o] = True
        for j, v in at.items():
            c.b[i, o, j] = v
    got = c.run(in_place).cpu()
    # rows and columns without one keep their bits
    touched = torch.stack([hit[i] if 0 <= i < 3 else torch.zeros(136, dtype=torch.bool)
                           for i in c.ids.tolist()])
    touched[5] = True
    assert torch.equal(got[~touched], finite[~touched])
    assert torch.equal(plain[~hit], c.b[~hit])
    count = 0
    for r, i in enumerate(c.ids.tolist()):
        if not 0 <= i < 3:
            continue
        x, a, b = np64(c.x[r]), np64(c.a[i]), np64(c.b[i])
        with np.errstate(invalid="ignore"):
            t = (a * x).sum(1) * float(c.s[i])
            # t's sign is sure where it is zero exactly or above the sum's error; a
            # column with an infinity at another rank (one of rank 64 has 1.9e-4, the
            # error is up to 2.4e-4) is not compared
            off = 1.01 * (264 + 66) * U * np.abs(a * x).sum(1) * float(c.s[i])
            sure = (t == 0) & (np.abs(a * x).sum(1) == 0) | (np.abs(t) > off) | np.isinf(t)
            want = (b * t).sum(1) + np64(c.base[r])
        for o in np.nonzero(touched[r].numpy())[0]:
            if not sure[~np.isfinite(b[o])].all():
                continue
            if np.isnan(want[o]):
                assert torch.isnan(got[r, o]), (r, o)
            elif np.isinf(want[o]):
                assert got[r, o] == want[o], (r, o, float(got[r, o]), want[o])
            count += 1
    assert count >= 136 + 20


@pytest.mark.parametrize("rank", [16, 64, 136])
def test_one_workspace_for_all_batches(rank):
    # sized for the most rows, and nothing behind a call's own size is touched
    k, n_out, most = 4096, 64, 4096
    ws = torch.empty(B.bfly_lora_matmul_workspace_bytes(most, n_out, k, rank), dtype=torch.uint8,
                     device="cuda")
    for rows in (most, 2048, 700, 64, 3):
        c = Case(rows, k, n_out, rank, 1, ids="0", y=F32)
        want = c.run()
        dev = [t.cuda() for t in (c.x, c.ids, c.a, c.b, c.s)]
        ws.fill_(0x7F)
        y = torch.empty_like(want)
        B.bfly_lora_matmul(*dev, y, ws, base=c.base.cuda())
        assert torch.equal(y, want)
        assert (ws[B.bfly_lora_matmul_workspace_bytes(rows, n_out, k, rank):] == 0x7F).all()
        if rows <= 700:
            c.check(y)


@pytest.mark.parametrize("rank", [8, 40, 72, 256])
@pytest.mark.parametrize("y", [F32, BF16])
def test_adapters_of_nothing_but_infinities_or_nan(rank, y):
    c = Case(300, 264, 136, rank, 4, y=y)
    c.x, c.a = c.x.abs() + 0.01, c.a.abs() + 0.01   # t is positive
    finite = c.run().cpu()
    c.b[1], c.b[2] = float("inf"), float("nan")
    c.b[3] = -float("inf")
    c.b[3, ::2, rank - 1] = float("inf")
    got = c.run().cpu()
    keep = (c.ids != 1) & (c.ids != 2) & (c.ids != 3)
    assert torch.equal(got[keep], finite[keep])
    assert (got[c.ids == 1] == float("inf")).all() and torch.isnan(got[c.ids == 2]).all()
    assert torch.isnan(got[c.ids == 3][:, ::2]).all()
    assert (got[c.ids == 3][:, 1::2] == -float("inf")).all()
    assert all((c.ids == i).any() for i in range(4))
