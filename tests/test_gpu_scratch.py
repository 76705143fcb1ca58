"""Calls on a stream of the caller's whose scratch the binding makes."""
import pytest

import learnable_butterfly_rotation_amd as B
from test_gpu_cache import U8, Batch, gpu, ints  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def bytes_of(stream):
    """The memory that torch keeps for a stream, by its handle."""
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == stream)


@pytest.mark.parametrize("handle", [False, True])
def test_scratch_of_the_attention(handle):
    """It is of that stream's memory, and what the current stream still works
    on in memory that torch has back is not touched, nor touches the call."""
    b = Batch("int8", [4000, 100], 8, 2, 64, 16, seed=31)
    t, n = ints(b.tables), ints(b.lens)
    want = b.run(tables=t, lens=n)[0].clone()
    need = B.bfly_cache_attention_workspace_bytes(2, 8, 2, 64, b.width * 16)
    assert need > 0
    s = torch.cuda.Stream()
    on = s.cuda_stream if handle else s
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = bytes_of(s.cuda_stream)
    b.out()
    s.wait_stream(torch.cuda.current_stream())
    b.run(tables=t, lens=n, stream=on)
    torch.cuda.synchronize()
    assert bytes_of(s.cuda_stream) >= before + need
    assert torch.equal(b.y, want)
    for _ in range(20):
        b.y.fill_(7.0)
        big = torch.randn((2048, 2048), device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            big = big @ big * 1e-2
        junk = torch.full((need,), 0x7F, dtype=U8, device="cuda")
        kept = junk + 1
        del junk, big                                   # their kernels may yet have to run
        b.run(tables=t, lens=n, stream=on)
        torch.cuda.synchronize()
        assert torch.equal(b.y, want) and (kept == 0x80).all()


def test_the_default_stream_by_its_handle():
    b = Batch("int8", [4000, 100], 8, 2, 64, 16, seed=32)
    want = b.run()[0].clone()
    b.out()
    b.run(stream=0)
    torch.cuda.synchronize()
    assert torch.equal(b.y, want)


def test_scratch_of_a_forward():
    x = torch.randn((64, 8192), device="cuda")
    theta = torch.randn((13, 4096), device="cuda")
    want, y = torch.empty_like(x), torch.empty_like(x)
    B.bfly_forward(x, want, theta=theta)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = bytes_of(s.cuda_stream)
    B.bfly_forward(x, y, theta=theta, stream=s)
    torch.cuda.synchronize()
    assert bytes_of(s.cuda_stream) >= before + B.bfly_forward_workspace_bytes(64, 8192)
    assert torch.equal(y, want)
