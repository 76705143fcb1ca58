"""Scratch that the binding makes for a call on a stream comes from that stream's
memory: only there is what lies in it before and afterwards in order with the
call.  With torch's allocation and streams replaced, so that these run on a
machine without a GPU."""
import contextlib
import os
from types import SimpleNamespace

import pytest

import learnable_butterfly_rotation_amd as B

torch = pytest.importorskip("torch")

DEVICE = torch.device("cuda", 0)


@pytest.fixture
def made(monkeypatch):
    """(bytes, stream) of every allocation; streams by their handles, 1 torch's
    current one."""
    if not os.path.exists(B.library_path):
        pytest.skip("libbfly.so not built")
    log, current = [], [1]
    stream = lambda handle: SimpleNamespace(cuda_stream=handle, device=DEVICE)

    @contextlib.contextmanager
    def on(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def external(handle, device=None):
        assert handle, "not a handle of a stream"  # torch makes a new stream of it
        return stream(handle)

    def empty(n, dtype, device):
        assert dtype == torch.uint8 and device == DEVICE
        log.append((n, current[-1]))
        return SimpleNamespace(record_stream=lambda s: None, element_size=lambda: 1,
                               numel=lambda: n, data_ptr=lambda: 0x10000)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: stream(0))
    return log, stream


def rows(*shape, dtype=torch.bfloat16):
    return SimpleNamespace(shape=shape, device=DEVICE, dtype=dtype, get_device=lambda: 0,
                           data_ptr=lambda: 0x20000)


def test_scratch_of_the_attention(made, monkeypatch):
    log, stream = made
    calls = []
    monkeypatch.setattr(B, "_ext", lambda: SimpleNamespace(cache_attention="attention"))
    monkeypatch.setattr(B, "_call", lambda f, like, s, *args: calls.append((s, args[-1])))
    need = B.bfly_cache_attention_workspace_bytes(3, 32, 8, 128, 64 * 100)
    assert need > 0
    q, cache, tables = rows(3, 32, 128), rows(9, 8, 64, 128), rows(3, 100)
    for given, expected in ((None, 1), (stream(77), 77), (78, 78), (0, 0), (stream(0), 0)):
        log.clear(), calls.clear()
        B.bfly_cache_attention(q, cache, cache, tables, None, None, stream=given)
        assert log == [(need, expected)]
        assert calls[0][0] is given and calls[0][1] is not None
    log.clear()
    B.bfly_cache_attention(q, cache, cache, tables, None, None, max_len=20, stream=stream(77))
    B.bfly_cache_attention(q, cache, cache, tables, None, None, workspace="mine", stream=77)
    assert log == [] and calls[-1][1] == "mine"


@pytest.mark.parametrize("call", ["forward", "forward_quant", "kron_forward"])
def test_scratch_of_the_forwards(made, monkeypatch, call):
    log, stream = made
    got = []
    library = SimpleNamespace(
        bfly_forward_workspace_bytes=B.lib().bfly_forward_workspace_bytes,
        **{"bfly_" + call: lambda *args: got.append(args[-1]) or 0})
    monkeypatch.setattr(B, "lib", lambda: library)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: stream(1))
    x, table = rows(6, 256), rows(8, 128, dtype=torch.float32)
    need = B.bfly_forward_workspace_bytes(6, 256)
    assert need > 0
    for given, handle in ((None, 1), (stream(77), 77), (78, 78), (0, 0)):
        log.clear(), got.clear()
        if call == "forward":
            B.bfly_forward(x, x, theta=table, stream=given)
        elif call == "forward_quant":
            B.bfly_forward_quant(x, x, x, x, theta=table, stream=given)
        else:
            B.bfly_kron_forward(rows(6, 512), x, rows(2, 2), theta_b=table, stream=given)
        assert log == [(need, handle)] and got == [handle]
