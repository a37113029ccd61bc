"""The attention's own workspace: of the stream and the device that the call runs on, however its arguments are given."""
import contextlib

import numpy as np
import pytest
import torch

import bit_quantized_matvec_q1_amd.lowbit as L
from gpu_util import dev, say
from test_serve_attention import Case


@pytest.fixture
def taken(monkeypatch):
    """On the host: where the workspace is allocated, (stream, device), and which stream the call gets.  The current
    device is 2, and its current stream 0x111."""
    seen, inside = [], []

    @contextlib.contextmanager
    def within(stream):
        inside.append(stream)
        yield
        inside.pop()

    def empty(n, dtype=None, device=None):
        seen.append((inside[-1] if inside else "current", torch.device(device).index))
        return torch.zeros(n, dtype=dtype)

    monkeypatch.setattr(L, "_raw_stream", lambda i: 0x111)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: raw)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "stream", within)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(L, "_call", lambda name, fn, stream, tensors, args: seen.append(stream))
    return seen


A = 1 << 20


@pytest.mark.parametrize("stream,where", [(0x222, 0x222), (0x111, "current"), (0, "default"), (None, "default")])
def test_addresses_alone(taken, stream, where):
    L.lowbit_kv_attention(L.F16, A, 1, 1, 8, 2, 128, A, A, A, 10000, A, 10000, 16, 1, 100000, 0.1, A, stream=stream)
    assert taken == [(where, 2), 0 if stream is None else stream]


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on GPU 1."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


@pytest.mark.parametrize("stream,where", [(0x222, 0x222), (None, "current"), (0, "default")])
def test_an_address_for_the_outputs_among_tensors(taken, stream, where):
    q = torch.zeros(1, 8, 128, dtype=torch.float16).as_subclass(OnDevice)
    L.lowbit_kv_attention(L.F16, q, 1, 1, 8, 2, 128, A, A, A, 10000, A, 10000, 16, 1, 100000, 0.1, A, stream=stream)
    assert taken == [(where, 1), stream]


@pytest.mark.gpu
@pytest.mark.parametrize("as_address", [False, True])
@pytest.mark.parametrize("which", ["side", "default"])
def test_memory_taken_right_after_the_call_is_left_alone(as_address, which):
    """The call waits on its stream while another stream takes and fills as much memory as its workspace."""
    say(f"case workspace {which} address={as_address}")
    c = Case(60, "f16", 128, 16, 4, 1, [1500, 700], [1, 1], extra=0)
    ref, tol = c.want()
    args = [dev(x) for x in (c.cu, np.array(c.lens, np.int32), c.table, c.cache)]
    q, out = c.q.cuda(), torch.empty_like(c.q, device="cuda")
    need = L.lowbit_kv_attention_workspace(c.T, 2, 4, 1, 128, 1, 1500)
    one, other = torch.cuda.Stream(), torch.cuda.Stream()
    run, fill = (one, other) if which == "side" else (torch.cuda.default_stream(), other)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(fill):
            spare = torch.empty(need, dtype=torch.uint8, device="cuda")  # this stream's pool has memory of the size
            del spare
            with torch.cuda.stream(run):
                torch.cuda._sleep(20_000_000)
            L.lowbit_kv_attention(L.F16, q.data_ptr() if as_address else q, c.T, 2, 4, 1, 128, args[0], args[1], args[2], c.stride, args[3],
                                  c.pages, 16, 1, 1500, c.scale, out.data_ptr() if as_address else out, stream=run)
            mine = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(7)
        torch.cuda.synchronize()
        assert (mine == 7).all()
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
