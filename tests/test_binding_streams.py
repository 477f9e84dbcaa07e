"""Tensors that a call makes belong to the stream it runs on: with ``stream=``
given, results and workspaces are taken under that stream, as inside
``torch.cuda.stream``.  (Taken under the current stream, memory that work queued
there still uses could be written by the call, and a workspace could be handed to
work queued there while the call still uses it.)  Stubs in place of the device, the
allocator and the kernels; the GPU's side is in test_gpu_streams.py.
"""
import contextlib

import pytest

import tiled_fp32_gemm_03_amd as g

torch = pytest.importorskip("torch")

DEV = torch.device("cuda", 0)
CURRENT, SIDE = 0x1000, 0x2000


class OnDevice(torch.Tensor):
    """A host tensor that says that it is on the device."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: DEV)


def _tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def taken(monkeypatch):
    """(stream, bytes) of every tensor made, under stubs."""
    now, made = [CURRENT], []
    plain_empty = torch.empty

    def empty(*shape, dtype=torch.float32, device=None):
        t = plain_empty(*shape, dtype=dtype).as_subclass(OnDevice)
        made.append((now[-1], t.numel() * t.element_size()))
        return t

    @contextlib.contextmanager
    def under(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    class Stream:
        def __init__(self, cuda_stream, device=None):
            self.cuda_stream = cuda_stream

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: now[-1], raising=False)
    for name in ("_launch", "gemm_f32_ex", "gemm_mixed", "gemm_f32_splitk"):
        monkeypatch.setattr(g, name, lambda *args: None)
    return made


def _calls():
    a, b = _tensor(64, 4096, dtype=torch.float32), _tensor(4096, 64, dtype=torch.float32)
    h = _tensor(8, 64)
    q = g.MxTensor(_tensor(8, 32, dtype=torch.uint8), _tensor(8, 16, dtype=torch.uint8), 64)
    return {
        "matmul": lambda s: g.matmul(a, b, stream=s),
        "matmul_mixed": lambda s: g.matmul_mixed(h, _tensor(64, 8), stream=s),
        "matmul_splitk": lambda s: g.matmul_splitk(a, b, splits=4, stream=s),
        "mx_quantize": lambda s: g.mx_quantize(h, stream=s),
        "mx_dequantize": lambda s: g.mx_dequantize(q, stream=s),
        "matmul_mx": lambda s: g.matmul_mx(q, q, stream=s),
        "matmul_mx of rows": lambda s: g.matmul_mx(h, q, stream=s),
        "moe_layer": lambda s: g.moe_layer(h, _tensor(4, 64), _tensor(4, 64, 64), _tensor(4, 64, 32), 2,
                                           stream=s),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_tensors_belong_to_the_stream(taken, name):
    call = _calls()[name]
    want = {"matmul_splitk": 2, "mx_quantize": 2, "moe_layer": 4}.get(name, 1)
    for stream, owner in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE), (0, 0)):
        taken.clear()
        call(stream)
        assert len(taken) == want, (name, stream, taken)
        assert all(s == owner for s, _ in taken), (name, stream, taken)
