"""Routing, the experts' products and adapters refuse wrong types, shapes and sizes before
anything is launched, and what they allocate belongs to the call's stream (no GPU needed:
stubs in place of the device and the kernels)."""
import contextlib
import ctypes

import pytest

import tiled_fp32_gemm_03_amd as g

torch = pytest.importorskip("torch")

DEV = torch.device("cuda", 0)
CURRENT, SIDE = 0x1000, 0x2000
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnDevice(torch.Tensor):
    """A tensor without memory that says that it is on the device."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: DEV)
    data_ptr = lambda self: 256  # noqa: E731


def T(*shape, dtype=BF, strides=None):
    if strides is None:
        strides = [1]
        for n in shape[:0:-1]:
            strides.insert(0, strides[0] * n)
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta").as_subclass(OnDevice)


def MX(lead, K):
    return g.MxTensor(T(*lead, (K + 31) // 32 * 16, dtype=torch.uint8), T(*lead, (K + 511) // 512 * 16, dtype=torch.uint8), K)


@pytest.fixture
def launched(monkeypatch):
    calls = []
    monkeypatch.setattr(g, "_launch", lambda *args: calls.append(args))
    plain = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None:
                        plain(*shape, dtype=dtype, device="meta").as_subclass(OnDevice))
    return calls


def _args():
    return dict(x=T(8, 64), ids=T(8, 2, dtype=I32), gates=T(8, 2, dtype=F32), w1=T(4, 96, 64), w2=T(4, 64, 48))


def _experts(save=False, **over):
    a = _args() | over
    return g.moe_experts(a["x"], a["ids"], a["gates"], a["w1"], a["w2"], save=save, out=over.get("out"), workspace=over.get("workspace"))


def _backward(**over):
    a = _args() | dict(dy=T(8, 64), saved=T(16, 96, dtype=F32)) | over
    return g.moe_experts_backward(a["dy"], a["x"], a["ids"], a["gates"], a["w1"], a["w2"], a["saved"])


def _adapters(**over):
    a = dict(x=T(8, 64), w=T(32, 64), a=T(3, 16, 64), b=T(3, 32, 16), ids=T(8, dtype=I32), scales=T(3, dtype=F32)) | over
    return g.matmul_adapters(a["x"], a["w"], a["a"], a["b"], a["ids"], a["scales"], out=over.get("out"))


BIG = 2 ** 32 + 64

REFUSED = {
    "route type": (TypeError, lambda: g.moe_route(T(8, 16, dtype=torch.int32), 2)),
    "route host": (TypeError, lambda: g.moe_route(torch.zeros(8, 16), 2)),
    "route dimensions": (ValueError, lambda: g.moe_route(T(8, 4, 4), 2)),
    "route columns": (ValueError, lambda: g.moe_route(T(8, 16, strides=(1, 8)), 2)),
    "route score": (ValueError, lambda: g.moe_route(T(8, 16), 2, score="relu")),
    "route group score": (ValueError, lambda: g.moe_route(T(8, 16), 2, groups=2, group_score="mean")),
    "route top": (ValueError, lambda: g.moe_route(T(8, 16), -1)),
    "route top past 32 bits": (ValueError, lambda: g.moe_route(T(8, 16), BIG)),
    "route groups past 32 bits": (ValueError, lambda: g.moe_route(T(8, 16), 2, groups=BIG)),
    "route pitch past 32 bits": (ValueError, lambda: g.moe_route(T(8, 16, strides=(BIG, 1)), 2)),
    "route bias type": (TypeError, lambda: g.moe_route(T(8, 16), 2, bias=T(16))),
    "route bias size": (ValueError, lambda: g.moe_route(T(8, 16), 2, bias=T(15, dtype=F32))),
    "unroute gates": (TypeError, lambda: g.moe_route_backward(T(8, 2), T(8, 16), T(8, 2, dtype=I32))),
    "unroute ids": (TypeError, lambda: g.moe_route_backward(T(8, 2, dtype=F32), T(8, 16), T(8, 2, dtype=torch.int64))),
    "unroute shapes": (ValueError, lambda: g.moe_route_backward(T(8, 3, dtype=F32), T(8, 16), T(8, 2, dtype=I32))),
    "unroute rows": (ValueError, lambda: g.moe_route_backward(T(7, 2, dtype=F32), T(8, 16), T(7, 2, dtype=I32))),
    "unroute out": (TypeError, lambda: g.moe_route_backward(T(8, 2, dtype=F32), T(8, 16), T(8, 2, dtype=I32), out=T(8, 16, dtype=F32))),
    "experts type": (TypeError, lambda: _experts(x=T(8, 64, dtype=F32))),
    "experts ids type": (TypeError, lambda: _experts(ids=T(8, 2, dtype=torch.int64))),
    "experts ids strides": (TypeError, lambda: _experts(ids=T(8, 2, dtype=I32, strides=(4, 1)))),
    "experts ids rows": (ValueError, lambda: _experts(ids=T(7, 2, dtype=I32), gates=T(7, 2, dtype=F32))),
    "experts gates type": (TypeError, lambda: _experts(gates=T(8, 2))),
    "experts gates shape": (ValueError, lambda: _experts(gates=T(8, 3, dtype=F32))),
    "experts w1 type": (TypeError, lambda: _experts(w1=T(4, 96, 64, dtype=torch.float16))),
    "experts w1 rows": (ValueError, lambda: _experts(w1=T(4, 95, 64))),
    "experts w1 width": (ValueError, lambda: _experts(w1=T(4, 96, 63))),
    "experts w1 experts": (ValueError, lambda: _experts(w1=T(5, 96, 64))),
    "experts w2 dimensions": (ValueError, lambda: _experts(w2=T(64, 48))),
    "experts w2 gaps": (ValueError, lambda: _experts(w2=T(4, 64, 48, strides=(64 * 48 + 8, 48, 1)))),
    "experts one MX": (TypeError, lambda: _experts(w2=MX((4, 64), 48))),
    "experts MX save": (ValueError, lambda: _experts(save=True, w1=MX((4, 96), 64), w2=MX((4, 64), 48))),
    "experts MX tokens": (ValueError, lambda: _experts(x=T(257, 64), ids=T(257, 2, dtype=I32), gates=T(257, 2, dtype=F32),
                                                       w1=MX((4, 96), 64), w2=MX((4, 64), 48))),
    "experts top": (ValueError, lambda: _experts(ids=T(8, 17, dtype=I32), gates=T(8, 17, dtype=F32))),
    "experts count": (ValueError, lambda: _experts(w1=T(513, 96, 64), w2=T(513, 64, 48))),
    "experts out": (TypeError, lambda: _experts(out=T(8, 64, dtype=F32))),
    "experts workspace": (TypeError, lambda: _experts(workspace=torch.zeros(16, dtype=torch.uint8))),
    "experts pitch past 32 bits": (ValueError, lambda: _experts(x=T(8, 64, strides=(BIG, 1)))),
    "backward MX": (TypeError, lambda: _backward(w1=MX((4, 96), 64), w2=MX((4, 64), 48))),
    "backward dy": (TypeError, lambda: _backward(dy=T(8, 63))),
    "backward dy type": (TypeError, lambda: _backward(dy=T(8, 64, dtype=F32))),
    "backward saved": (TypeError, lambda: _backward(saved=T(16, 95, dtype=F32))),
    "backward saved type": (TypeError, lambda: _backward(saved=T(16, 96))),
    "adapters type": (TypeError, lambda: _adapters(x=T(8, 64, dtype=F32))),
    "adapters w type": (TypeError, lambda: _adapters(w=T(32, 64, dtype=torch.float16))),
    "adapters w width": (ValueError, lambda: _adapters(w=T(32, 63))),
    "adapters a dimensions": (ValueError, lambda: _adapters(a=T(48, 64))),
    "adapters a width": (ValueError, lambda: _adapters(a=T(3, 16, 63))),
    "adapters b rank": (ValueError, lambda: _adapters(b=T(3, 32, 15))),
    "adapters b rows": (ValueError, lambda: _adapters(b=T(3, 31, 16))),
    "adapters b type": (TypeError, lambda: _adapters(b=T(3, 32, 16, dtype=torch.float16))),
    "adapters MX": (TypeError, lambda: _adapters(a=MX((3, 16), 64))),
    "adapters ids": (TypeError, lambda: _adapters(ids=T(8, dtype=torch.int64))),
    "adapters ids size": (ValueError, lambda: _adapters(ids=T(7, dtype=I32))),
    "adapters scales": (TypeError, lambda: _adapters(scales=T(3))),
    "adapters scales size": (ValueError, lambda: _adapters(scales=T(2, dtype=F32))),
    "adapters count": (ValueError, lambda: _adapters(a=T(512, 16, 64), b=T(512, 32, 16), scales=None)),
    "adapters rank": (ValueError, lambda: _adapters(a=T(3, 513, 64), b=T(3, 32, 513))),
    "adapters out": (TypeError, lambda: _adapters(out=T(8, 33))),
    "adapters pitch past 32 bits": (ValueError, lambda: _adapters(w=T(32, 64, strides=(BIG, 1)))),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused(launched, name):
    kind, call = REFUSED[name]
    with pytest.raises(kind):
        call()
    assert not launched


def test_accepted(launched):
    g.moe_route(T(8, 16), 2, bias=T(16, dtype=F32), groups=4, top_groups=2, group_score="top2", score="sigmoid")
    g.moe_route_backward(T(8, 2, dtype=F32), T(8, 16), T(8, 2, dtype=I32))
    assert _experts().shape == (8, 64)
    y, saved = _experts(save=True)
    assert saved.shape == (16, 96) and saved.dtype == F32
    _experts(w1=MX((4, 96), 64), w2=MX((4, 64), 48))
    assert [tuple(t.shape) for t in _backward()] == [(8, 64), (8, 2), (4, 96, 64), (4, 64, 48)]
    assert _adapters().shape == (8, 32)
    _adapters(scales=None)
    assert len(launched) == 8


# ---- the C interface's own checks -------------------------------------------------------------

P = 256  # a pointer that is never followed: every call here is refused before that


def _raw(fn, base, **over):
    a = dict(base)
    assert set(over) <= set(a)
    a.update(over)
    return getattr(g._lib, fn)(*a.values())


ROUTE = dict(T=4, E=8, top=2, Z=P, ldz=8, format=2, score=0, bias=None, groups=2, top_groups=1, group_score=0, renormalize=1, scale=1.0, ids=P,
             gates=P, stream=None)
UNROUTE = dict(T=4, E=8, top=2, dgates=P, Z=P, ldz=8, format=0, score=1, renormalize=0, scale=1.0, ids=P, dZ=P, lddz=8, stream=None)
EXPERTS = dict(T=4, E=3, top=2, H=16, I=8, X=P, ldx=16, ids=P, gates=P, format=0, W1=P, ld1=16, S1=None, lds1=0, W2=P, ld2=8, S2=None, lds2=0,
               weights=0, Y=P, ldy=16, saved=None, workspace=P, bytes=1 << 20, stream=None)
BACKWARD = dict(T=4, E=3, top=2, H=16, I=8, dY=P, lddy=16, X=P, ldx=16, ids=P, gates=P, format=0, W1=P, ld1=16, W2=P, ld2=8, saved=P, dX=P, lddx=16,
                dgates=P, dW1=P, lddw1=16, dW2=P, lddw2=8, workspace=P, bytes=1 << 20, stream=None)
ADAPTERS = dict(T=4, N=8, K=16, R=4, count=3, X=P, ldx=16, W=P, ldw=16, A=P, lda=16, B=P, ldb=4, ids=P, scales=None, format=0, Y=P, ldy=8,
                workspace=P, bytes=1 << 20, stream=None)
INVALID_DIM, INVALID_LD, NULL_PTR, MISALIGNED, BAD_ARG, BAD_WORKSPACE = 1, 2, 3, 6, 8, 9

RAW = [
    ("gemm_moe_route", ROUTE, [(dict(T=-1), INVALID_DIM), (dict(T=(1 << 22) + 1), BAD_ARG), (dict(E=513, ldz=513, groups=1), BAD_ARG),
                               (dict(top=0), BAD_ARG), (dict(top=9), BAD_ARG), (dict(top=5), BAD_ARG), (dict(groups=3), BAD_ARG),
                               (dict(groups=0), BAD_ARG), (dict(top_groups=3), BAD_ARG), (dict(top_groups=0), BAD_ARG), (dict(ldz=7), INVALID_LD),
                               (dict(format=3), BAD_ARG), (dict(score=2), BAD_ARG), (dict(group_score=2), BAD_ARG),
                               (dict(scale=float("inf")), BAD_ARG), (dict(scale=float("nan")), BAD_ARG), (dict(Z=None), NULL_PTR),
                               (dict(Z=P + 2), MISALIGNED), (dict(bias=P + 1), MISALIGNED), (dict(ids=None), NULL_PTR), (dict(gates=P + 2), MISALIGNED),
                               (dict(T=0, Z=None, ids=None, gates=None), 0)]),
    ("gemm_moe_route_backward", UNROUTE, [(dict(T=-1), INVALID_DIM), (dict(top=9), BAD_ARG), (dict(ldz=7), INVALID_LD), (dict(lddz=7), INVALID_LD),
                                          (dict(format=-1), BAD_ARG), (dict(score=-1), BAD_ARG), (dict(scale=float("nan")), BAD_ARG),
                                          (dict(dgates=None), NULL_PTR), (dict(Z=P + 1), MISALIGNED), (dict(ids=None), NULL_PTR),
                                          (dict(dZ=None), NULL_PTR), (dict(T=0, Z=None, dZ=None, ids=None, dgates=None), 0)]),
    ("gemm_experts", EXPERTS, [(dict(T=-1), INVALID_DIM), (dict(H=0), INVALID_DIM), (dict(I=0), INVALID_DIM), (dict(E=0), BAD_ARG), (dict(E=513), BAD_ARG),
                               (dict(top=17), BAD_ARG), (dict(T=(1 << 22) + 1), BAD_ARG), (dict(H=(1 << 17) + 1, ldx=1 << 18, ldy=1 << 18, ld1=1 << 18), BAD_ARG),
                               (dict(format=2), BAD_ARG), (dict(weights=2), BAD_ARG), (dict(weights=1, saved=P), BAD_ARG), (dict(weights=1, T=257), BAD_ARG),
                               (dict(ldx=15), INVALID_LD), (dict(ldy=15), INVALID_LD), (dict(ld1=15), INVALID_LD), (dict(ld2=7), INVALID_LD),
                               (dict(weights=1, ld1=16, lds1=16, ld2=8, lds2=16), INVALID_LD), (dict(X=None), NULL_PTR), (dict(X=P + 1), MISALIGNED),
                               (dict(ids=None), NULL_PTR), (dict(ids=P + 2), MISALIGNED), (dict(gates=None), NULL_PTR), (dict(W1=None), NULL_PTR),
                               (dict(W2=P + 1), MISALIGNED), (dict(Y=None), NULL_PTR), (dict(saved=P + 2), MISALIGNED), (dict(workspace=None), BAD_WORKSPACE),
                               (dict(workspace=P + 8), BAD_WORKSPACE), (dict(bytes=64), BAD_WORKSPACE), (dict(T=0, X=None, workspace=None), 0)]),
    ("gemm_experts_backward", BACKWARD, [(dict(T=-1), INVALID_DIM), (dict(E=0), BAD_ARG), (dict(format=2), BAD_ARG), (dict(lddy=15), INVALID_LD),
                                         (dict(lddx=15), INVALID_LD), (dict(lddw1=15), INVALID_LD), (dict(lddw2=7), INVALID_LD), (dict(dY=None), NULL_PTR),
                                         (dict(saved=None), NULL_PTR), (dict(X=P + 1), MISALIGNED), (dict(dX=P + 1), MISALIGNED),
                                         (dict(dgates=P + 2), MISALIGNED), (dict(dW1=P + 1), MISALIGNED), (dict(dW2=P + 1), MISALIGNED),
                                         (dict(workspace=None), BAD_WORKSPACE), (dict(bytes=64), BAD_WORKSPACE)]),
    ("gemm_adapters", ADAPTERS, [(dict(T=-1), INVALID_DIM), (dict(N=0), INVALID_DIM), (dict(K=0), INVALID_DIM), (dict(R=0), INVALID_DIM),
                                 (dict(count=-1), INVALID_DIM), (dict(count=512), BAD_ARG), (dict(R=513, ldb=513), BAD_ARG), (dict(T=(1 << 22) + 1), BAD_ARG),
                                 (dict(format=2), BAD_ARG), (dict(ldx=15), INVALID_LD), (dict(ldw=15), INVALID_LD), (dict(lda=15), INVALID_LD),
                                 (dict(ldb=3), INVALID_LD), (dict(ldy=7), INVALID_LD), (dict(X=None), NULL_PTR), (dict(W=P + 1), MISALIGNED),
                                 (dict(A=None), NULL_PTR), (dict(B=P + 1), MISALIGNED), (dict(ids=None), NULL_PTR), (dict(scales=P + 2), MISALIGNED),
                                 (dict(Y=None), NULL_PTR), (dict(workspace=None), BAD_WORKSPACE), (dict(workspace=P + 8), BAD_WORKSPACE),
                                 (dict(bytes=16), BAD_WORKSPACE), (dict(T=0, X=None, workspace=None), 0)]),
]


@pytest.mark.parametrize("fn,base,cases", RAW, ids=[r[0] for r in RAW])
def test_status_before_any_gpu_call(fn, base, cases):
    for over, want in cases:
        assert _raw(fn, base, **over) == want, (fn, over)


def test_workspace_bytes():
    for args in ((4, 8, 2, 64, 32), (4096, 64, 4, 2048, 1024), (1 << 22, 512, 16, 1 << 17, 1 << 17)):
        forward, backward = (g.gemm_experts_workspace_bytes(*args, b) for b in (0, 1))
        pairs = args[0] * args[2]
        assert forward >= 2 * pairs * args[4] + 4 * pairs * args[3] and backward >= forward + 4 * pairs * args[4]
    assert g.gemm_experts_workspace_bytes(4, 0, 1, 8, 8) == -1 and g.gemm_experts_workspace_bytes(-1, 2, 1, 8, 8) == -1
    assert g.gemm_adapters_workspace_bytes(5, 64, 64, 8, 512) == -1 and g.gemm_adapters_workspace_bytes(5, 64, 64, 8, 511) >= 2 * 5 * 8
    for call in (lambda: g.gemm_experts_workspace_bytes(BIG, 4, 2, 64, 32), lambda: g.gemm_adapters_workspace_bytes(5, BIG, 64, 8, 3),
                 lambda: g.gemm_moe_route(0, BIG, 2, P, 8, "f32", "softmax", 0, 1, 1, "max", 1, 1.0, P, P),
                 lambda: g.gemm_moe_route_backward(0, 8, 2, P, P, BIG, "f32", "softmax", 1, 1.0, P, P, 8),
                 lambda: g.gemm_experts(0, 4, 2, 64, 32, P, BIG, P, P, "bf16", P, 64, 0, 0, P, 32, 0, 0, "w16", P, 64, 0, P, 1),
                 lambda: g.gemm_experts_backward(0, 4, 2, 64, 32, P, 64, P, 64, P, P, "bf16", P, BIG, P, 32, P, P, 64, P, P, 64, P, 32, P, 1),
                 lambda: g.gemm_adapters(0, 4, 4, 4, BIG, P, 4, P, 4, P, 4, P, 4, P, 0, "bf16", P, 4, P, 1)):
        with pytest.raises(ValueError):
            call()


# ---- whose tensors ------------------------------------------------------------------------------

@pytest.fixture
def taken(monkeypatch):
    """Streams of the tensors made, under stubs."""
    now, made = [CURRENT], []
    plain = torch.empty

    def empty(*shape, dtype=torch.float32, device=None):
        made.append(now[-1])
        return plain(*shape, dtype=dtype, device="meta").as_subclass(OnDevice)

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
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: now[-1], raising=False)
    monkeypatch.setattr(g, "_launch", lambda *args: None)
    return made


def test_tensors_belong_to_the_stream(taken):
    a = _args()
    calls = {
        2: lambda s: g.moe_route(T(8, 16), 2, stream=s),
        1: lambda s: g.moe_route_backward(T(8, 2, dtype=F32), T(8, 16), T(8, 2, dtype=I32), stream=s),
        3: lambda s: g.moe_experts(a["x"], a["ids"], a["gates"], a["w1"], a["w2"], save=True, stream=s),
        5: lambda s: g.moe_experts_backward(T(8, 64), a["x"], a["ids"], a["gates"], a["w1"], a["w2"], T(16, 96, dtype=F32), stream=s),
    }
    adapters = lambda s: g.matmul_adapters(T(8, 64), T(32, 64), T(3, 16, 64), T(3, 32, 16), T(8, dtype=I32), stream=s)  # noqa: E731
    for want, call in [*calls.items(), (2, adapters)]:
        for stream, owner in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE), (0, 0)):
            taken.clear()
            call(stream)
            assert taken == [owner] * want, (want, stream, taken)


def test_bounds_of_the_headers():
    """The refusals above use the headers' bounds."""
    import os
    import re
    text = "".join(open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", n)).read()
                   for n in ("gemm_route.h", "gemm_experts.h", "gemm_adapters.h"))
    found = dict(re.findall(r"#define (GEMM_\w+_MAX_\w+) (.+)", text))
    assert found["GEMM_ROUTE_MAX_TOKENS"] == found["GEMM_EXPERTS_MAX_TOKENS"] == found["GEMM_ADAPTERS_MAX_ROWS"] == "(1 << 22)"
    assert found["GEMM_ADAPTERS_MAX_COUNT"] == "511" and found["GEMM_ADAPTERS_MAX_RANK"] == "512"
    assert ctypes.sizeof(ctypes.c_int) == 4
