"""Calls on a stream that is not the current one (``stream=``): equal results while
the current stream is given memory and writes it, which must not be memory of the
call's.  Which stream a call's tensors belong to is checked without a GPU in
test_binding_streams.py.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_moe import DT, _dev, _make, _on_gpu  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _others(nbytes):
    """Memory of the same sizes for the current stream, written there at once."""
    t = [torch.empty(n, dtype=torch.uint8, device=_dev()) for n in nbytes for _ in range(2)]
    for x in t:
        x.fill_(255)
    return {x.untyped_storage().data_ptr() for x in t}, t


def _on(side, call):
    side.wait_stream(torch.cuda.current_stream())
    return call(side.cuda_stream)


@pytest.mark.parametrize("T", [1, 6, 40])
def test_layer_on_another_stream(g, T, monkeypatch):
    E, top, H, I = 16, 4, 256, 96
    x, r, w1, w2 = _make(np.random.default_rng(41), T, E, H, I, "bf16", "mx")
    g1, g2, _, _ = _on_gpu(g, w1, w2, E, H, I)
    x, r = x.to(_dev()), r.to(_dev())
    want = g.moe_layer(x, r, g1, g2, top)
    need = g.gemm_moe_workspace_bytes(T, E, top, H, I)
    used = []
    launch = g._launch
    monkeypatch.setattr(g, "_launch", lambda *a: (used.append(a[4][-2]), launch(*a)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = _on(side, lambda s: g.moe_layer(x, r, g1, g2, top, stream=s))
        taken, keep = _others([need, *(t.numel() * t.element_size() for t in got)])
        assert used[-1] not in taken
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_splitk_on_another_stream(g, monkeypatch):
    gen = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(64, 8192, generator=gen, device=_dev())
    b = torch.randn(8192, 64, generator=gen, device=_dev())
    want = g.matmul_splitk(a, b, splits=8)
    need = g.gemm_f32_splitk_plan(64, 64, 8192, -1, 8)["workspace_bytes"]
    used = []
    call = g.gemm_f32_splitk
    monkeypatch.setattr(g, "gemm_f32_splitk", lambda *p: (used.append(p[11]), call(*p)))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = _on(side, lambda s: g.matmul_splitk(a, b, splits=8, stream=s))
        taken, keep = _others([need, 64 * 64 * 4])
        assert used[-1] not in taken
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)


def test_products_and_conversions_on_another_stream(g):
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(70, 300, generator=gen, device=_dev()).to(DT["bf16"])
    w = g.mx_quantize(torch.randn(90, 300, generator=gen, device=_dev()))
    f = torch.randn(300, 90, generator=gen, device=_dev())

    def calls(s):
        q = g.mx_quantize(x, stream=s)
        return [q.codes, q.scales, g.mx_dequantize(q, torch.bfloat16, stream=s), g.matmul_mx(q, w, stream=s),
                g.matmul_mx(x, w, stream=s), g.matmul(x.float(), f, stream=None),
                g.matmul_mixed(x, f.to(DT["bf16"]), stream=None)]

    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = _on(side, calls)
        _, keep = _others([t.numel() * t.element_size() for t in got])
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):  # the null stream, from another one
        side.synchronize()
        q = g.mx_quantize(x, stream=0)
        y = g.matmul_mx(q, w, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(y, want[3])
