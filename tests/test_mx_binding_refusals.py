"""The MX binding refuses wrong types and sizes before anything is launched (no GPU
needed)."""
import pytest

import tiled_fp32_gemm_03_amd as g

torch = pytest.importorskip("torch")


def test_dequantize_takes_an_mx_tensor_only():
    for bad in (torch.zeros(3, 64), None, [1.0], torch.zeros(3, 32, dtype=torch.uint8)):
        with pytest.raises(TypeError):
            g.mx_dequantize(bad)


# ---- sizes past the C ABI's int -----------------------------------------------------------


class OnDevice(torch.Tensor):
    """A tensor without memory that says that it is on the device."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))
    data_ptr = lambda self: 256  # noqa: E731


def _rows(rows, width, dtype=torch.bfloat16, pitch=None):
    t = torch.empty_strided((rows, width), (width if pitch is None else pitch, 1), dtype=dtype, device="meta")
    return t.as_subclass(OnDevice)


def _mx(rows, K, pitch=None, scale_pitch=None):
    return g.MxTensor(_rows(rows, (K + 31) // 32 * 16, torch.uint8, pitch),
                      _rows(rows, (K + 511) // 512 * 16, torch.uint8, scale_pitch), K)


BIG = 2 ** 32 + 32  # 32, if it were cut to 32 bits


@pytest.fixture
def launched(monkeypatch):
    calls = []
    monkeypatch.setattr(g, "_launch", lambda *args: calls.append(args))
    plain = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None:
                        plain(*shape, dtype=dtype, device="meta").as_subclass(OnDevice))
    return calls


def _calls():
    x, q = _rows(8, 64), _mx(8, 64)
    f = torch.float32
    r, w1, w2 = _rows(4, 64), (4, 64, 64), (4, 64, 32)
    meta = lambda shape: torch.empty(shape, dtype=torch.bfloat16, device="meta").as_subclass(OnDevice)  # noqa: E731
    w1, w2 = meta(w1), meta(w2)
    return {
        "quantize rows": lambda: g.mx_quantize(_rows(BIG, 64)),
        "quantize K": lambda: g.mx_quantize(_rows(2, BIG)),
        "quantize pitch": lambda: g.mx_quantize(_rows(2, 64, pitch=BIG * 2)),
        "quantize code pitch": lambda: g.mx_quantize(x, out=_mx(8, 64, pitch=BIG)),
        "quantize scale pitch": lambda: g.mx_quantize(x, out=_mx(8, 64, scale_pitch=BIG)),
        "quantize columns": lambda: g.mx_quantize(_rows(64, BIG), along="columns"),
        "dequantize rows": lambda: g.mx_dequantize(_mx(BIG, 64)),
        "dequantize K": lambda: g.mx_dequantize(_mx(2, BIG)),
        "dequantize pitch": lambda: g.mx_dequantize(q, out=_rows(8, 64, f, pitch=BIG * 2)),
        "product rows": lambda: g.matmul_mx(_mx(BIG, 64), q),
        "product columns": lambda: g.matmul_mx(q, _mx(BIG, 64)),
        "product K": lambda: g.matmul_mx(_mx(2, BIG), _mx(3, BIG)),
        "product pitch of A": lambda: g.matmul_mx(_mx(8, 64, pitch=BIG), q),
        "product scale pitch of B": lambda: g.matmul_mx(q, _mx(8, 64, scale_pitch=BIG)),
        "product pitch of C": lambda: g.matmul_mx(q, q, out=_rows(8, 8, f, pitch=BIG)),
        "rows of 16 bits": lambda: g.matmul_mx(_rows(BIG, 64), q),
        "pitch of 16-bit rows": lambda: g.matmul_mx(_rows(8, 64, pitch=2 * BIG), q),
        "layer tokens": lambda: g.moe_layer(_rows(BIG, 64), r, w1, w2, 2),
        "layer top": lambda: g.moe_layer(x, r, w1, w2, 2 ** 32 + 2),
        "layer pitch": lambda: g.moe_layer(_rows(8, 64, pitch=2 * BIG), r, w1, w2, 2),
        "layer weights' pitch": lambda: g.moe_layer(
            x, r, torch.empty_strided((4, 64, 64), (128 * BIG, 2 * BIG, 1), dtype=torch.bfloat16,
                                      device="meta").as_subclass(OnDevice), w2, 2),
        "layer out pitch": lambda: g.moe_layer(x, r, w1, w2, 2, out=_rows(8, 64, pitch=2 * BIG)),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_sizes_past_32_bits_are_refused(launched, name):
    """They would reach the library cut to their low 32 bits."""
    with pytest.raises(ValueError):
        _calls()[name]()
    assert not launched


def test_sizes_within_32_bits_are_not(launched):
    x, q = _rows(8, 64), _mx(8, 64)
    g.mx_quantize(_rows(2 ** 31 - 1, 32))
    g.mx_dequantize(q)
    g.matmul_mx(q, _mx(2 ** 31 - 1, 64), out=_rows(8, 2 ** 31 - 1, torch.float32))
    g.matmul_mx(x, q)
    g.mx_quantize(x, out=_mx(8, 64, pitch=2 ** 31 - 16, scale_pitch=2 ** 31 - 16))
    assert len(launched) == 5


def test_raw_calls_refuse_them_too():
    p = 256
    for call in (lambda: g.gemm_mx_code_bytes(BIG), lambda: g.gemm_mx_scale_bytes(BIG),
                 lambda: g.gemm_mx_quantize(BIG, 64, p, 64, "bf16", "rows", p, 32, p, 16),
                 lambda: g.gemm_mx_dequantize(0, BIG, p, 32, p, 16, p, 64, "bf16", "rows"),
                 lambda: g.gemm_mx(0, 4, 64, p, BIG, p, 16, p, 32, p, 16, p, 4, "f32"),
                 lambda: g.gemm_mx_a16(0, 4, 64, p, 64, "bf16", p, 32, p, BIG, p, 4, "f32"),
                 lambda: g.gemm_mx_tile(-1, BIG, 4, 64), lambda: g.gemm_mx_tile(2 ** 32 - 1, 4, 4, 64),
                 lambda: g.gemm_moe_workspace_bytes(BIG, 4, 2, 64, 32),
                 lambda: g.gemm_moe(0, 4, 2, 64, 32, p, BIG, p, 64, "bf16", p, 64, 0, 0, p, 32, 0, 0, "w16",
                                    True, p, 64, "bf16", 0, 0, p, 1 << 20)):
        with pytest.raises(ValueError):
            call()
