"""The MX binding refuses wrong types and sizes before anything is launched (no GPU
needed)."""
import pytest

import tiled_fp32_gemm_03_amd as g

torch = pytest.importorskip("torch")


def test_dequantize_takes_an_mx_tensor_only():
    for bad in (torch.zeros(3, 64), None, [1.0], torch.zeros(3, 32, dtype=torch.uint8)):
        with pytest.raises(TypeError):
            g.mx_dequantize(bad)
