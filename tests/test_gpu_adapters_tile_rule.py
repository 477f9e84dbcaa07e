"""Adapters of many rows on both sides of the rule by which tiles are 256 x 256: tiles of 128
that fit the chip at once, more than that, and wide tiles that would be mostly empty."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_adapters as adapters  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# (the last two: rows that are not loaded directly)
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(2048, 4096, 1032, 24, 9), (700, 10_900, 2056, 16, 5), (2150, 4100, 264, 40, 30), (20_000, 300, 128, 16, 5), (20_000, 390, 128, 16, 5),
                                  (66_000, 100, 72, 8, 3), (2150, 4100, 1025, 9, 3), (20_001, 390, 67, 16, 5)])
def test_tiles(g, case, fmt):
    print(f"case: adapters tile rule {case} {fmt}", flush=True)
    args = adapters._make(*case, adapters.DT[fmt])
    adapters.check(g.matmul_adapters(*args), adapters.reference(*args), (case, fmt))
