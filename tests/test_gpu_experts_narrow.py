"""The experts' products and their gradients where inner widths are below 8 and rows of H are
read by words (H of at least 8, no multiple of 8): values of rows that end before eight."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_experts as experts  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(300, 4, 2, 9, 3), (200, 3, 2, 1001, 7), (700, 5, 2, 131, 1), (40, 3, 2, 12, 5), (513, 2, 1, 260, 2), (65, 1, 1, 15, 6)])
def test_narrow(g, case, fmt):
    print(f"case: experts narrow {case} {fmt}", flush=True)
    experts._all(g, experts._make(*case, experts.DT[fmt]), (case, fmt))
