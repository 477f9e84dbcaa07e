"""Many rows: the experts' products and adapters where sizes ask for the large tiles but rows
cannot be loaded directly (widths that are no multiple of 8, a matrix that starts in the middle
of a word, rows of fewer than 8 values), in some of a pass's products or in all; and more pairs
than are listed in one launch."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_adapters as adapters  # noqa: E402
import test_gpu_experts as experts  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# widths odd both, H whole 16 bytes alone, I alone, both
@pytest.mark.parametrize("case", [(3001, 4, 2, 2051, 1025), (3001, 4, 2, 2056, 1026), (3001, 4, 2, 2050, 1032), (3001, 4, 2, 2056, 1032)])
def test_experts_of_many_rows(g, case):
    print(f"case: experts {case}", flush=True)
    experts._all(g, experts._make(*case, torch.bfloat16), case)


@pytest.mark.parametrize("case", [(4000, 3333, 131, 9, 5), (4000, 3336, 5, 3, 40), (3300, 4001, 520, 24, 3)])
def test_adapters_of_many_rows(g, case):
    print(f"case: adapters {case}", flush=True)
    args = adapters._make(*case, torch.bfloat16)
    ref = adapters.reference(*args)
    adapters.check(g.matmul_adapters(*args), ref, case)
    x, w, a, b, ids, scales = args
    wide = torch.zeros(x.shape[0], x.shape[1] + 3, dtype=x.dtype, device=x.device)
    wide[:, 1:-2] = x
    adapters.check(g.matmul_adapters(wide[:, 1:-2], w, a, b, ids, scales), ref, (case, "in the middle of a word"))


@pytest.mark.parametrize("case", [(22_000, 5, 3, 40, 24), (70_000, 512, 1, 24, 8), (65_537, 1, 1, 8, 9)])
def test_experts_of_more_pairs_than_one_launch_lists(g, case):
    print(f"case: experts {case}", flush=True)
    experts._all(g, experts._make(*case, torch.float16, drop=0.1), case)


@pytest.mark.parametrize("case", [(65_536, 24, 32, 8, 7), (70_001, 40, 24, 5, 300)])
def test_adapters_of_more_rows_than_one_launch_lists(g, case):
    print(f"case: adapters {case}", flush=True)
    args = adapters._make(*case, torch.float16)
    adapters.check(g.matmul_adapters(*args), adapters.reference(*args), case)
