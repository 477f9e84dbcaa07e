"""More columns than one grid takes (2^32 threads in x): products with 2^27 to 2^30
rows of MX weights, and a conversion of 2^31 - 1 columns.  The weights repeat a few
rows of small integers, so every result is exact and known.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_mx import _dev, _mx  # noqa: E402

PERIOD = 1021  # prime: no column tile sees the same rows


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _many(g, N, K):
    rng = np.random.default_rng(K)
    c, s = mx.random_rows(rng, PERIOD, K, 127, 128)
    q = _mx(g, c, s, K)
    times = -(-N // PERIOD)
    return g.MxTensor(q.codes.repeat(times, 1)[:N], q.scales.repeat(times, 1)[:N], K), mx.values(c, s, K)


def _check(got, ref, N):
    """Rows of ref (M x PERIOD) repeated along N."""
    want = torch.from_numpy(ref).to(got.device, got.dtype)
    whole = N // PERIOD * PERIOD
    assert torch.equal(got[:, :whole].unflatten(1, (-1, PERIOD)), want[:, None].expand(-1, N // PERIOD, -1))
    assert torch.equal(got[:, whole:], want[:, :N - whole])


# (entry, M, N, K): gemm_mx's few-row form and its entry 0 (64 columns a workgroup).
@pytest.mark.parametrize("entry,M,N", [(3, 1, 2 ** 28 + 40), (0, 2, 2 ** 30 + 65)])
def test_product(g, entry, M, N):
    K = 32
    b, bv = _many(g, N, K)
    rng = np.random.default_rng(M)
    a, sa = mx.random_rows(rng, M, K, 127, 128)
    got = g.matmul_mx(_mx(g, a, sa, K), b, dtype=torch.float32, config=entry)
    _check(got, mx.values(a, sa, K) @ bv.T, N)


# The wide form, and the small one, which takes K < 8.
@pytest.mark.parametrize("M,N,K", [(2, 2 ** 28 + 40, 32), (1, 2 ** 27 + 40, 7)])
def test_a16(g, M, N, K):
    b, bv = _many(g, N, K)
    rng = np.random.default_rng(M)
    a = rng.integers(-4, 5, (M, K)).astype(np.float64)
    got = g.matmul_mx(torch.from_numpy(a).to(_dev(), torch.bfloat16), b, dtype=torch.float32)
    _check(got, a @ bv.T, N)


def test_conversion_of_columns(g):
    rows = 2 ** 31 - 1
    x = torch.ones(1, rows, dtype=torch.bfloat16, device=_dev())
    x[0, -3:] = torch.tensor([3.0, -0.5, 0.0])
    q = g.mx_quantize(x, along="columns")
    assert q.shape == (rows, 1)
    # 1 = 4 2^-2: code 6, scale byte 125
    assert bool((q.codes[:-3, 0] == 6).all()) and bool((q.scales[:-3, 0] == 125).all())
    assert q.codes[-3:, 0].tolist() == [7, 14, 0] and q.scales[-3:, 0].tolist() == [126, 124, 0]
    assert bool((q.codes[-4:, 1:] == 0).all()) and bool((q.scales[-4:, 1:] == 0).all())
    assert torch.equal(g.mx_dequantize(q, torch.bfloat16, along="columns"), x)
