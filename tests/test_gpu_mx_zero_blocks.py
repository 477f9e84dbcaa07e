"""Blocks of zeros among the weights, under the scale byte that mx_quantize gives them
(0) and any other: they add exact zeros, and NaN under 255.  The rest is small
integers, so results are exact; and quantised weights with columns of zeros.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_mx import DT, _dev, _host, _mx, check_product  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# The small form, whole pieces and K's end; the wide form.
@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("byte", [0, 1, 90, 200, 252, 253, 254])
@pytest.mark.parametrize("shape", [(2, 40, 1024), (20, 70, 1601), (40, 6145, 1601), (70, 6145, 1024)])
def test_a16(g, shape, byte, af):
    M, N, K = shape
    rng = np.random.default_rng(byte + M)
    a = torch.from_numpy(rng.integers(-4, 5, (M, K)).astype(np.float32)).to(DT[af])
    b, sb = mx.random_rows(rng, N, K, 127, 128, pad=255)
    nb = -(-K // 32)
    zero = rng.random((N, nb)) < 1 / 8
    b.reshape(N, nb, 16)[zero] = 0
    sb[:, :nb][zero] = byte
    bv = mx.values(b, sb, K)
    assert (np.abs(bv) <= 6).all()
    got = _host(g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K)))
    # halves of at most 24 K: exact
    assert np.array_equal(got, (a.float().numpy() @ bv.T.astype(np.float32)))
    sb[N - 1, 1], b[N - 1, 16:32] = 255, 0
    sb[0, 0], b[0, :16] = 255, 0
    got = _host(g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K)))
    assert np.isnan(got[:, [0, N - 1]]).all() and np.isfinite(got[:, 1:N - 1]).all()


@pytest.mark.parametrize("af", ["bf16", "f16"])
def test_quantised_weights_with_zeros(g, af):
    M, N, K = 5, 300, 1700
    rng = np.random.default_rng(4)
    w = rng.standard_normal((N, K)).astype(np.float32)
    w[:, 640:704] = 0.0
    w[7] = 0.0
    q = g.mx_quantize(torch.from_numpy(w).to(_dev()))
    assert bool((q.scales[:, 20:22] == 0).all())
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DT[af])
    y = g.matmul_mx(x.to(_dev()), q)
    check_product(y, x.double().numpy(), _host(g.mx_dequantize(q)), "f32", af)
    assert bool((y[:, 7] == 0).all())


@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("byte", [0, 1, 2, 103, 104, 140, 141, 252])
@pytest.mark.parametrize("shape", [(2, 40, 1024), (40, 6145, 1024)])
def test_every_element_at_the_conversions_borders(g, shape, byte, af):
    """Where the weights are widened by one conversion, and just past it: a row of
    all elements under one byte, against powers of two.  Exact."""
    M, N, K = shape
    rng = np.random.default_rng(byte)
    b, sb = mx.random_rows(rng, N, K, byte, byte + 1, pad=255)
    bv = mx.values(b, sb, K)
    # sums of K multiples of 2^(byte - 128) of at most 6 2^(byte - 127): exact, after a
    # factor that keeps them within fp32's normal numbers (or its range)
    a = np.full((M, K), 2.0 ** (15 if byte < 128 else -15))
    got = _host(g.matmul_mx(torch.from_numpy(a).to(_dev(), DT[af]), _mx(g, b, sb, K)))
    assert np.array_equal(got, a @ bv.T)


@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("byte", [0, 1, 103, 141, 252])
def test_layer_at_the_conversions_borders(g, byte, af):
    """W2 under one byte, one token and several, against the layer's bars."""
    from test_gpu_moe import _check, _layer, _make, _on_gpu

    for T, E, top, H, I in ((1, 3, 2, 512, 1024), (20, 3, 2, 100, 600)):
        rng = np.random.default_rng(byte + T)
        x, r, w1, w2 = _make(rng, T, E, H, I, af, "mx")
        c2, s2 = w2[0], w2[1].copy()
        s2[:, :-(-I // 32)] = byte
        c2.reshape(E * H, -1, 16)[:, 1] = 0
        w2 = c2, s2, mx.values(c2, s2, I).reshape(E, H, I)
        g1, g2, v1, v2 = _on_gpu(g, w1, w2, E, H, I)
        if byte > 200:  # sums are held in fp32: small inner values
            x = x * 2.0 ** -8
            r = r * 2.0 ** 6
        ref, bar, ids, _ = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
        y, gi, _ = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
        assert np.array_equal(gi.cpu().numpy(), ids)
        got = _host(y)
        # sums below fp32's normal numbers are rounded to its smallest step, 2^-149
        limit = bar + 2.0 ** -24 * np.abs(ref) + 2.0 ** -149 * I * top
        assert (np.abs(got - ref) <= limit).all(), (byte, T)
