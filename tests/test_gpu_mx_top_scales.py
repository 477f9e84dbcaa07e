"""Weights at the top of the scales' range: bytes 253 and 254 stand for 2^126 and
2^127, so elements of 4 and 6 (and 2 and 3 under 254) are past fp32's and bf16's
largest values, and their products with activations below 1 are not.  (The
product of two MX matrices has them in test_gpu_mx.py.)  The bars are the other
tests': (K + 8) 2^-23 of the sum of magnitudes, and the layer's.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_moe import _check, _layer, _make, _on_gpu  # noqa: E402
from test_gpu_mx import DT, _dev, _host, _mx  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _some_at_the_top(rng, scales, nb, share):
    top = rng.random((scales.shape[0], nb)) < share
    scales[:, :nb] = np.where(top, rng.integers(252, 255, top.shape), scales[:, :nb])
    scales[0, 0] = 254


# The small form (whole pieces, the end of K alone, both), the wide form.
@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(3, 40, 1024), (3, 17, 33), (20, 70, 1601), (40, 6145, 1601)])
def test_a16(g, shape, af):
    M, N, K = shape
    rng = np.random.default_rng(K + M)
    a = rng.standard_normal((M, K)) * 2.0 ** -14
    a[rng.random((M, K)) < 0.2] = 0.0
    a[0] = 0.0
    a = torch.from_numpy(a.astype(np.float32)).to(DT[af])
    b, sb = mx.random_rows(rng, N, K, 100, 140, pad=255)
    _some_at_the_top(rng, sb, -(-K // 32), 0.1)
    av, bv = a.double().numpy(), mx.values(b, sb, K)
    assert (np.abs(bv) >= 2.0 ** 128).any()
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    assert mag.max() < 2.0 ** 127
    got = _host(g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K)))
    assert (np.abs(got - ref) <= (K + 8) * 2.0 ** -23 * mag).all()
    # Infinite and NaN activations, NaN scales.
    a[1, 5], a[M - 1, K - 1] = float("inf"), float("nan")
    b |= np.uint8(0x11)  # no zero elements
    b[:, mx.code_bytes(K) - 16:] &= np.uint8(0x0f) if K % 32 == 1 else np.uint8(0xff)
    b[:, mx.code_bytes(K) - 16 + (K % 32 + 1) // 2 if K % 32 else mx.code_bytes(K):] = 0
    sb[3, 0] = 255
    got = _host(g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K)))
    with np.errstate(invalid="ignore"):
        ref = a.double().numpy() @ mx.values(b, sb, K).T
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)]) and np.isinf(ref).any()
    assert np.isfinite(got[np.isfinite(ref)]).all()


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(1, 4, 2, 64, 40), (9, 4, 2, 600, 1100), (30, 3, 1, 96, 64)])
def test_layer(g, case, fmt):
    """W1's second rows at the top with first ones that make small gates, W2 at the
    bottom; and W2 at the top of small inner values."""
    T, E, top, H, I = case
    rng = np.random.default_rng(T)
    x, r, w1, w2 = _make(rng, T, E, H, I, fmt, "mx")
    # The first product's sums are held in fp32, so they have to stay below 2^128
    # (checked): tokens of about 2^-16.
    x, r = x * 2.0 ** -16, r * 2.0 ** 14
    for up in (True, False):
        c1, s1 = w1[0], w1[1].copy().reshape(E, 2 * I, -1)
        c2, s2 = w2[0], w2[1].copy()
        nb1, nb2 = -(-H // 32), -(-I // 32)
        s1[:, :I, :nb1] -= 40  # a about 2^-56, silu(a) half of it
        if up:
            flat = s1[:, I:].reshape(E * I, -1)
            _some_at_the_top(rng, flat, nb1, 0.2)
            s1[:, I:] = flat.reshape(E, I, -1)
            s2[:, :nb2] -= 90
        else:
            s1[:, I:, :nb1] -= 40
            _some_at_the_top(rng, s2, nb2, 0.2)
        s1 = s1.reshape(E * 2 * I, -1)
        q1 = (c1, s1, mx.values(c1, s1, H).reshape(E, 2 * I, H))
        q2 = (c2, s2, mx.values(c2, s2, I).reshape(E, H, I))
        g1, g2, v1, v2 = _on_gpu(g, q1, q2, E, H, I)
        assert (np.abs(v1 if up else v2) >= 2.0 ** 128).any()
        assert (np.abs(x.double().numpy()) @ np.abs(v1).reshape(-1, H).T).max() < 2.0 ** 127
        ref, bar, ids, _ = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
        y, gi, _ = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
        assert np.array_equal(gi.cpu().numpy(), ids)
        _check(y, ref, bar, "f32", (case, fmt, up))
