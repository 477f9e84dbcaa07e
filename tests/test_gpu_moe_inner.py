"""The layer's inner values keep their 32 bits through the second product.

The inputs make everything else exact: one expert, so its gate is 1; gate rows
that give 64, whose silu is 64 (1 + e^-64 rounds to 1); other rows that give
chosen values b of 24 significant bits, as sums of digits with powers of two
(exact in fp32 in any order).  So u = 64 b, and each row of W2 has one value v
in some place: y = u v.

Bars: v = 1 gives y = u, equal.  Otherwise u enters as three terms of 8 bits and
v as one (two of fp16), each product of two terms exact: at most 6 additions, each
off by at most 2^-23 of what was added up so far, which is below (1 + 2^-6) |u v|:
|y - u v| <= 6.1 2^-23 |u v| (two additions, 2.1 2^-23, where v is one term).  Two
terms of 8 bits alone are off by up to 2^-17.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_moe import DT, _dev, _host  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _rows(values, K):
    """MX rows (codes, scales) of values that are elements, scale 1."""
    code = np.argmin(np.abs(np.abs(values)[..., None] - mx.ELEMENTS), -1).astype(np.uint8)
    code |= np.where(values < 0, 8, 0).astype(np.uint8)
    nib = np.zeros((values.shape[0], 2 * mx.code_bytes(K)), np.uint8)
    nib[:, :K] = code
    scales = np.full((values.shape[0], mx.scale_bytes(K)), 127, np.uint8)
    out = nib[:, 0::2] | (nib[:, 1::2] << 4), scales
    assert np.array_equal(mx.values(*out, K), values)
    return out


def _case(rng, T, H, I, weights):
    """x, the other rows and u = 64 b, per token (the digits' places are shifted by
    a power of two that differs between tokens)."""
    digits = 12 if weights == "mx" else 3
    bits = 24 // digits
    d = rng.integers(0, 1 << bits, (I, digits)).astype(np.float64)
    d[:, 0] = rng.integers(1 << (bits - 1), 1 << bits, I)
    d *= rng.choice([-1.0, 1.0], (I, 1))
    x = np.zeros((T, H))
    x[:, 0] = 1.0
    shift = np.ldexp(1.0, -rng.integers(0, 3, T))
    x[:, 1:1 + digits] = np.ldexp(1.0, -bits * np.arange(digits)) * shift[:, None]
    other = np.zeros((I, H))
    other[:, 1:1 + digits] = d
    return x, other, 64.0 * (x @ other.T)


def _layer(g, x, other, w2, fmt, weights):
    I, H = other.shape
    gate = np.zeros((I, H))
    gate[:, 0] = 1.0
    x = x.copy()
    x[:, 0] = 64.0
    w1 = np.concatenate([gate, other])
    r = torch.zeros(1, H, dtype=DT[fmt], device=_dev())
    if weights == "mx":
        def stack(q, K):
            return g.MxTensor(*(torch.from_numpy(t).to(_dev())[None] for t in q), K)
        g1, g2 = stack(_rows(w1, H), H), stack(_rows(w2, I), I)
    else:
        g1, g2 = (torch.from_numpy(w).to(DT[fmt]).to(_dev())[None] for w in (w1, w2))
    xt = torch.from_numpy(x).to(DT[fmt])
    assert np.array_equal(xt.double().numpy(), x, equal_nan=True)
    return _host(g.moe_layer(xt.to(_dev()), r, g1, g2, 1, dtype=torch.float32)[0])


# (T, H, I): one token and several, one piece of I and many, odd ends, more columns than I.
SIZES = [(1, 64, 5), (1, 300, 129), (3, 1030, 257), (20, 96, 513), (9, 33, 2050), (2, 16, 7)]


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_inner_values_keep_24_bits(g, size, fmt, weights):
    T, H, I = size
    print(f"case: moe inner {size} {fmt} {weights}", flush=True)
    rng = np.random.default_rng(T + H + I)
    x, other, u = _case(rng, T, H, I, weights)
    assert np.array_equal(u, u.astype(np.float32)) and (np.abs(u) > 0).all()
    at = rng.permutation(max(H, I))[:H] % I
    w2 = np.zeros((H, I))
    w2[np.arange(H), at] = 1.0
    assert np.array_equal(_layer(g, x, other, w2, fmt, weights), u[:, at])
    if weights == "mx":
        v, bar = rng.choice([1.5, 3.0, -6.0, 0.5], H), 2.1 * 2.0 ** -23
    elif fmt == "bf16":
        v, bar = rng.integers(128, 256, H) / 64.0, 2.1 * 2.0 ** -23
    else:
        v, bar = rng.integers(1024, 2048, H) / 512.0, 6.1 * 2.0 ** -23
    w2[np.arange(H), at] = v
    ref = u[:, at] * v
    assert (np.abs(_layer(g, x, other, w2, fmt, weights) - ref) <= bar * np.abs(ref)).all()


@pytest.mark.parametrize("weights", ["w16", "mx"])
def test_inner_values_past_the_range(g, weights):
    """Infinite inner values (from finite tokens) give infinities where I = 1 and W2
    has no zeros, NaN tokens NaN, and neither changes other tokens; the largest
    finite inner values stay finite."""
    rng = np.random.default_rng(3)
    T, H = 6, 40
    x, other, u = _case(rng, T, H, 1, weights)
    other = np.abs(other)
    w2 = rng.choice([1.5, 3.0, -6.0, 0.5], (H, 1))
    clean = _layer(g, x, other, w2, "bf16", weights)
    x[1, 1:4] = 2.0 ** 127
    x[3, 1:4] = -2.0 ** 127
    x[4, 1] = np.nan
    y = _layer(g, x, other, w2, "bf16", weights)
    assert np.array_equal(y[[0, 2, 5]], clean[[0, 2, 5]])
    assert np.array_equal(y[1], np.inf * np.sign(w2[:, 0]))
    assert np.array_equal(y[3], -np.inf * np.sign(w2[:, 0]))
    assert np.isnan(y[4]).all()
    # b = (2 - 2^-7) 2^121 + ..., so u is the largest bf16 value and a bit: two terms'
    # first would round to an infinity.
    other[:] = 0.0
    other[0, 1:4] = 1.0
    x[5, 1:4] = (2 - 2.0 ** -7) * 2.0 ** 121, 2.0 ** 114 * (1 - 2.0 ** -8), 0.0
    w2[:] = 0.5
    want = 32.0 * (x[5, 1] + x[5, 2])
    assert 2 * want > 2.0 ** 128 * (1 - 2.0 ** -9)
    assert np.array_equal(_layer(g, x, other, w2, "bf16", weights)[5], np.full(H, want))
