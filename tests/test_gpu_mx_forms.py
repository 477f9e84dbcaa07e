"""The forms that gemm_mx, gemm_mx_a16 and gemm_moe take at sizes past the
small ones: wide a16 tiles, rows past whole gemm_mx tiles, experts' products
whose activations come in several tiles, rows of fewer than 8 values.  The bars
are the ones of the operators' other tests: an fp32 sum of K exact products,
(K + 8) 2^-23 of the sum of magnitudes, and the half step of C's format.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_moe import _check, _layer, _make, _on_gpu  # noqa: E402
from test_gpu_mx import DT, _dev, _host, _mx, check_product  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# (M, N, K): wide tiles, with a partial last block of rows, columns and k each.
WIDE = [(17, 6145, 2817), (33, 6200, 1361), (64, 6144, 1536), (130, 2100, 2049), (9, 12289, 1400),
        (7904, 2050, 33), (2080, 2050, 250)]


@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("shape", WIDE)
def test_a16_wide(g, shape, af):
    M, N, K = shape
    print(f"case: a16 wide {af} {shape}", flush=True)
    rng = np.random.default_rng(M + N + K)
    a = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DT[af])
    b, sb = mx.random_rows(rng, N, K, 110, 130, pad=255)
    c = g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K))
    check_product(c, a.double().numpy(), mx.values(b, sb, K), af, (shape, af))


@pytest.mark.parametrize("af", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(40, 6145, 1601), (6, 130, 1601)])
def test_a16_wide_scales_and_special_values(g, shape, af):
    """Scales past what fp16 and bf16 hold, NaN scales, infinite and NaN
    activations, at the wide form's sizes and at the small one's."""
    M, N, K = shape
    rng = np.random.default_rng(K)
    a = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DT[af])
    b, sb = mx.random_rows(rng, N, K, 60, 200)
    b |= np.uint8(0x11)  # no zero elements
    b[:, mx.code_bytes(K) - 16:] &= np.uint8(0x0f) if K % 32 == 1 else np.uint8(0xff)
    b[:, mx.code_bytes(K) - 16 + (K % 32 + 1) // 2:] = 0
    sb[11, 4], sb[N - 1, 50] = 255, 255
    sb[5, :3] = 0
    a[2, 5], a[3, 6], a[M - 1, K - 1] = float("inf"), float("nan"), float("-inf")
    got = _host(g.matmul_mx(a.to(_dev()), _mx(g, b, sb, K), dtype=torch.float32))
    av, bv = a.double().numpy(), mx.values(b, sb, K)
    with np.errstate(invalid="ignore"):
        ref = av @ bv.T
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isinf(got), np.isinf(ref))
    assert (np.sign(got) == np.sign(ref))[np.isinf(ref)].all()
    fine = np.isfinite(ref)
    mag = np.abs(np.where(np.isfinite(av), av, 0)) @ np.abs(np.nan_to_num(bv, nan=0.0)).T
    assert (np.abs(got[fine] - ref[fine]) <= ((K + 8) * 2.0 ** -23 * mag)[fine]).all()


def test_a16_wide_in_a_larger_buffer(g):
    """Odd pitches and starts; what is around C stays; two equal calls agree."""
    M, N, K = 37, 6150, 1601
    rng = np.random.default_rng(8)
    buf = torch.full((1 + M * (K + 2),), float("nan"), dtype=torch.bfloat16, device=_dev())
    a = torch.as_strided(buf, (M, K), (K + 2, 1), 1)
    a.copy_(torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16))
    b, sb = mx.random_rows(rng, N, K, 120, 130, pad=255)
    q = _mx(g, b, sb, K)
    out = torch.full((M + 2, N + 3), 5.0, device=_dev())
    g.matmul_mx(a, q, out=out[1:-1, 1:1 + N])
    check_product(out[1:-1, 1:1 + N], _host(a), mx.values(b, sb, K), "f32", "buffer")
    again = g.matmul_mx(a, q, dtype=torch.float32)
    assert torch.equal(again, out[1:-1, 1:1 + N])
    out[1:-1, 1:1 + N] = 5.0
    assert bool((out == 5.0).all())


@pytest.mark.parametrize("shape", [(4097, 4096, 96), (4128, 4095, 33), (4129, 4096, 64)])
def test_rows_past_whole_tiles(g, shape):
    """Small integers: exact in every format."""
    M, N, K = shape
    rng = np.random.default_rng(M)
    a, sa = mx.random_rows(rng, M, K, 127, 128, pad=255)
    b, sb = mx.random_rows(rng, N, K, 127, 128, pad=255)
    ref = mx.values(a, sa, K) @ mx.values(b, sb, K).T
    out = torch.full((M + 1, N + 5), 3.0, device=_dev())
    g.matmul_mx(_mx(g, a, sa, K), _mx(g, b, sb, K), out=out[:M, 2:2 + N])
    assert np.array_equal(_host(out[:M, 2:2 + N]), ref)
    assert bool((out[M] == 3).all()) and bool((out[:, :2] == 3).all()) and bool((out[:, 2 + N:] == 3).all())


MOE = [(40, 4, 4, 4100, 70), (20, 3, 2, 130, 2101), (64, 8, 2, 2049, 257), (12, 40, 4, 515, 130),
       (1, 64, 8, 2049, 1023), (3, 4, 2, 7, 5), (1, 3, 1, 8, 7), (16, 2, 1, 600, 1999),
       (9, 300, 16, 40, 100)]


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("case", MOE)
def test_layer(g, case, fmt, weights):
    T, E, top, H, I = case
    print(f"case: moe forms {case} {fmt} {weights}", flush=True)
    rng = np.random.default_rng(T + E + H + I)
    x, r, w1, w2 = _make(rng, T, E, H, I, fmt, weights)
    z = -np.sort(-(x.double().numpy() @ r.double().numpy().T), axis=1)
    assert (z[:, :-1] - z[:, 1:]).min() > 1e-11  # the choice does not hang on last bits
    g1, g2, v1, v2 = _on_gpu(g, w1, w2, E, H, I)
    ref, bar, ids, gates = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
    y, gi, gg = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
    assert np.array_equal(gi.cpu().numpy(), ids), case
    assert (np.abs(_host(gg) - gates) <= 2.0 ** -23 * gates).all()
    _check(y, ref, bar, "f32", (case, fmt, weights))


@pytest.mark.parametrize("H,I", [(257, 130), (256, 128)])
def test_layer_with_odd_pitches(g, H, I):
    """Weights and tokens whose rows start in the middle of 4-byte words, between
    NaN paddings, and rows that all do not."""
    T, E, top = 6, 4, 2
    rng = np.random.default_rng(H)
    x, r, w1, w2 = _make(rng, T, E, H, I, "bf16", "w16")

    def padded(t, extra):
        buf = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=_dev())
        buf[..., :t.shape[-1]] = t.to(_dev())
        return buf[..., :t.shape[-1]]

    ref, bar, ids, _ = _layer(x.double().numpy(), r.double().numpy(), w1.double().numpy(),
                              w2.double().numpy(), top, True)
    for extra in ((0, 0, 0), (1, 2, 3), (2, 1, 1), (3, 3, 2)):
        y, gi, _ = g.moe_layer(padded(x, extra[0]), padded(r, extra[1]), padded(w1, extra[2]),
                               padded(w2, extra[0]), top, dtype=torch.float32)
        assert np.array_equal(gi.cpu().numpy(), ids)
        _check(y, ref, bar, "f32", (H, I, extra))


def test_a16_more_rows_than_one_grid_holds(g):
    """65,535 grid rows of 64 or 32 rows, and some: exact on small integers."""
    for M, N, K in ((65535 * 64 + 70, 16, 32), (65535 * 32 + 33, 3, 7)):
        rng = np.random.default_rng(N)
        b, sb = mx.random_rows(rng, N, K, 127, 128)
        bv = torch.from_numpy(mx.values(b, sb, K)).to(_dev(), torch.float32)
        gen = torch.Generator(device=_dev()).manual_seed(N)
        a = torch.randint(-4, 5, (M, K), device=_dev(), dtype=torch.int8, generator=gen).to(torch.bfloat16)
        got = g.matmul_mx(a, _mx(g, b, sb, K))
        # halves of at most 6 * 4 * 32: exact in fp32 in any order
        assert torch.equal(got, a.float() @ bv.T), (M, N, K)


def test_quantize_into_an_empty_matrix(g):
    x = torch.randn(5, 70, device=_dev())
    q = g.MxTensor.empty(5, 70, x.device)
    assert g.mx_quantize(x, out=q) is q
    ref = g.mx_quantize(x)
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
    with pytest.raises(ValueError):
        g.mx_quantize(x, out=g.MxTensor.empty(5, 71, x.device))
