"""Loops that go from one piece of work to the next: gemm_mx tiles where a workgroup
takes several, each of more than one k step; experts' products where a wave takes
several groups of columns and the tile of activations, which does not hold a row,
is brought again for each; one token whose first tile does not hold its row.  Exact
on small integers, or within the layer's bars.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import mx  # noqa: E402
from test_gpu_moe import DT, _check, _dev, _layer, _make, _on_gpu  # noqa: E402
from test_gpu_mx import _host, _mx  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# 17 x 17 tiles of 256 on 256 compute units, 24 x 24 of 128 on two workgroups each;
# 2, 3 and 4 steps of 256, whole and (600, 1000) with a partial last one.
@pytest.mark.parametrize("K", [512, 768, 600, 1000])
@pytest.mark.parametrize("entry,M,N", [(1, 4352, 4300), (2, 2950, 3000)])
def test_several_tiles_of_several_steps(g, entry, M, N, K):
    rng = np.random.default_rng(K + M)
    a, sa = mx.random_rows(rng, M, K, 126, 129, pad=255)
    b, sb = mx.random_rows(rng, N, K, 126, 129, pad=255)
    # multiples of 1/16 of at most 144 each: below 2^18 for K <= 1000, exact in fp32
    ref = mx.values(a, sa, K).astype(np.float32) @ mx.values(b, sb, K).T.astype(np.float32)
    qa, qb = _mx(g, a, sa, K), _mx(g, b, sb, K)
    for fmt in DT:
        got = g.matmul_mx(qa, qb, dtype=DT[fmt], config=entry)
        assert np.array_equal(_host(got), mx.round_to(ref.astype(np.float64), fmt)), fmt


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_tiles_brought_again_second_product(g, fmt, weights):
    """32 experts of 129 groups of columns: two groups to a wave; 2000 inner values."""
    T, E, top, H, I = 40, 32, 2, 2049, 2000
    rng = np.random.default_rng(77)
    x, r, w1, w2 = _make(rng, T, 4, H, I, fmt, weights)  # 4 experts' weights, in turn
    r = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(DT[fmt])
    _run(g, x, r, w1, w2, T, E, top, H, I, fmt, weights)


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_tiles_brought_again_first_product(g, fmt, weights):
    """512 experts of 8 groups: two to a wave; tokens of 2,100 values, of which a tile
    of 16 rows holds 2,048; every token asks the same 7 experts and one more."""
    T, E, top, H, I = 70, 512, 8, 2100, 113
    rng = np.random.default_rng(78)
    x, r, w1, w2 = _make(rng, T, 4, H, I, fmt, weights)
    r = torch.from_numpy((rng.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).to(DT[fmt])
    x[:, 0] = 4.0
    r[:, 0] = 0.0
    r[100:107, 0] = 8.0
    _run(g, x, r, w1, w2, T, E, top, H, I, fmt, weights)


def _run(g, x, r, w1, w2, T, E, top, H, I, fmt, weights):
    turn = np.arange(E) % 4
    if weights == "mx":
        def spread(q, rows):
            return tuple(t.reshape(4, rows, -1)[turn].reshape(E * rows, -1) if k < 2 else t[turn]
                         for k, t in enumerate(q))
        w1, w2 = spread(w1, 2 * I), spread(w2, H)
    else:
        w1, w2 = w1[turn], w2[turn]
    g1, g2, v1, v2 = _on_gpu(g, w1, w2, E, H, I)
    z = -np.sort(-(x.double().numpy() @ r.double().numpy().T), axis=1)
    assert (z[:, :-1] - z[:, 1:])[:, :top].min() > 1e-11  # the choice does not hang on last bits
    ref, bar, ids, gates = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
    y, gi, gg = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
    assert np.array_equal(gi.cpu().numpy(), ids)
    assert (np.abs(_host(gg) - gates) <= 2.0 ** -23 * gates).all()
    _check(y, ref, bar, "f32", (fmt, weights))


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("H", [7168, 7501])
def test_one_token_in_several_tiles(g, H, fmt, weights):
    T, E, top, I = 1, 8, 2, 100
    rng = np.random.default_rng(H)
    x, r, w1, w2 = _make(rng, T, E, H, I, fmt, weights)
    g1, g2, v1, v2 = _on_gpu(g, w1, w2, E, H, I)
    ref, bar, ids, _ = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
    for _ in range(2):
        y, gi, _ = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
        assert np.array_equal(gi.cpu().numpy(), ids)
        _check(y, ref, bar, "f32", (H, fmt, weights))


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [4, 50])
def test_two_waves_to_a_group(g, T, fmt, weights):
    """8 experts of 129 and 131 groups, which 16-bit weights' waves share by twos."""
    E, top, H, I = 8, 2, 2057, 2090
    rng = np.random.default_rng(T)
    x, r, w1, w2 = _make(rng, T, E, H, I, fmt, weights)
    g1, g2, v1, v2 = _on_gpu(g, w1, w2, E, H, I)
    ref, bar, ids, _ = _layer(x.double().numpy(), r.double().numpy(), v1, v2, top, True)
    y, gi, _ = g.moe_layer(x.to(_dev()), r.to(_dev()), g1, g2, top, dtype=torch.float32)
    assert np.array_equal(gi.cpu().numpy(), ids)
    _check(y, ref, bar, "f32", (T, fmt, weights))
