"""GPU parity of the experts' products and their gradients (moe_experts,
moe_experts_backward) with their definition in 64 bits; bounds in experts_util.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from experts_util import check, reference  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _make(T, E, top, H, I, dtype, seed=0, drop=0.0, uneven=False):
    rng = np.random.default_rng(1000 * seed + T + 7 * E + 11 * top + 13 * H + 17 * I)
    dev = torch.device("cuda:0")
    to = lambda a: torch.from_numpy(a.astype(np.float32)).to(dev)  # noqa: E731
    x, dy = (to(rng.standard_normal((T, H))).to(dtype) for _ in range(2))
    w1 = to(rng.standard_normal((E, 2 * I, H)) / np.sqrt(H)).to(dtype)
    w2 = to(rng.standard_normal((E, H, I)) / np.sqrt(I)).to(dtype)
    z = rng.standard_normal((T, E)) + (8.0 * (np.arange(E) == E // 2) if uneven else 0.0)
    ids = np.argsort(-z, axis=1)[:, :top] if top <= E else rng.integers(0, E, (T, top))
    ids = np.where(rng.random((T, top)) < drop, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, top)), ids)
    gates = to(rng.random((T, top)) - 0.2)
    return x, torch.from_numpy(ids.astype(np.int32)).to(dev), gates, w1, w2, dy


def _all(g, args, what, forward=True):
    x, ids, gates, w1, w2, dy = args
    ref = reference(*args)
    y, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    check(y, ref["y"], (what, "y"))
    if forward:
        check(g.moe_experts(x, ids, gates, w1, w2), ref["y"], (what, "y alone"))
    got = g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved)
    for name, v in zip(("dx", "dgates", "dw1", "dw2"), got):
        check(v, ref[name], (what, name))
    assert (got[1][(ids < 0) | (ids >= w1.shape[0])] == 0).all(), what


# tokens, experts, choices, widths: one of each, tiles of one row and of several, blocks that
# end inside, rows of fewer than 8 values, odd rows and rows of whole 16 bytes
CASES = [(1, 1, 1, 1, 1), (1, 4, 2, 64, 32), (2, 3, 2, 5, 7), (3, 16, 1, 129, 130), (17, 3, 2, 96, 200),
         (64, 8, 4, 128, 64), (130, 2, 1, 256, 136), (257, 5, 3, 257, 65), (300, 1, 1, 72, 600),
         (333, 8, 2, 513, 257), (500, 70, 7, 40, 24), (1021, 7, 3, 200, 119), (100, 512, 16, 16, 8)]


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_products_and_gradients(g, case, fmt):
    print(f"case: experts {case} {fmt}", flush=True)
    _all(g, _make(*case, DT[fmt]), (case, fmt))


@pytest.mark.parametrize("case", [(40, 6, 3, 64, 48), (700, 6, 2, 72, 40)])
def test_dropped_choices_and_uneven_experts(g, case):
    print(f"case: experts dropped {case}", flush=True)
    _all(g, _make(*case, torch.bfloat16, drop=0.4), (case, "dropped"))
    _all(g, _make(*case, torch.bfloat16, uneven=True), (case, "uneven"))
    _all(g, _make(*case, torch.bfloat16, drop=1.0), (case, "all dropped"))


def test_the_same_expert_twice(g):
    for T in (3, 300):
        print(f"case: experts twice {T}", flush=True)
        args = list(_make(T, 4, 3, 64, 40, torch.float16))
        args[1] = args[1].clone()
        args[1][:, 2] = args[1][:, 0]
        ref = reference(*args)
        x, ids, gates, w1, w2, dy = args
        y, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
        check(y, ref["y"], "y")
        check(g.moe_experts(x, ids, gates, w1, w2), ref["y"], "y alone")
        for name, v in zip(("dx", "dgates", "dw1", "dw2"), g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved)):
            check(v, ref[name], name)


# the large tiles: 256 x 256
@pytest.mark.parametrize("case,fmt", [((2048, 8, 2, 1024, 1024), "bf16"), ((1500, 4, 4, 2048, 1016), "f16"),
                                      ((900, 16, 4, 1032, 1040), "bf16")])
def test_large_tiles(g, case, fmt):
    print(f"case: experts large {case} {fmt}", flush=True)
    _all(g, _make(*case, DT[fmt]), (case, fmt))


# more than the one workgroup's pairs: the listing in three launches
def test_many_pairs(g):
    print("case: experts many pairs", flush=True)
    _all(g, _make(5000, 37, 5, 64, 32, torch.bfloat16, drop=0.05), "many pairs")


def test_strides(g):
    """Row pitches, of odd numbers of values too, and NaN around the rows."""
    for off, pad in ((0, 8), (8, 24), (1, 3)):
        print(f"case: experts strides {off} {pad}", flush=True)
        x, ids, gates, w1, w2, dy = _make(290, 3, 2, 72, 40, torch.bfloat16)

        def wide(t):
            big = torch.full((*t.shape[:-1], t.shape[-1] + off + pad), float("nan"), dtype=t.dtype, device=t.device)
            v = big[..., off:off + t.shape[-1]]
            v.copy_(t)
            return v

        args = wide(x), ids, gates, wide(w1), wide(w2), wide(dy)
        ref = reference(x, ids, gates, w1, w2, dy)
        out = torch.full((290, 72 + pad), 5.0, dtype=x.dtype, device=x.device)
        y, saved = g.moe_experts(*args[:5], save=True, out=out[:, :72])
        check(y, ref["y"], (off, "y"))
        assert (out[:, 72:] == 5).all()
        got = g.moe_experts_backward(args[5], *args[:5], saved)
        for name, v in zip(("dx", "dgates", "dw1", "dw2"), got):
            check(v, ref[name], (off, name))


def test_no_tokens(g):
    x, ids, gates, w1, w2, dy = _make(4, 3, 2, 16, 8, torch.bfloat16)
    y, saved = g.moe_experts(x[:0], ids[:0], gates[:0], w1, w2, save=True)
    assert y.shape == (0, 16) and saved.shape == (0, 16)
    dx, dg, dw1, dw2 = g.moe_experts_backward(dy[:0], x[:0], ids[:0], gates[:0], w1, w2, saved)
    torch.cuda.synchronize()
    assert dx.shape == (0, 16) and dg.shape == (0, 2)
    assert (dw1 == 0).all() and (dw2 == 0).all()


def test_without_the_weights_gradients(g):
    x, ids, gates, w1, w2, dy = _make(300, 4, 2, 64, 40, torch.bfloat16)
    _, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    full = g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved)
    some = g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved, weights=False)
    assert len(some) == 2 and torch.equal(some[0], full[0]) and torch.equal(some[1], full[1])
