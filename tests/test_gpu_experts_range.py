"""The experts' products in fp16 at the ends of its range: what gemm_experts.h says of the
inner values.  Bounds, element by element, in experts_util.py (half a step of a value, or of
fp16's smallest ones)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from experts_util import reference  # noqa: E402

HS, TINY = 2.0 ** -11, 2.0 ** -25


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _make(T, E, H, I, by, back, seed):
    """Inner values of the order of by^2, results of by^2 back."""
    rng = np.random.default_rng(seed)
    dev = torch.device("cuda:0")
    to = lambda s, f: torch.from_numpy((rng.standard_normal(s) * f).astype(np.float32)).to(dev, torch.float16)  # noqa: E731
    x, w1, w2 = to((T, H), 1.0), to((E, 2 * I, H), by * H ** -0.5), to((E, H, I), back * I ** -0.5)
    ids = torch.from_numpy(rng.integers(0, E, (T, 2)).astype(np.int32)).to(dev)
    gates = torch.from_numpy((rng.random((T, 2)) + 0.5).astype(np.float32)).to(dev)
    return x, ids, gates, w1, w2


def _off(got, ref):
    value, bound = ref
    return (got.double() - value).abs() - (bound * (1 + HS) + HS * value.abs() + TINY)


@pytest.mark.parametrize("T,E", [(6, 16), (300, 4)])
def test_past_the_largest_value(g, T, E):
    """Kept in fp32: finite.  Kept in fp16: a row with such a value is not, and no other row is
    touched."""
    print(f"case: experts past fp16 {T}", flush=True)
    x, ids, gates, w1, w2 = _make(T, E, 264, 200, 600.0, 2.0 ** -13, T)
    x[::3] *= 2.0 ** -9  # these rows' inner values are of the order of one
    ref = reference(x, ids, gates, w1, w2)["y"]
    h = torch.stack([x[t].double() @ w1[ids[t].long()].double().transpose(1, 2).contiguous() for t in range(T)])
    u = torch.nn.functional.silu(h[..., :200]) * h[..., 200:]
    large = (u.abs() > 65600).any(-1).any(-1)
    inside = (u.abs() < 65400).all(-1).all(-1)
    assert large[1] and inside[0] and float(ref[0].abs().max()) < 60000
    for save in (False, True):
        got = g.moe_experts(x, ids, gates, w1, w2, save=save)
        y = got[0] if save else got
        assert float(_off(y, ref)[inside].max()) <= 0, (T, save)
        if T == 6 and not save:
            assert torch.isfinite(y).all() and float(_off(y, ref).max()) <= 0
        else:
            assert (~torch.isfinite(y[large])).any(1).all(), (T, save)


@pytest.mark.parametrize("T,E", [(6, 16), (300, 4)])
def test_below_the_smallest_normal_value(g, T, E):
    print(f"case: experts below fp16 {T}", flush=True)
    x, ids, gates, w1, w2 = _make(T, E, 264, 200, 2.0 ** -9, 2.0 ** 9, T + 1)
    dy = x.flip(0).contiguous()
    ref = reference(x, ids, gates, w1, w2, dy)
    y, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    assert float(_off(y, ref["y"]).max()) <= 0 and float(ref["y"][0].abs().max()) > 2.0 ** -10
    assert float(_off(g.moe_experts(x, ids, gates, w1, w2), ref["y"]).max()) <= 0
    for name, got in zip(("dx", "dgates", "dw1", "dw2"), g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved)):
        assert float(_off(got, ref[name]).max()) <= 0, name
