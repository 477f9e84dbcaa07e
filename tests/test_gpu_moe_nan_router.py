"""NaN in the router, from the definition: a NaN logit counts as the lowest z in the
choice; gate[s] = exp(z[chosen s]) over the sum of all experts' exp(z), which a NaN
logit makes NaN, or with ``renormalize`` over the chosen ones' alone, which it makes
NaN only where it was chosen.  Bar: as the layer's other tests, a gate 2^-23 of
itself; results are equal to those of a router without the NaN expert.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_moe import _dev, _host, _make, _on_gpu  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# One token, one workgroup's choice, and the choice in two launches; more than 64 experts.
@pytest.mark.parametrize("T,E", [(1, 5), (9, 8), (30, 8), (3, 100)])
@pytest.mark.parametrize("weights", ["w16", "mx"])
def test_nan_row_of_the_router(g, T, E, weights):
    top, H, I, bad = 2, 96, 64, E - 2
    rng = np.random.default_rng(7 + T)
    x, r, w1, w2 = _make(rng, T, E, H, I, "bf16", weights)
    g1, g2, _, _ = _on_gpu(g, w1, w2, E, H, I)
    x, r = x.to(_dev()), r.to(_dev())
    low = r.clone()  # the same expert, never chosen
    low[bad] = 0.0
    low[bad, 0] = -30000.0
    x[:, 0] = 1.0
    r[bad, 3] = float("nan")
    r[:bad, 0], r[bad + 1:, 0] = 0.125, 0.125
    low[:bad, 0], low[bad + 1:, 0] = 0.125, 0.125
    y, ids, gates = g.moe_layer(x, r, g1, g2, top, renormalize=True)
    want, wi, wg = g.moe_layer(x, low, g1, g2, top, renormalize=True)
    assert torch.equal(ids, wi) and not bool((ids == bad).any())
    assert torch.equal(gates, wg) and torch.equal(y, want)
    z = _host(x) @ np.delete(_host(r), bad, 0).T
    ex = np.exp(np.sort(z, 1)[:, :-top - 1:-1] - z.max(1, keepdims=True))
    assert (np.abs(_host(gates) - ex / ex.sum(1, keepdims=True)) <= 2.0 ** -23).all()
    # Over all experts: the sum holds the NaN.
    y, ids, gates = g.moe_layer(x, r, g1, g2, top, renormalize=False)
    assert torch.equal(ids, wi) and bool(torch.isnan(gates).all()) and bool(torch.isnan(y).all())


def test_a_chosen_nan_expert(g):
    """All experts chosen, the NaN one last: its gate and the sum are NaN."""
    T, E, H, I = 3, 4, 64, 32
    rng = np.random.default_rng(3)
    x, r, w1, w2 = (t.to(_dev()) for t in _make(rng, T, E, H, I, "bf16", "w16"))
    r[1, 5] = float("nan")
    for renormalize in (False, True):
        y, ids, gates = g.moe_layer(x, r, w1, w2, E, renormalize=renormalize)
        assert bool((ids[:, -1] == 1).all())
        assert bool(torch.isnan(gates).all()) and bool(torch.isnan(y).all())
