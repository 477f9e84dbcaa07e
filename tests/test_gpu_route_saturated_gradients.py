"""Routing where scores are rounded to 1 or 0, or nearly: the gradients.

Their terms are products of what nothing has been subtracted from: with r the
choices' shares, dz[e] = c r[e] (sum_j r[j] (d[e] - d[j]) + (share of the experts that are
not chosen) d[e]), and 1 - s = 1 / (1 + exp(z)).  Their definition is formed in 50 decimal
digits; the bar is one rounding of the logits' type and 2^-40 of the sum of those terms'
magnitudes."""
import decimal

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D = decimal.Decimal


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _gradient(z, ids, d, score, renorm):
    """(dz, sum of the terms' magnitudes) of one token, in decimals."""
    E, zero, one = len(z), D(0), D(1)
    z, d = [D(float(v)) for v in z], [D(float(v)) for v in d]
    if score == "softmax":
        ex = [(v - max(z)).exp() for v in z]
        s = [v / sum(ex) for v in ex]
    else:
        s = [one / (one + (-v).exp()) for v in z]
    slope = [one if score == "softmax" else one / (one + v.exp()) for v in z]
    valid = [j for j, e in enumerate(ids) if 0 <= e < E]
    dz, mag = [zero] * E, [zero] * E
    if renorm or score == "sigmoid":
        total = sum(s[ids[j]] for j in valid) if renorm else one
        for j in valid:
            e = ids[j]
            r = s[e] / total
            terms = [s[ids[i]] / total * (d[j] - d[i]) for i in valid] if renorm else [d[j]]
            dz[e] += r * slope[e] * sum(terms)
            mag[e] += r * slope[e] * sum(abs(t) for t in terms)
    else:
        of = {}
        for j in valid:
            of[ids[j]] = of.get(ids[j], zero) + d[j]
        size = {}
        for j in valid:
            size[ids[j]] = size.get(ids[j], zero) + abs(d[j])
        for e in range(E):
            mine, most = of.get(e, zero), size.get(e, zero)
            dz[e] = s[e] * sum(s[f] * (mine - of.get(f, zero)) for f in range(E))
            mag[e] = s[e] * sum(s[f] * (most + size.get(f, zero)) for f in range(E) if f != e)
    return [float(v) for v in dz], [float(v) for v in mag]


ROWS = [[30.0, 0.0, 1.0, -1.0, 0.5, 2.0], [36.0, 34.0, -3.0, 0.0, 5.0, -40.0], [80.0, 20.0, 50.0, 60.0, 0.0, 10.0],
        [-30.0, -80.0, -36.0, -50.0, -90.0, -60.0], [0.25, -0.5, 1.0, 0.75, -1.0, 0.0], [25.0, 25.0, 0.0, -25.0, 24.0, 3.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradients_of_saturated_scores(g, score, renorm):
    print(f"case: saturated gradients {score} {renorm}", flush=True)
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(3)
    choices = [[0, 1, 2], [2, 1, 5], [0, 0, 3], [5, -1, 0], [4, 6, 4]]
    z = np.repeat(np.asarray(ROWS, np.float32), len(choices), 0)
    ids = np.asarray(choices * len(ROWS), np.int32)
    d = rng.standard_normal(ids.shape).astype(np.float32)
    got = g.moe_route_backward(torch.from_numpy(d).to(dev), torch.from_numpy(z).to(dev), torch.from_numpy(ids).to(dev), score=score,
                               renormalize=renorm).double().cpu().numpy()
    with decimal.localcontext() as ctx:
        ctx.prec = 50
        for t in range(len(z)):
            want, mag = (np.asarray(v) for v in _gradient(z[t], ids[t].tolist(), d[t], score, renorm))
            off = np.abs(got[t] - want) - (2.0 ** -24 * np.abs(want) + 2.0 ** -40 * mag + 2.0 ** -150)
            assert (off <= 0).all(), (score, renorm, z[t].tolist(), ids[t].tolist(), got[t].tolist(), want.tolist())
