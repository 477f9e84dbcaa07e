"""GPU parity of routing (moe_route, moe_route_backward) with its definition in 64 bits.

Bars.  The choice is equal: keys are 64-bit values, and the test's inputs hold either
exact ties or keys that are further apart than 64-bit roundings (checked).  A gate is
one fp32 rounding of a 64-bit value, 2^-24 of it, with as much again for the 64-bit
exponentials (below 2^-40); a gradient one rounding of its type of a 64-bit value whose
terms cancel: 2^-40 of the sum of the terms' magnitudes besides."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _scores(z, score):
    if score == "sigmoid":
        return 1 / (1 + np.exp(-z))
    top = z.max(axis=1, keepdims=True)
    ex = np.exp(z - np.where(np.isfinite(top), top, 0.0))
    total = ex.sum(axis=1, keepdims=True)
    return ex / np.where(total > 0, total, 1.0)


def route(z, top, score, bias, groups, keep, by, renorm, scale):
    """(ids, gates, least distance of two keys next to each other that differ)."""
    T, E = z.shape
    s = _scores(z, score)
    masked = np.isneginf(z)
    by_score = bias is not None or (keep < groups and by == "top2")
    key = s + (bias if bias is not None else 0.0) if by_score else z.copy()
    key = np.where(masked, -np.inf, key)
    if keep < groups:
        part = -np.sort(-key.reshape(T, groups, -1), axis=2)
        total = part[:, :, 0].copy()
        if by == "top2" and part.shape[2] > 1:
            two = np.isfinite(part[:, :, 1])
            total[two] += part[:, :, 1][two]
        kept = np.argsort(-total, axis=1, kind="stable")[:, :keep]
        allowed = np.zeros((T, groups), bool)
        np.put_along_axis(allowed, kept, True, 1)
        allowed = np.repeat(allowed, E // groups, 1)
    else:
        allowed = np.ones((T, E), bool)
    ids = np.zeros((T, top), int)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (not allowed[t, e], -key[t, e], e))
        ids[t] = order[:top]
    gates = np.take_along_axis(s, ids, 1)
    gates = np.where(np.take_along_axis(masked, ids, 1), 0.0, gates)
    if renorm:
        if score == "softmax":  # not over a sum that has lost the chosen ones
            zc = np.take_along_axis(z, ids, 1)
            m = zc.max(axis=1, keepdims=True)
            gates = np.where(np.isneginf(zc), 0.0, np.exp(zc - np.where(np.isfinite(m), m, 0.0)))
        total = gates.sum(axis=1, keepdims=True)
        gates = gates / np.where(total > 0, total, 1.0)
    return ids, scale * gates


def _logits(rng, T, E, fmt, ties=False, mask=0.0):
    z = rng.standard_normal((T, E)).astype(np.float32) * 2
    if ties:
        z = np.round(z * 2) / 2
    z[rng.random((T, E)) < mask] = -np.inf
    t = torch.from_numpy(z).to(DT[fmt])
    return t, t.double().numpy()


CASES = [(1, 1, 1, 1, 1), (1, 64, 8, 1, 1), (3, 5, 5, 1, 1), (7, 63, 6, 1, 1), (65, 128, 8, 8, 4), (33, 256, 8, 8, 3),
         (257, 100, 10, 10, 2), (9, 512, 16, 64, 5), (20, 512, 16, 1, 1), (50, 6, 2, 3, 2), (40, 7, 1, 7, 1), (4, 130, 3, 65 // 5, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES)
def test_route(g, case, score):
    T, E, top, groups, keep = case
    if groups > 1 and E % groups:
        groups, keep = 1, 1
    print(f"case: route {case} {score}", flush=True)
    rng = np.random.default_rng(sum(case))
    dev = torch.device("cuda:0")
    for fmt in ("f32", "bf16", "f16"):
        for ties, mask in ((False, 0.0), (True, 0.0), (False, 0.5), (True, 1.0)):
            t, z = _logits(rng, T, E, fmt, ties, mask)
            for with_bias in (False, True):
                # multiples of 1/8 and distinct exponentials: equal keys are exactly equal
                bias = np.round(rng.standard_normal(E) * 4).astype(np.float32) / 8 if with_bias else None
                for by in ("max", "top2") if groups > 1 else ("max",):
                    for renorm in (False, True):
                        ids, gates = route(z, top, score, bias, groups, keep, by, renorm, 2.5)
                        gi, gg = g.moe_route(t.to(dev), top, score=score, bias=None if bias is None else torch.from_numpy(bias).to(dev),
                                             groups=groups, top_groups=keep, group_score=by, renormalize=renorm, scale=2.5)
                        what = (case, score, fmt, ties, mask, with_bias, by, renorm)
                        assert gi.dtype == torch.int32 and gg.dtype == torch.float32
                        assert np.array_equal(gi.cpu().numpy(), ids), what
                        assert (np.abs(gg.double().cpu().numpy() - gates) <= 2.0 ** -23 * gates).all(), what


def _gradient(z, ids, dg, score, renorm, scale):
    """(dz, sum of its terms' magnitudes)."""
    s = _scores(z, score)
    T, E = z.shape
    rows = np.arange(T)[:, None]
    valid = (ids >= 0) & (ids < E)
    at = np.where(valid, ids, 0)
    d = np.where(valid, scale * dg, 0.0)
    picked = np.where(valid, s[rows, at], 0.0)
    total = picked.sum(1, keepdims=True) if renorm else np.ones((T, 1))
    r = picked / np.where(total > 0, total, 1.0)
    dz, mag = np.zeros_like(z), np.zeros_like(z)
    if score == "softmax" and not renorm:
        mean, size = (d * r).sum(1, keepdims=True), np.abs(d * r).sum(1, keepdims=True)
        dz -= s * mean
        mag += s * size
        np.add.at(dz, (rows, at), np.where(valid, d * r, 0.0))
        np.add.at(mag, (rows, at), np.where(valid, np.abs(d * r), 0.0))
        return dz, mag
    slope = 1 - picked if score == "sigmoid" else 1.0
    mean = (d * r).sum(1, keepdims=True) if renorm else 0.0
    size = np.abs(d * r).sum(1, keepdims=True) if renorm else 0.0
    np.add.at(dz, (rows, at), np.where(valid, r * slope * (d - mean), 0.0))
    np.add.at(mag, (rows, at), np.where(valid, r * (np.abs(d) + size), 0.0))
    return dz, mag


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", CASES)
def test_gradient(g, case, score):
    T, E, top = case[:3]
    print(f"case: route gradient {case} {score}", flush=True)
    rng = np.random.default_rng(sum(case) + 1)
    dev = torch.device("cuda:0")
    for fmt in ("f32", "bf16", "f16"):
        for mask in (0.0, 0.5, 1.0):
            t, z = _logits(rng, T, E, fmt, mask=mask)
            dg = rng.standard_normal((T, top)).astype(np.float32)
            ids, _ = g.moe_route(t.to(dev), top, score=score)
            more = rng.integers(-1, E + 1, (T, top)).astype(np.int32)  # repeated and dropped choices
            for ids in (ids.cpu().numpy(), more):
                for renorm in (False, True):
                    out = torch.full((T, E + 3), 7.0, dtype=DT[fmt], device=dev)
                    got = g.moe_route_backward(torch.from_numpy(dg).to(dev), t.to(dev), torch.from_numpy(ids).to(dev), score=score,
                                               renormalize=renorm, scale=1.5, out=out[:, :E])
                    dz, mag = _gradient(z, ids, dg.astype(np.float64), score, renorm, 1.5)
                    off = np.abs(got.double().cpu().numpy() - dz)
                    limit = HALF_STEP[fmt] * np.abs(dz) + 2.0 ** -40 * mag + TINY[fmt]
                    assert (off <= limit).all(), (case, score, fmt, mask, renorm, float((off - limit).max()))
                    assert (out[:, E:] == 7).all()


def test_gradient_by_differences(g):
    """The gates' change over a step against their gradient: central differences of
    64-bit gates (the definition above) at a step of 2^-12, whose error is of the square."""
    rng = np.random.default_rng(5)
    dev = torch.device("cuda:0")
    z = rng.standard_normal((6, 12)).astype(np.float32).astype(np.float64)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            dg = rng.standard_normal((6, 3)).astype(np.float32)
            ids, _ = route(z, 3, score, None, 1, 1, "max", renorm, 1.0)

            def total(y):
                s = np.take_along_axis(_scores(y, score), ids, 1)
                return ((s / s.sum(1, keepdims=True) if renorm else s) * dg).sum(1)

            want = np.zeros_like(z)
            for e in range(12):
                up, down = z.copy(), z.copy()
                up[:, e] += 2.0 ** -12
                down[:, e] -= 2.0 ** -12
                want[:, e] = (total(up) - total(down)) * 2.0 ** 11
            got = g.moe_route_backward(torch.from_numpy(dg).to(dev), torch.from_numpy(z.astype(np.float32)).to(dev),
                                       torch.from_numpy(ids.astype(np.int32)).to(dev), score=score, renormalize=renorm)
            # third derivatives of these functions stay below 6: 6 / 6 * 2^-24 per unit of dg
            assert np.abs(got.double().cpu().numpy() - want).max() <= 2.0 ** -22 * np.abs(dg).sum(1).max()


def test_infinities_and_nan(g):
    dev = torch.device("cuda:0")
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[0.0, inf, 1.0, inf], [nan, 0.0, 1.0, -inf], [-inf, -inf, -inf, -inf], [nan, nan, nan, nan]], device=dev)
    ids, gates = g.moe_route(z, 2, renormalize=False)
    assert ids.tolist() == [[1, 3], [2, 1], [0, 1], [0, 1]]
    assert gates[0].tolist() == [0.5, 0.5] and gates[1].isnan().all() and (gates[2] == 0).all() and gates[3].isnan().all()
    ids, gates = g.moe_route(z, 2)
    assert gates[0].tolist() == [0.5, 0.5] and (gates[1] > 0).all() and (gates[2] == 0).all() and gates[3].isnan().all()
    ids, gates = g.moe_route(z, 2, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[1, 3], [2, 1], [0, 1], [0, 1]]
    assert gates[0].tolist() == [1.0, 1.0] and (gates[1] > 0).all() and (gates[2] == 0).all() and gates[3].isnan().all()
    # a bias does not bring a masked expert before others
    ids, gates = g.moe_route(z[1:2], 3, bias=torch.tensor([9.0, 0.0, 0.0, 9.0], device=dev), renormalize=False, score="sigmoid")
    assert ids.tolist() == [[2, 1, 0]]
    # sigmoid scores that are rounded to 1 or 0 are still ordered by their logits
    ids, _ = g.moe_route(torch.tensor([[50.0, 60.0, 70.0, -900.0, -800.0]], device=dev), 5, score="sigmoid")
    assert ids.tolist() == [[2, 1, 0, 4, 3]]


def test_pitch_and_no_tokens(g):
    dev = torch.device("cuda:0")
    big = torch.full((9, 40), float("nan"), device=dev)
    big[:, 3:20] = torch.randn(9, 17, device=dev)
    ids, gates = g.moe_route(big[:, 3:20], 4)
    want = g.moe_route(big[:, 3:20].contiguous(), 4)
    assert torch.equal(ids, want[0]) and torch.equal(gates, want[1])
    ids, gates = g.moe_route(big[:0, 3:20], 4)
    assert ids.shape == (0, 4) and gates.shape == (0, 4)
    assert g.moe_route_backward(gates, big[:0, 3:20], ids).shape == (0, 17)


# ---- many tokens: several to a wave ---------------------------------------------------------

MANY = [(2049, 63, 6, 1, 1), (2048, 16, 2, 4, 2), (4097, 5, 5, 1, 1), (10241, 256, 8, 8, 4), (5500, 128, 8, 16, 3),
        (2100, 512, 16, 2, 1), (4444, 100, 10, 10, 2), (4050, 64, 4, 32, 4), (2060, 30, 3, 15, 14), (3001, 256, 8, 8, 4)]


def _route_many(z, top, score, bias, groups, keep, by, renorm):
    """`route` without its loop over tokens."""
    T, E = z.shape
    s = _scores(z, score)
    masked = np.isneginf(z)
    by_score = bias is not None or (keep < groups and by == "top2")
    key = np.where(masked, -1e300, s + (bias if bias is not None else 0.0) if by_score else z)
    if keep < groups:
        part = -np.sort(-key.reshape(T, groups, -1), axis=2)
        total = part[:, :, 0].copy()
        if by == "top2" and part.shape[2] > 1:
            total += np.where(part[:, :, 1] > -1e300, part[:, :, 1], 0.0)
        kept = np.argsort(-total, axis=1, kind="stable")[:, :keep]
        allowed = np.zeros((T, groups), bool)
        np.put_along_axis(allowed, kept, True, 1)
        key = np.where(np.repeat(allowed, E // groups, 1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top]
    gates = np.where(np.take_along_axis(masked, ids, 1), 0.0, np.take_along_axis(s, ids, 1))
    if renorm:
        if score == "softmax":
            zc = np.take_along_axis(z, ids, 1)
            m = zc.max(axis=1, keepdims=True)
            gates = np.where(np.isneginf(zc), 0.0, np.exp(zc - np.where(np.isfinite(m), m, 0.0)))
        total = gates.sum(axis=1, keepdims=True)
        gates = gates / np.where(total > 0, total, 1.0)
    return ids, gates


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", MANY)
def test_route_many_tokens(g, case, score):
    T, E, top, groups, keep = case
    print(f"case: route many {case} {score}", flush=True)
    rng = np.random.default_rng(sum(case) + 7)
    dev = torch.device("cuda:0")
    for fmt, ties, mask in (("f32", False, 0.0), ("bf16", True, 0.3), ("f16", False, 0.6)):
        t, z = _logits(rng, T, E, fmt, ties, mask)
        z[5], z[T - 1] = -np.inf, -np.inf
        t = torch.from_numpy(z.astype(np.float32)).to(DT[fmt])
        for bias in (None, np.round(rng.standard_normal(E) * 4).astype(np.float32) / 8):
            for by in ("max", "top2") if groups > 1 else ("max",):
                for renorm in (False, True):
                    ids, gates = _route_many(z, top, score, bias, groups, keep, by, renorm)
                    gi, gg = g.moe_route(t.to(dev), top, score=score, bias=None if bias is None else torch.from_numpy(bias).to(dev),
                                         groups=groups, top_groups=keep, group_score=by, renormalize=renorm)
                    what = (case, score, fmt, bias is not None, by, renorm)
                    assert np.array_equal(gi.cpu().numpy(), ids), what
                    assert (np.abs(gg.double().cpu().numpy() - gates) <= 2.0 ** -23 * gates).all(), what


def test_many_tokens_with_nan_and_infinities(g):
    """The same rows as a few tokens give."""
    dev = torch.device("cuda:0")
    inf, nan = float("inf"), float("nan")
    few = torch.tensor([[0.0, inf, 1.0, inf, -2.0], [nan, 0.0, 1.0, -inf, 0.5], [-inf] * 5, [nan] * 5, [3.0, 2.0, nan, -inf, 1.0]], device=dev)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            want = g.moe_route(few, 3, score=score, renormalize=renorm)
            got = g.moe_route(few.repeat(500, 1), 3, score=score, renormalize=renorm)
            assert torch.equal(got[0], want[0].repeat(500, 1))
            assert torch.equal(got[1].nan_to_num(-1.0), want[1].repeat(500, 1).nan_to_num(-1.0))
