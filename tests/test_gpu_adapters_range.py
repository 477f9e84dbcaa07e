"""Adapters in fp16 whose scale A x lies far outside fp16's range, above and below, between
values that do not.

Bars, from the arithmetic: as in test_gpu_adapters.py, but for scale A x between the products:
it is off by half a step of fp16 relative to itself, and, where it is far below the largest of
its row's ranks, by 2^-28 of that (fp16's normal range below a value of 2^14 at least)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from experts_util import _mm  # noqa: E402

EPS, HS, TINY = 2.0 ** -23, 2.0 ** -11, 2.0 ** -25


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _reference(x, w, a, b, ids, scales):
    K, R = x.shape[1], a.shape[1]
    xd, wd = x.double(), w.double()
    y, bar = _mm(xd, wd.t()), (K + 8) * EPS * _mm(xd.abs(), wd.abs().t())
    most = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    for r in range(a.shape[0]):
        rows = torch.nonzero(ids == r).squeeze(1)
        if not rows.numel():
            continue
        ad, bd, s = a[r].double(), b[r].double(), scales[r].double()
        v, ev = s * _mm(xd[rows], ad.t()), abs(s) * (K + 24) * EPS * _mm(xd[rows].abs(), ad.abs().t())
        most[rows] = v.abs().max(1).values
        ev = ev + HS * (v.abs() + ev) + 2.0 ** -28 * (v.abs() + ev).max(1, keepdim=True).values
        y[rows] += _mm(v, bd.t())
        bar[rows] += _mm(ev, bd.abs().t()) + (R + 8) * EPS * _mm(v.abs() + ev, bd.abs().t())
    return y, bar + 4 * EPS * y.abs(), most


# rows: thin products of one and of four blocks, by rows of whole 16 bytes, odd ones and ones of
# fewer than 8 values; tiles with K whole and in parts, rows in the same three ways
CASES = [(1, 64, 128, 16, 3), (5, 17, 5, 3, 2), (40, 100, 301, 100, 8), (64, 4096, 512, 64, 9), (61, 200, 96, 512, 5), (200, 264, 520, 33, 7),
         (600, 130, 4096, 16, 5), (700, 264, 2049, 65, 30), (560, 129, 7, 40, 9), (3000, 4096, 512, 32, 6)]


@pytest.mark.parametrize("case", CASES)
def test_fp16_range(g, case):
    T, N, K, R, count = case
    print(f"case: adapters range {case}", flush=True)
    rng = np.random.default_rng(sum(case))
    dev = torch.device("cuda:0")
    to = lambda v, by=1.0: torch.from_numpy((v * by).astype(np.float32)).to(dev, torch.float16)  # noqa: E731
    normal = rng.standard_normal
    ids = torch.from_numpy(rng.integers(-1, count, T).astype(np.int32)).to(dev)
    ids[0] = 0
    # A x of 2^20 by B of 2^-20 in the first adapter, 2^-24 (from scales of 2^-20) by 2^10 in the last,
    # of the order of one between, beside W x of 2^-10; the first one's last ranks 2^-12 times its first ones
    a = normal((count, R, K)) / K ** 0.5
    b = normal((count, N, R)) / R ** 0.5
    scales = (rng.random(count) + 0.5).astype(np.float32)
    scales[0], scales[-1] = 2.0 ** 20, 2.0 ** -20
    a[0, R // 2:] *= 2.0 ** -12
    b[0] *= 2.0 ** -12
    b[-1] *= 2.0 ** 10
    x, w, a, b = to(normal((T, K))), to(normal((N, K)), 2.0 ** -10 * K ** -0.5), to(a), to(b)
    scales = torch.from_numpy(scales).to(dev)
    value, bound, most = _reference(x, w, a, b, ids, scales)
    assert float(most[0]) > 70000 and float(value.abs().max()) < 60000
    got = g.matmul_adapters(x, w, a, b, ids, scales)
    off = (got.double() - value).abs() - (bound * (1 + HS) + HS * value.abs() + TINY)
    assert torch.isfinite(got).all() and float(off.max()) <= 0, (case, float(off.max()))


@pytest.mark.parametrize("T", [1, 30, 64, 65, 700])
def test_one_requests_infinities_are_its_own(g, T):
    """As for bf16 in test_gpu_adapters.py: the other rows' results as they are, to the bit."""
    import test_gpu_adapters as adapters
    print(f"case: adapters fp16 infinities {T}", flush=True)
    x, w, a, b, i, s = adapters._make(T, 200, 256, 70, 4, torch.float16, ids=np.arange(T) % 4)
    want = g.matmul_adapters(x, w, a, b, i, s)
    own = i == 2
    for name in ("a nan", "a inf", "b", "scale", "scale nan"):
        a2, b2, s2 = a.clone(), b.clone(), s.clone()
        if name[0] == "a":
            a2[2, 5] = float(name[2:])
        elif name == "b":
            b2[2, ::2] = float("inf")
            b2[2, 1::2] = float("nan")
        else:
            s2[2] = float("inf") if name == "scale" else float("nan")
        got = g.matmul_adapters(x, w, a2, b2, i, s2)
        assert torch.equal(got[~own], want[~own]), (T, name)
        assert not torch.isfinite(got[own]).any() if name != "b" else not own.any() or not torch.isfinite(got[own]).all(), (T, name)
