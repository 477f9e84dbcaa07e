"""Routing, the experts' products, their gradients and adapters together, as a layer uses
them; captured and replayed; on another stream; their results' bits; and their largest
tensors."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from experts_util import check, reference  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


def _dev():
    return torch.device("cuda:0")


def _layer(T, E, H, I, count, R, dtype, seed=3):
    rng = np.random.default_rng(seed)
    to = lambda *s, by=1.0: torch.from_numpy((rng.standard_normal(s) / by).astype(np.float32)).to(_dev(), dtype)  # noqa: E731
    s = {"x": to(T, H), "dy": to(T, H), "w": to(H, H, by=H ** .5), "a": to(count, R, H, by=H ** .5), "b": to(count, H, R, by=R ** .5),
         "router": to(E, H, by=H ** .5), "w1": to(E, 2 * I, H, by=H ** .5), "w2": to(E, H, I, by=I ** .5)}
    s["rows"] = torch.from_numpy(rng.integers(-1, count, T).astype(np.int32)).to(_dev())
    s["scales"] = torch.from_numpy(rng.random(count).astype(np.float32)).to(_dev())
    s["bias"] = torch.from_numpy((rng.standard_normal(E) / 10).astype(np.float32)).to(_dev())
    return s


def _run(g, s, train=True, **kw):
    """A projection with adapters, its logits, the choice of experts, their products; and back."""
    h = g.matmul_adapters(s["x"], s["w"], s["a"], s["b"], s["rows"], s["scales"], **kw)
    logits = g.matmul_mixed(h, s["router_t"], **kw)
    ids, gates = g.moe_route(logits, 2, score="sigmoid", bias=s["bias"], groups=2, top_groups=1, group_score="top2", scale=1.5, **kw)
    if not train:
        return h, ids, gates, g.moe_experts(h, ids, gates, s["w1"], s["w2"], **kw)
    y, saved = g.moe_experts(h, ids, gates, s["w1"], s["w2"], save=True, **kw)
    dh, dgates, dw1, dw2 = g.moe_experts_backward(s["dy"], h, ids, gates, s["w1"], s["w2"], saved, **kw)
    dz = g.moe_route_backward(dgates, logits, ids, score="sigmoid", scale=1.5, **kw)
    return h, ids, gates, y, dh, dgates, dw1, dw2, dz


def _state(g, *args):
    s = _layer(*args)
    s["router_t"] = s["router"].t().contiguous()
    return s


@pytest.mark.parametrize("size", [(3, 8, 64, 48, 3, 8), (200, 8, 72, 40, 5, 6), (1500, 16, 256, 128, 4, 16)])
def test_a_layer(g, size):
    """Each part against its definition on the part before it; the logits' gradient by
    automatic differentiation of the gates' formula in 64 bits."""
    print(f"case: layer {size}", flush=True)
    s = _state(g, *size, torch.bfloat16)
    h, ids, gates, y, dh, dgates, dw1, dw2, dz = _run(g, s)
    ref = reference(h, ids, gates, s["w1"], s["w2"], s["dy"])
    for name, got in (("y", y), ("dx", dh), ("dgates", dgates), ("dw1", dw1), ("dw2", dw2)):
        check(got, ref[name], (size, name))
    z = g.matmul_mixed(h, s["router_t"]).double().requires_grad_(True)
    picked = torch.sigmoid(z).gather(1, ids.long())
    want = 1.5 * picked / picked.sum(1, keepdim=True)
    assert ((gates.double() - want).abs() <= 2.0 ** -22 * want).all()
    (want * dgates.double()).sum().backward()
    # fp32 logits' gradient: one rounding of a 64-bit value whose terms cancel
    terms = 1.5 * dgates.double().abs().sum(1, keepdim=True)
    assert ((dz.double() - z.grad).abs() <= 2.0 ** -24 * z.grad.abs() + 2.0 ** -40 * terms).all()


def test_gradients_by_differences(g):
    """Central differences of the 64-bit definition along random directions, against the
    gradients: its third derivative times the step's square is below 2^-14 of the sum of
    magnitudes here, and the gradients' own errors are the bounds of experts_util.py."""
    s = _state(g, 40, 4, 32, 24, 2, 4, torch.float16)
    x, w1, w2 = s["x"], s["w1"], s["w2"]
    ids = torch.from_numpy(np.random.default_rng(1).integers(0, 4, (40, 2)).astype(np.int32)).to(_dev())
    gates = torch.rand(40, 2, device=_dev())
    _, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    grads = g.moe_experts_backward(s["dy"], x, ids, gates, w1, w2, saved)
    ref = reference(x, ids, gates, w1, w2, s["dy"])

    def loss(x, gates, w1, w2):
        total = 0.0
        for e in range(4):
            tok, slot = torch.nonzero(ids == e, as_tuple=True)
            h = x[tok] @ w1[e].t().contiguous()
            u = torch.nn.functional.silu(h[:, :24]) * h[:, 24:]
            total = total + (gates[tok, slot].unsqueeze(1) * (u @ w2[e].t().contiguous()) * s["dy"][tok].double()).sum()
        return total

    at = [t.double() for t in (x, gates, w1, w2)]
    step = 2.0 ** -12
    for i, (name, got) in enumerate(zip(("dx", "dgates", "dw1", "dw2"), grads)):
        way = torch.randn_like(at[i])
        up, down = ([t + (step * way if j == i else 0.0) * sign for j, t in enumerate(at)] for sign in (1, -1))
        want = (loss(*up) - loss(*down)) / (2 * step)
        value, bound = ref[name]
        half = {torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[got.dtype]
        slack = ((bound + half * (value.abs() + bound)) * way.abs()).sum() + 2.0 ** -14 * (value * way).abs().sum()
        assert (got.double() * way).sum() - want <= slack and want - (got.double() * way).sum() <= slack, name


@pytest.mark.parametrize("size", [(1, 8, 64, 48, 3, 8), (20, 8, 64, 48, 3, 8), (300, 8, 256, 128, 4, 8), (1200, 16, 264, 72, 40, 16)])
def test_same_bits(g, size):
    s = _state(g, *size, torch.bfloat16)
    first = _run(g, s)
    for _ in range(3):
        for a, b in zip(first, _run(g, s)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("size", [(1, 8, 64, 48, 3, 8), (40, 16, 72, 40, 6, 17), (900, 8, 256, 128, 4, 8), (3000, 16, 128, 72, 9, 16)])
def test_captured_and_replayed(g, size, train):
    """Every replay, on new inputs and with eager work between, against the eager results."""
    print(f"case: captured {size} {train}", flush=True)
    s = _state(g, *size, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(g, s, train)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _run(g, s, train)
    for turn in range(4):
        new = _state(g, *size, torch.bfloat16, 10 + turn)
        for name in ("x", "dy", "rows", "w1", "bias"):
            s[name].copy_(new[name])
        want = [t.clone() for t in _run(g, s, train)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, captured):
            assert torch.equal(a, b), (size, train, turn)


def test_two_captured_graphs_and_two_streams(g):
    """Two calls at once, each with tensors of its own."""
    states = [_state(g, 700, 8, 128, 64, 4, 8, torch.bfloat16, seed) for seed in (1, 2)]
    want = [[t.clone() for t in _run(g, s)] for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, stream in zip(states, streams):
            got.append(_run(g, s, stream=stream.cuda_stream))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, o))
    graphs, outs = [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_run(g, s))
        graphs.append(graph)
    for _ in range(3):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_a_workspace_of_the_callers_own(g):
    s = _state(g, 300, 8, 64, 48, 3, 8, torch.bfloat16)
    h, ids, gates, y, dh, dgates, dw1, dw2, dz = _run(g, s)
    for fill in (0, 255):
        ws = torch.full((g.gemm_experts_workspace_bytes(300, 8, 2, 64, 48, 1),), fill, dtype=torch.uint8, device=_dev())
        y2, saved = g.moe_experts(h, ids, gates, s["w1"], s["w2"], save=True, workspace=ws)
        got = g.moe_experts_backward(s["dy"], h, ids, gates, s["w1"], s["w2"], saved, workspace=ws)
        assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip((dh, dgates, dw1, dw2), got))
        wa = torch.full((g.gemm_adapters_workspace_bytes(300, 64, 64, 8, 3),), fill, dtype=torch.uint8, device=_dev())
        assert torch.equal(h, g.matmul_adapters(s["x"], s["w"], s["a"], s["b"], s["rows"], s["scales"], workspace=wa))
    with pytest.raises(g.GemmError):
        g.moe_experts(h, ids, gates, s["w1"], s["w2"], workspace=torch.empty(64, dtype=torch.uint8, device=_dev()))


@pytest.mark.parametrize("weights", ["w16", "mx"])
@pytest.mark.parametrize("T,E,top,H,I", [(1, 8, 3, 64, 48), (1, 16, 16, 257, 130), (5, 40, 4, 96, 33), (60, 64, 2, 128, 64)])
def test_few_tokens_by_the_layers_thin_products(g, T, E, top, H, I, weights):
    """With the layer's own choice the same bits as the layer; dropped choices add nothing."""
    rng = np.random.default_rng(T + E)
    to = lambda *s, by=1.0: torch.from_numpy((rng.standard_normal(s) / by).astype(np.float32)).to(_dev(), torch.bfloat16)  # noqa: E731
    x, router, w1, w2 = to(T, H), to(E, H, by=H ** .5), to(E, 2 * I, H, by=H ** .5), to(E, H, I, by=I ** .5)
    v1, v2 = w1, w2
    if weights == "mx":
        q1, q2 = g.mx_quantize(w1.reshape(-1, H)), g.mx_quantize(w2.reshape(-1, I))
        v1 = g.mx_dequantize(q1, dtype=torch.bfloat16).reshape(w1.shape)
        v2 = g.mx_dequantize(q2, dtype=torch.bfloat16).reshape(w2.shape)
        w1 = g.MxTensor(q1.codes.reshape(E, 2 * I, -1), q1.scales.reshape(E, 2 * I, -1), H)
        w2 = g.MxTensor(q2.codes.reshape(E, H, -1), q2.scales.reshape(E, H, -1), I)
    y, ids, gates = g.moe_layer(x, router, w1, w2, top)
    assert torch.equal(g.moe_experts(x, ids, gates, w1, w2), y)
    for keep in (0.5, 0.0):
        some = torch.where(torch.rand(ids.shape, device=_dev()) < keep, ids, torch.tensor(-1, dtype=torch.int32, device=_dev()))
        check(g.moe_experts(x, some, gates, w1, w2), reference(x, some, gates, v1, v2)["y"], (T, E, weights, keep))
    twice = ids.clone()
    twice[:, -1] = twice[:, 0]
    check(g.moe_experts(x, twice, gates, w1, w2), reference(x, twice, gates, v1, v2)["y"], (T, E, weights, "twice"))


def test_a_rows_nan_stays_in_its_row(g):
    for T, save in ((6, False), (300, False), (300, True)):
        s = _state(g, T, 64 if T == 6 else 4, 64, 48, 3, 8, torch.bfloat16)
        ids = torch.from_numpy(np.random.default_rng(2).integers(0, s["w1"].shape[0], (T, 2)).astype(np.int32)).to(_dev())
        gates = torch.rand(T, 2, device=_dev())
        want = g.moe_experts(s["x"], ids, gates, s["w1"], s["w2"], save=save)
        x = s["x"].clone()
        x[T // 2] = float("nan")
        got = g.moe_experts(x, ids, gates, s["w1"], s["w2"], save=save)
        rest = torch.arange(T, device=_dev()) != T // 2
        a, b = (got[0], want[0]) if save else (got, want)
        assert torch.equal(a[rest], b[rest]) and a[T // 2].isnan().all()
        if save:
            dx, dg, dw1, dw2 = g.moe_experts_backward(s["dy"], x, ids, gates, s["w1"], s["w2"], got[1])
            full = g.moe_experts_backward(s["dy"], s["x"], ids, gates, s["w1"], s["w2"], want[1])
            assert torch.equal(dx[rest], full[0][rest]) and torch.equal(dg[rest], full[1][rest])
            asked = torch.zeros(4, dtype=torch.bool, device=_dev())
            asked[ids[T // 2].long()] = True
            assert torch.equal(dw1[~asked], full[2][~asked]) and torch.equal(dw2[~asked], full[3][~asked])


def test_more_than_2_to_31_bytes_and_elements(g):
    """Tokens past 32-bit byte and element offsets: rows of both ends against the definition."""
    T, H, I, E = 600_000, 4096, 32, 2
    print("case: experts 2^31", flush=True)
    gen = torch.Generator(device=_dev()).manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=_dev()).normal_(generator=gen)
    w1 = (torch.randn(E, 2 * I, H, generator=gen, device=_dev()) / 64).bfloat16()
    w2 = (torch.randn(E, H, I, generator=gen, device=_dev()) / 6).bfloat16()
    ids = (torch.arange(T, device=_dev(), dtype=torch.int32) % 3 == 0).int().unsqueeze(1)
    gates = torch.rand(T, 1, generator=gen, device=_dev())
    y, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    at = torch.cat((torch.arange(50), torch.arange(T // 2, T // 2 + 50), torch.arange(T - 50, T))).to(_dev())
    ref = reference(x[at], ids[at], gates[at], w1, w2, x[at])
    check(y[at], ref["y"], "y")
    del y
    dx, dg = g.moe_experts_backward(x, x, ids, gates, w1, w2, saved, weights=False)
    check(dx[at], ref["dx"], "dx")
    check(dg[at], ref["dgates"], "dgates")
    del dx, saved
    print("case: adapters 2^31", flush=True)
    w, a, b = w1.reshape(-1, H)[:48].contiguous(), w1[:, :8].contiguous(), (torch.randn(2, 48, 8, generator=gen, device=_dev()) / 3).bfloat16()
    rows = (torch.arange(T, device=_dev(), dtype=torch.int32) % 4) - 1
    got = g.matmul_adapters(x, w, a, b, rows)
    from test_gpu_adapters import check as check_adapters
    from test_gpu_adapters import reference as adapters
    check_adapters(got[at], adapters(x[at], w, a, b, rows[at], None), "adapters")
