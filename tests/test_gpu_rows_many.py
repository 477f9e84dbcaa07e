"""Many rows: the experts' products and adapters where sizes ask for the large tiles but rows
cannot be loaded directly (widths that are no multiple of 8, a matrix that starts in the middle
of a word, rows of fewer than 8 values), in some of a pass's products or in all; and more pairs
than are listed in one launch."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_adapters as adapters  # noqa: E402
import test_gpu_experts as experts  # noqa: E402


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


# widths odd both, H whole 16 bytes alone, I alone, both
@pytest.mark.parametrize("case", [(3001, 4, 2, 2051, 1025), (3001, 4, 2, 2056, 1026), (3001, 4, 2, 2050, 1032), (3001, 4, 2, 2056, 1032)])
def test_experts_of_many_rows(g, case):
    print(f"case: experts {case}", flush=True)
    experts._all(g, experts._make(*case, torch.bfloat16), case)


@pytest.mark.parametrize("case", [(4000, 3333, 131, 9, 5), (4000, 3336, 5, 3, 40), (3300, 4001, 520, 24, 3)])
def test_adapters_of_many_rows(g, case):
    print(f"case: adapters {case}", flush=True)
    args = adapters._make(*case, torch.bfloat16)
    ref = adapters.reference(*args)
    adapters.check(g.matmul_adapters(*args), ref, case)
    x, w, a, b, ids, scales = args
    wide = torch.zeros(x.shape[0], x.shape[1] + 3, dtype=x.dtype, device=x.device)
    wide[:, 1:-2] = x
    adapters.check(g.matmul_adapters(wide[:, 1:-2], w, a, b, ids, scales), ref, (case, "in the middle of a word"))


@pytest.mark.parametrize("case", [(22_000, 5, 3, 40, 24), (70_000, 512, 1, 24, 8), (65_537, 1, 1, 8, 9)])
def test_experts_of_more_pairs_than_one_launch_lists(g, case):
    print(f"case: experts {case}", flush=True)
    experts._all(g, experts._make(*case, torch.float16, drop=0.1), case)


@pytest.mark.parametrize("case", [(65_536, 24, 32, 8, 7), (70_001, 40, 24, 5, 300)])
def test_adapters_of_more_rows_than_one_launch_lists(g, case):
    print(f"case: adapters {case}", flush=True)
    args = adapters._make(*case, torch.float16)
    adapters.check(g.matmul_adapters(*args), adapters.reference(*args), case)


@pytest.mark.parametrize("T", [1, 61, 130, 600])
def test_adapters_past_2_to_31_bytes(g, T):
    """W and B longer than 32-bit offsets reach; columns of both ends."""
    print(f"case: adapters 2^31 {T}", flush=True)
    N, K, R, count = 131_072, 8200, 20, 511
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(T)
    make = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev).normal_(generator=gen)  # noqa: E731
    x, w, a, b = make(T, K), make(N, K).mul_(1 / 91), make(count, R, K).mul_(1 / 91), make(count, N, R).mul_(1 / 4)
    ids = torch.randint(-1, count, (T,), generator=gen, device=dev, dtype=torch.int32)
    ids[0] = count - 1
    y = g.matmul_adapters(x, w, a, b, ids)
    at = torch.cat((torch.arange(70), torch.arange(N // 2, N // 2 + 50), torch.arange(N - 70, N))).to(dev)
    adapters.check(y[:, at], adapters.reference(x, w[at], a, b[:, at].contiguous(), ids, None), T)


@pytest.mark.parametrize("T", [2, 300])
def test_experts_past_2_to_31_bytes(g, T):
    """Both weights and their gradients longer than 32-bit offsets reach."""
    print(f"case: experts 2^31 {T}", flush=True)
    E, H, I = 144, 2048, 4096
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(T)
    make = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev).normal_(generator=gen)  # noqa: E731
    x, dy, w1, w2 = make(T, H), make(T, H), make(E, 2 * I, H).mul_(1 / 45), make(E, H, I).mul_(1 / 64)
    few = torch.tensor([0, 70, E - 1], device=dev)
    of = torch.randint(0, 3, (T, 2), generator=gen, device=dev)
    ids, gates = few[of].int(), torch.rand(T, 2, generator=gen, device=dev)
    ref = experts.reference(x, of.int(), gates, w1[few], w2[few], dy)
    experts.check(g.moe_experts(x, ids, gates, w1, w2), ref["y"], (T, "y alone"))
    y, saved = g.moe_experts(x, ids, gates, w1, w2, save=True)
    experts.check(y, ref["y"], (T, "y"))
    dx, dgates, dw1, dw2 = g.moe_experts_backward(dy, x, ids, gates, w1, w2, saved)
    for name, v in (("dx", dx), ("dgates", dgates), ("dw1", dw1[few]), ("dw2", dw2[few])):
        experts.check(v, ref[name], (T, name))
    for dw in (dw1, dw2):
        assert not dw[1:70].any() and not dw[71:E - 1].any()
