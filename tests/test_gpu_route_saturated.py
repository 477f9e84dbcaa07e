"""Routing where scores are rounded to 1 or 0: the order of experts."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    import tiled_fp32_gemm_03_amd as lib
    return lib


@pytest.mark.parametrize("T", [1, 3, 2000])  # a wave to a token, and four tokens to a wave
def test_groups_by_two_keys_order_experts_by_their_logits(g, T):
    print(f"case: saturated groups {T}", flush=True)
    dev = torch.device("cuda:0")
    cases = [("sigmoid", [40.0, 50.0, 60.0, 45.0, 1.0, 2.0, 3.0, 4.0], [2, 1, 3, 0]),
             ("sigmoid", [-5.0, -6.0, -7.0, -8.0, -800.0, 90.0, -900.0, 80.0], [5, 7, 4, 6]),
             ("softmax", [0.0, -800.0, -900.0, -750.0, -5.0, -5.0, -5.0, -5.0], [0, 3, 1, 2])]
    for score, z, want in cases:
        for top in (1, 3, 4):
            logits = torch.tensor([z], device=dev).repeat(T, 1)
            ids, _ = g.moe_route(logits, top, score=score, groups=2, top_groups=1, group_score="top2")
            assert torch.equal(ids, torch.tensor([want[:top]], dtype=torch.int32, device=dev).repeat(T, 1)), (score, z, top)
