"""The MX operators' front end on the host: sizes, argument checks in order
(nothing is launched, no GPU needed) and the numpy oracle's pins."""
import numpy as np
import pytest

import tiled_fp32_gemm_03_amd as g
from oracle import mx

torch = pytest.importorskip("torch")

OK, DIM, LD, NULL, MISALIGNED, CONFIG, ARG = 0, 1, 2, 3, 6, 7, 8
L = g._lib


def test_row_sizes():
    for K in (0, 1, 31, 32, 33, 511, 512, 513, 4097, 2**31 - 1):
        assert g.gemm_mx_code_bytes(K) == mx.code_bytes(K) == 16 * -(-K // 32)
        assert g.gemm_mx_scale_bytes(K) == mx.scale_bytes(K)
        assert g.gemm_mx_scale_bytes(K) >= -(-K // 32)


def _quant(rows=4, K=64, X=256, ldx=64, fmt=2, along=0, codes=256, ld=32, scales=256, lds=16,
           fn="gemm_mx_quantize"):
    if fn == "gemm_mx_quantize":
        return L.gemm_mx_quantize(rows, K, X or None, ldx, fmt, along, codes or None, ld,
                                  scales or None, lds, None)
    return L.gemm_mx_dequantize(rows, K, codes or None, ld, scales or None, lds, X or None, ldx,
                                fmt, along, None)


@pytest.mark.parametrize("fn", ["gemm_mx_quantize", "gemm_mx_dequantize"])
def test_conversion_refusals(fn):
    def q(**kw):
        return _quant(fn=fn, **kw)
    assert q(rows=-1) == DIM and q(K=-1) == DIM
    assert q(fmt=3) == ARG and q(fmt=-1) == ARG and q(along=2) == ARG
    assert q(ldx=63) == LD
    assert q(along=1, ldx=3) == LD
    assert q(ld=16) == LD and q(lds=0) == LD and q(K=0, ld=0) == LD
    assert q(ld=40) == MISALIGNED and q(lds=24) == MISALIGNED
    assert q(X=0) == NULL and q(codes=0) == NULL and q(scales=0) == NULL
    assert q(X=258) == MISALIGNED and q(fmt=0, X=257) == MISALIGNED
    assert q(codes=264) == MISALIGNED and q(scales=260) == MISALIGNED
    # nothing to do: no pointers needed
    assert q(rows=0, X=0, codes=0, scales=0) == OK
    assert q(K=0, X=0, codes=0, scales=0) == OK


def _prod(M=4, N=4, K=64, A=256, lda=32, SA=256, ldsa=16, B=256, ldb=32, SB=256, ldsb=16, C=256,
          ldc=4, fmt=2, config=-1):
    return L.gemm_mx(M, N, K, A or None, lda, SA or None, ldsa, B or None, ldb, SB or None, ldsb,
                     C or None, ldc, fmt, config, None)


def test_product_refusals():
    assert _prod(M=-1) == DIM and _prod(N=-1) == DIM and _prod(K=-1) == DIM
    for name in ("lda", "ldb"):
        assert _prod(**{name: 16}) == LD and _prod(**{name: 40}) == MISALIGNED
    for name in ("ldsa", "ldsb"):
        assert _prod(**{name: 0}) == LD and _prod(**{name: 24}) == MISALIGNED
    assert _prod(ldc=3) == LD
    assert _prod(fmt=3) == ARG
    assert _prod(config=-2) == CONFIG and _prod(config=g.gemm_mx_num_configs()) == CONFIG
    for name in ("A", "SA", "B", "SB", "C"):
        assert _prod(**{name: 0}) == NULL
    for name in ("A", "SA", "B", "SB"):
        assert _prod(**{name: 264}) == MISALIGNED
    assert _prod(C=258) == MISALIGNED and _prod(C=257, fmt=0) == MISALIGNED
    assert _prod(M=0, A=0, SA=0, B=0, SB=0, C=0) == OK
    assert _prod(N=0, A=0, SA=0, B=0, SB=0, C=0) == OK


def _a16(M=4, N=4, K=64, A=256, lda=64, af=0, B=256, ldb=32, SB=256, ldsb=16, C=256, ldc=4, fmt=2):
    return L.gemm_mx_a16(M, N, K, A or None, lda, af, B or None, ldb, SB or None, ldsb, C or None,
                         ldc, fmt, None)


def test_a16_refusals():
    assert _a16(M=-1) == DIM and _a16(N=-1) == DIM and _a16(K=-1) == DIM
    assert _a16(lda=63) == LD and _a16(ldb=16) == LD and _a16(ldsb=0) == LD and _a16(ldc=3) == LD
    assert _a16(ldb=40) == MISALIGNED and _a16(ldsb=24) == MISALIGNED
    assert _a16(af=2) == ARG and _a16(af=-1) == ARG and _a16(fmt=3) == ARG
    for name in ("A", "B", "SB", "C"):
        assert _a16(**{name: 0}) == NULL
    assert _a16(A=257) == MISALIGNED and _a16(B=264) == MISALIGNED and _a16(SB=264) == MISALIGNED
    assert _a16(M=0, A=0, B=0, SB=0, C=0) == OK


def test_tile_query():
    for cfg in range(-1, g.gemm_mx_num_configs()):
        t = g.gemm_mx_tile(cfg, 300, 200, 100)
        assert t["BM"] > 0 and t["BN"] > 0 and t["BK"] % 32 == 0 and t["threads"] % 64 == 0
        assert cfg == -1 or t["config"] == cfg
    with pytest.raises(g.GemmError):
        g.gemm_mx_tile(99, 1, 1, 1)
    with pytest.raises(g.GemmError):
        g.gemm_mx_tile(-1, -1, 1, 1)


def _empty(rows, K):
    return g.MxTensor(torch.zeros(rows, mx.code_bytes(K), dtype=torch.uint8),
                      torch.zeros(rows, mx.scale_bytes(K), dtype=torch.uint8), K)


def test_mx_tensor_refusals():
    q = _empty(3, 100)
    assert q.shape == (3, 100)
    with pytest.raises(TypeError):
        g.MxTensor(q.codes.int(), q.scales, 100)
    with pytest.raises(ValueError):
        g.MxTensor(q.codes[:, :48], q.scales, 100)
    with pytest.raises(ValueError):
        g.MxTensor(q.codes, q.scales[:2], 100)
    with pytest.raises(ValueError):
        g.MxTensor(q.codes, q.scales, -1)


def test_binding_refusals_on_host_tensors():
    """Host tensors and wrong types are refused before anything is launched."""
    q = _empty(3, 100)
    with pytest.raises(TypeError):
        g.mx_quantize(torch.zeros(3, 100))
    with pytest.raises(TypeError):
        g.mx_quantize(torch.zeros(3, 100, dtype=torch.float64))
    with pytest.raises(TypeError):
        g.mx_dequantize(q)
    with pytest.raises(TypeError):
        g.mx_dequantize(q, dtype=torch.float64)
    with pytest.raises(TypeError):
        g.matmul_mx(q, q)
    with pytest.raises(TypeError):
        g.matmul_mx(q, torch.zeros(3, 100))
    with pytest.raises(TypeError):
        g.matmul_mx(q, q, dtype=torch.int32)


# ---- the mixture-of-experts layer ------------------------------------------------


def _moe(T=2, E=4, top=2, H=64, I=32, X=256, ldx=64, R=256, ldr=64, fmt=0, W1=256, ld1=64, S1=0,
         lds1=0, W2=256, ld2=32, S2=0, lds2=0, weights=0, renorm=1, Y=256, ldy=64, yf=0, ids=0,
         gates=0, ws=256, ws_bytes=1 << 20):
    p = lambda v: v or None  # noqa: E731
    return L.gemm_moe(T, E, top, H, I, p(X), ldx, p(R), ldr, fmt, p(W1), ld1, p(S1), lds1, p(W2),
                      ld2, p(S2), lds2, weights, renorm, p(Y), ldy, yf, p(ids), p(gates), p(ws),
                      ws_bytes, None)


def test_moe_refusals():
    workspace = 9
    for kw in (dict(T=-1), dict(E=-1), dict(top=-1), dict(H=0), dict(I=0), dict(H=-5)):
        assert _moe(**kw) == DIM, kw
    for kw in (dict(T=257), dict(E=513), dict(top=0), dict(top=5), dict(E=32, top=17),
               dict(H=(1 << 24) + 1), dict(fmt=2), dict(yf=1), dict(weights=2), dict(yf=3)):
        assert _moe(**kw) == ARG, kw
    for kw in (dict(ldx=63), dict(ldr=63), dict(ldy=63), dict(ld1=63), dict(ld2=31)):
        assert _moe(**kw) == LD, kw
    mx_kw = dict(weights=1, ld1=32, lds1=16, ld2=16, lds2=16, S1=256, S2=256)
    for kw in (dict(ld1=16), dict(lds1=0), dict(ld2=0), dict(lds2=0)):
        assert _moe(**{**mx_kw, **kw}) == LD, kw
    for kw in (dict(ld1=40), dict(lds1=24), dict(W1=264), dict(S2=264)):
        assert _moe(**{**mx_kw, **kw}) == MISALIGNED, kw
    for name in ("X", "R", "W1", "W2", "Y"):
        assert _moe(**{name: 0}) == NULL, name
        assert _moe(**{name: 257}) == MISALIGNED, name
    assert _moe(**{**mx_kw, "S1": 0}) == NULL
    assert _moe(yf=2, Y=258) == MISALIGNED
    assert _moe(ids=258) == MISALIGNED and _moe(gates=258) == MISALIGNED
    need = g.gemm_moe_workspace_bytes(2, 4, 2, 64, 32)
    assert need > 0 and need % 16 == 0
    assert _moe(ws=0) == workspace and _moe(ws=264) == workspace and _moe(ws_bytes=need - 1) == workspace
    assert _moe(T=0, X=0, R=0, W1=0, W2=0, Y=0, ws=0) == OK
    assert g.gemm_moe_workspace_bytes(257, 4, 2, 64, 32) == -1
    assert g.gemm_moe_workspace_bytes(1, 4, 5, 64, 32) == -1


def test_moe_binding_refusals_on_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        g.moe_layer(x, torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 64),
                    torch.zeros(4, 64, 32), 2)
    with pytest.raises(TypeError):
        g.moe_layer(x.float(), x, x, x, 1)


# ---- the oracle's own pins -----------------------------------------------------


def test_oracle_rounds_to_the_nearest_element():
    """Against a search over all elements, ties to the even code."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 96)) * np.ldexp(1.0, rng.integers(-20, 20, (40, 96)))
    x[0, :32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4)  # the midpoints, scale 1
    codes, scales = mx.quantize(x)
    v = mx.values(codes, scales, 96)
    for r in range(40):
        for b in range(3):
            unit = np.ldexp(1.0, int(scales[r, b]) - 127)
            m = np.abs(x[r, 32 * b:32 * b + 32]).max()
            assert 4 * unit <= m < 8 * unit
            for k in range(32 * b, 32 * b + 32):
                d = np.abs(np.abs(x[r, k]) / unit - mx.ELEMENTS)
                best = np.flatnonzero(d == d.min())
                want = best[best % 2 == 0][0] if len(best) > 1 else best[0]
                assert abs(v[r, k]) == mx.ELEMENTS[want] * unit, (r, k)
                assert v[r, k] == 0 or np.sign(v[r, k]) == np.sign(x[r, k])


def test_oracle_fixes_what_is_representable():
    rng = np.random.default_rng(6)
    codes, scales = mx.random_rows(rng, 5, 96)
    codes[:, 0::16] |= 7  # an element of 6 in every block, so its scale is found again
    v = mx.values(codes, scales, 96)
    again, s2 = mx.quantize(v)
    assert np.array_equal(s2[:, :3], scales[:, :3])
    assert np.array_equal(mx.values(again, s2, 96), v)


def test_oracle_bf16_rounding_is_torch_s():
    rng = np.random.default_rng(7)
    x = (rng.standard_normal(4000) * np.exp2(rng.integers(-140, 127, 4000))).astype(np.float32)
    x = np.concatenate([x, np.float32([0, -0.0, np.inf, -np.inf, 3.4e38, 1e-45])])
    want = torch.from_numpy(x).bfloat16().double().numpy()
    assert np.array_equal(mx.round_to(x.astype(np.float64), "bf16"), want)


def test_the_choice_of_entry_by_size():
    """Sizes where every entry was timed: the fastest, or one within a tenth."""
    for (M, N, K), want in {(17, 64, 16384): 3, (33, 8192, 512): 0, (64, 2048, 16384): 3,
                            (128, 8192, 4096): 2, (256, 512, 16384): 3, (256, 2048, 4096): 2,
                            (256, 8192, 512): 2, (300, 300, 300): 3, (700, 1000, 8000): 2,
                            (1024, 8192, 4096): 2, (4096, 4096, 4096): 1}.items():
        assert g.gemm_mx_tile(-1, M, N, K)["config"] == want, (M, N, K)
