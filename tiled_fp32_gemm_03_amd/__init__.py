"""Python binding of the gfx950 fp32 matrix-multiply library ``libgemm_f32.so``.

Argument marshalling only: every step of C = A x B runs in the library's HIP
kernels.  If the library is missing the import fails loudly; there is no
CPU or PyTorch fallback.

Raw C-ABI mirrors (same names and argument order as ``include/gemm_f32.h``):
  gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, variant, stream)
  gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, variant, config, stream)
  gemm_f32_tile(variant, config, M, N, K) -> dict
  gemm_f32_num_configs(variant), gemm_f32_status_string(rc), gemm_f32_version()
  gemm_f32_probe_stream(kind, n, x, y, z, stream)      (include/gemm_f32_probes.h)
  gemm_f32_probe_mfma(workgroups, iters, out, stream), gemm_f32_probe_mfma_flops(...)
  gemm_f32_probe_mfma16(shape, workgroups, iters, out, stream), gemm_f32_probe_mfma16_flops(...)
  gemm_f32_probe_valu(workgroups, iters, out, stream), gemm_f32_probe_valu_flops(...)
  gemm_f32_probe_lds(workgroups, iters, out, stream), gemm_f32_probe_lds_bytes(...)
  gemm_f32_probe_fused(mode, workgroups, trips, out, out_bytes, clocks, stream),
  gemm_f32_probe_fused_flops(mode, ...), gemm_f32_probe_fused_bytes(mode, ...)
  gemm_f32_device_props(device) -> dict
  gemm_f32_splitk(M, N, K, A, lda, B, ldb, C, ldc, config, splits, workspace,
                  workspace_bytes, stream), gemm_f32_splitk_plan(M, N, K, config, splits)
  gemm_f32_splitk_noalloc(M, N, K, A, lda, B, ldb, C, ldc, config, splits, stream)
  gemm_mixed(M, N, K, A, lda, B, ldb, C, ldc, format, config, stream)
  gemm_mixed_tile(config, M, N, K) -> dict, gemm_mixed_num_configs()
                                                        (include/gemm_mixed.h)
  gemm_mx_quantize(rows, K, X, ldx, format, along, codes, ld, scales, lds, stream)
  gemm_mx_dequantize(rows, K, codes, ld, scales, lds, Y, ldy, format, along, stream)
  gemm_mx(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_format, config, stream)
  gemm_mx_tile(config, M, N, K) -> dict, gemm_mx_num_configs()
  gemm_mx_a16(M, N, K, A, lda, a_format, B, ldb, SB, ldsb, C, ldc, c_format, stream)
  gemm_mx_code_bytes(K), gemm_mx_scale_bytes(K)         (include/gemm_mx.h)
  gemm_moe(T, E, top, H, I, X, ldx, R, ldr, format, W1, ld1, S1, lds1, W2, ld2, S2, lds2, weights,
           renormalize, Y, ldy, y_format, ids, gates, workspace, workspace_bytes, stream),
  gemm_moe_workspace_bytes(T, E, top, H, I)             (include/gemm_moe.h)
  gemm_moe_route(T, E, top, Z, ldz, format, score, bias, groups, top_groups, group_score,
                 renormalize, scale, ids, gates, stream),
  gemm_moe_route_backward(T, E, top, dgates, Z, ldz, format, score, renormalize, scale, ids, dZ,
                          lddz, stream)                 (include/gemm_route.h)
  gemm_experts(T, E, top, H, I, X, ldx, ids, gates, format, W1, ld1, S1, lds1, W2, ld2, S2, lds2,
               weights, Y, ldy, saved, workspace, workspace_bytes, stream),
  gemm_experts_backward(T, E, top, H, I, dY, lddy, X, ldx, ids, gates, format, W1, ld1, W2, ld2,
                        saved, dX, lddx, dgates, dW1, lddw1, dW2, lddw2, workspace,
                        workspace_bytes, stream),
  gemm_experts_workspace_bytes(T, E, top, H, I, backward)  (include/gemm_experts.h)
  gemm_adapters(T, N, K, R, count, X, ldx, W, ldw, A, lda, B, ldb, ids, scales, format, Y, ldy,
                workspace, workspace_bytes, stream),
  gemm_adapters_workspace_bytes(T, N, K, R, count)      (include/gemm_adapters.h)
Pointers are device addresses (ints); ``stream`` is a hipStream_t as int
(0 = null stream).  A non-zero status raises ``GemmError``.

Tensor conveniences: ``matmul(A, B, out=None, variant="prod", config=-1)``
takes float32 CUDA tensors whose last stride is 1 and passes ``stride(0)`` as
the leading dimension, on torch's current stream.  ``matmul_mixed(A, B,
out=None, config=-1)`` does the same for bfloat16 or float16 tensors (fp32
result); ``format`` names the 16-bit format when A and B hold raw codes
(int16 / uint16).  ``matmul_splitk(A, B, out=None, config=-1, splits=0,
workspace=None)`` runs the split-K form; it allocates the workspace as a torch
tensor when none is given.

Every one of these and of the calls below takes ``stream``, a hipStream_t as int,
in place of torch's current stream; results and workspaces that the call allocates
then belong to that stream, as inside ``torch.cuda.stream``.

4-bit microscaled (MX) matrices are ``MxTensor``s, rows of K values in blocks
of 32 along K.  ``mx_quantize(X, along="rows")`` makes one from a float32,
bfloat16 or float16 matrix; ``along="columns"`` takes its columns as the rows
(a product's right operand).  ``mx_dequantize(q, dtype, along)`` reads the
values back.  ``matmul_mx(A, B, dtype=torch.float32)`` is the product of the
rows of A (an ``MxTensor``, or a bfloat16 or float16 matrix) with the rows of
the ``MxTensor`` B, C[i][j] = sum_k A[i][k] B[j][k].

``moe_layer(X, router, w1, w2, top)`` is a mixture-of-experts layer for a few
tokens, the experts' weights being 16-bit tensors or stacks of MX matrices; it
returns the result, the chosen experts and their gates.

The same in parts, for other routers, any number of tokens and training:
``moe_route(logits, top)`` chooses experts and gates from logits (softmax or
sigmoid scores, a bias for balance, groups of experts), ``moe_experts(X, ids,
gates, w1, w2)`` is the experts' products for a choice, and
``moe_route_backward`` and ``moe_experts_backward`` are their gradients.

``matmul_adapters(X, w, a, b, ids)`` is a shared projection with low-rank adapters
of many requests, one to a row or none.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "GemmError", "VARIANTS", "config_name", "PROBE_COPY", "PROBE_FILL", "PROBE_VADD",
    "gemm_f32", "gemm_f32_ex", "gemm_f32_tile", "gemm_f32_num_configs",
    "gemm_f32_status_string", "gemm_f32_version", "gemm_f32_last_error", "gemm_f32_probe_stream",
    "gemm_f32_probe_mfma", "gemm_f32_probe_mfma_flops", "gemm_f32_probe_mfma16",
    "gemm_f32_probe_mfma16_flops", "gemm_f32_probe_valu",
    "gemm_f32_probe_valu_flops", "gemm_f32_probe_lds", "gemm_f32_probe_lds_bytes",
    "gemm_f32_probe_fused", "gemm_f32_probe_fused_flops", "gemm_f32_probe_fused_bytes",
    "FUSED_BOTH", "FUSED_MFMA", "FUSED_STORE",
    "gemm_f32_device_props", "matmul",
    "gemm_f32_splitk", "gemm_f32_splitk_plan", "matmul_splitk", "gemm_f32_splitk_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "gemm_mixed", "gemm_mixed_tile", "gemm_mixed_num_configs", "matmul_mixed", "MIXED_FORMATS",
    "mixed_config_name",
    "MxTensor", "MX_FORMATS", "MX_ALONG", "mx_quantize", "mx_dequantize", "matmul_mx",
    "gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx", "gemm_mx_tile", "gemm_mx_num_configs",
    "gemm_mx_a16", "gemm_mx_code_bytes", "gemm_mx_scale_bytes",
    "gemm_moe", "gemm_moe_workspace_bytes", "moe_layer", "MOE_WEIGHTS",
    "gemm_moe_route", "gemm_moe_route_backward", "moe_route", "moe_route_backward",
    "ROUTE_SCORES", "ROUTE_GROUP_SCORES",
    "gemm_experts", "gemm_experts_backward", "gemm_experts_workspace_bytes", "moe_experts",
    "moe_experts_backward",
    "gemm_adapters", "gemm_adapters_workspace_bytes", "matmul_adapters",
    "library_path",
    "exported_symbols",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgemm_f32.so")

# One HIP runtime per process: PyTorch ships its own libamdhip64 (same
# soname).  Loading torch first makes this library bind to that copy instead
# of pulling in a second runtime from /opt/rocm, which could not launch on
# memory that torch's runtime allocated.
import torch  # noqa: E402,F401

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is not built; run __graft_entry__.build() or "
        "python tiled_fp32_gemm_03_amd/build_lib.py (needs ROCm hipcc)")

_lib = ctypes.CDLL(_LIB_PATH)

_i = ctypes.c_int
_ll = ctypes.c_longlong
_f = ctypes.c_float
_p = ctypes.c_void_p
_ip = ctypes.POINTER(ctypes.c_int)

_SIGS = {
    "gemm_f32": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _i, _p], _i),
    "gemm_f32_ex": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p], _i),
    "gemm_f32_num_configs": ([_i], _i),
    "gemm_f32_tile": ([_i, _i, _i, _i, _i, _ip, _ip, _ip, _ip, _ip], _i),
    "gemm_f32_status_string": ([_i], ctypes.c_char_p),
    "gemm_f32_version": ([], ctypes.c_char_p),
    "gemm_f32_last_error": ([], ctypes.c_char_p),
    "gemm_f32_probe_stream": ([_i, _ll, _p, _p, _p, _p], _i),
    "gemm_f32_probe_mfma": ([_i, _i, _p, _p], _i),
    "gemm_f32_probe_mfma_flops": ([_i, _i], _ll),
    "gemm_f32_probe_mfma16": ([_i, _i, _i, _p, _p], _i),
    "gemm_f32_probe_mfma16_flops": ([_i, _i, _i], _ll),
    "gemm_f32_probe_valu": ([_i, _i, _p, _p], _i),
    "gemm_f32_probe_valu_flops": ([_i, _i], _ll),
    "gemm_f32_probe_lds": ([_i, _i, _p, _p], _i),
    "gemm_f32_splitk": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p, _ll, _p], _i),
    "gemm_f32_splitk_plan": ([_i, _i, _i, _i, _i, _ip, _ip, _ip, ctypes.POINTER(_ll)], _i),
    "gemm_f32_splitk_noalloc": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p], _i),
    "gemm_mixed": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p], _i),
    "gemm_mixed_num_configs": ([], _i),
    "gemm_mixed_tile": ([_i, _i, _i, _i, _ip, _ip, _ip, _ip, _ip], _i),
    "gemm_mx_code_bytes": ([_i], _ll),
    "gemm_mx_scale_bytes": ([_i], _ll),
    "gemm_mx_quantize": ([_i, _i, _p, _i, _i, _i, _p, _i, _p, _i, _p], _i),
    "gemm_mx_dequantize": ([_i, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p], _i),
    "gemm_mx": ([_i, _i, _i, _p, _i, _p, _i, _p, _i, _p, _i, _p, _i, _i, _i, _p], _i),
    "gemm_mx_num_configs": ([], _i),
    "gemm_mx_tile": ([_i, _i, _i, _i, _ip, _ip, _ip, _ip, _ip], _i),
    "gemm_mx_a16": ([_i, _i, _i, _p, _i, _i, _p, _i, _p, _i, _p, _i, _i, _p], _i),
    "gemm_moe_workspace_bytes": ([_i, _i, _i, _i, _i], _ll),
    "gemm_moe": ([_i, _i, _i, _i, _i, _p, _i, _p, _i, _i, _p, _i, _p, _i, _p, _i, _p, _i, _i, _i,
                  _p, _i, _i, _p, _p, _p, _ll, _p], _i),
    "gemm_moe_route": ([_i, _i, _i, _p, _i, _i, _i, _p, _i, _i, _i, _i, _f, _p, _p, _p], _i),
    "gemm_moe_route_backward": ([_i, _i, _i, _p, _p, _i, _i, _i, _i, _f, _p, _p, _i, _p], _i),
    "gemm_experts_workspace_bytes": ([_i, _i, _i, _i, _i, _i], _ll),
    "gemm_experts": ([_i, _i, _i, _i, _i, _p, _i, _p, _p, _i, _p, _i, _p, _i, _p, _i, _p, _i, _i,
                      _p, _i, _p, _p, _ll, _p], _i),
    "gemm_experts_backward": ([_i, _i, _i, _i, _i, _p, _i, _p, _i, _p, _p, _i, _p, _i, _p, _i, _p,
                               _p, _i, _p, _p, _i, _p, _i, _p, _ll, _p], _i),
    "gemm_adapters_workspace_bytes": ([_i, _i, _i, _i, _i], _ll),
    "gemm_adapters": ([_i, _i, _i, _i, _i, _p, _i, _p, _i, _p, _i, _p, _i, _p, _p, _i, _p, _i, _p,
                       _ll, _p], _i),
    "gemm_f32_probe_lds_bytes": ([_i, _i], _ll),
    "gemm_f32_device_props": ([_i, _ip, _ip, _ip, _ip, _ip], _i),
    "gemm_f32_probe_fused": ([_i, _i, _i, _p, _ll, _p, _p], _i),
    "gemm_f32_probe_fused_flops": ([_i, _i, _i], _ll),
    "gemm_f32_probe_fused_bytes": ([_i, _i, _i], _ll),
}
for _name, (_args, _ret) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _ret

# Variant ids of include/gemm_f32.h.
VARIANTS = {"naive": 0, "tiled": 1, "prod": 2, "tiled32": 3, "tiled4": 4, "tiled32_pad": 5,
            "valu": 6}
PROBE_COPY, PROBE_FILL, PROBE_VADD = 0, 1, 2
FUSED_BOTH, FUSED_MFMA, FUSED_STORE = 0, 1, 2
# GEMM_F32_NOALLOC_SCRATCH_BYTES of include/gemm_f32.h: the fixed split-K
# scratch of gemm_f32_splitk_noalloc on each GPU.
NOALLOC_SCRATCH_BYTES = 64 << 20
# Input formats of include/gemm_mixed.h.
MIXED_FORMATS = {"bf16": 0, "f16": 1}
# Formats of unquantised matrices and the ways blocks run (include/gemm_mx.h).
MX_FORMATS = {"bf16": 0, "f16": 1, "f32": 2}
MX_ALONG = {"rows": 0, "columns": 1}
# Kinds of expert weights (include/gemm_moe.h).
MOE_WEIGHTS = {"w16": 0, "mx": 1}
# Scores of experts and of their groups (include/gemm_route.h).
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
ROUTE_GROUP_SCORES = {"max": 0, "top2": 1}
_MX_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = gemm_f32_last_error() if status == 5 else ""
        super().__init__(f"{where}: status {status} ({gemm_f32_status_string(status)})"
                         + (f": {detail}" if detail else ""))


def library_path() -> str:
    return _LIB_PATH


def exported_symbols() -> tuple[str, ...]:
    return tuple(_SIGS)


def _variant(v) -> int:
    if isinstance(v, str):
        try:
            return VARIANTS[v]
        except KeyError:
            raise ValueError(f"unknown variant {v!r}; one of {sorted(VARIANTS)}") from None
    return int(v)


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise GemmError(rc, where)


def gemm_f32_status_string(status: int) -> str:
    return _lib.gemm_f32_status_string(int(status)).decode()


def gemm_f32_last_error() -> str:
    return _lib.gemm_f32_last_error().decode()


def gemm_f32_version() -> str:
    return _lib.gemm_f32_version().decode()


def gemm_f32_num_configs(variant) -> int:
    return int(_lib.gemm_f32_num_configs(_variant(variant)))


def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, variant, stream=0) -> None:
    rc = _lib.gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, _variant(variant), stream or None)
    _check(rc, "gemm_f32")


def gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, variant, config, stream=0) -> None:
    rc = _lib.gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, _variant(variant), int(config),
                          stream or None)
    _check(rc, "gemm_f32_ex")


def gemm_f32_tile(variant, config, M, N, K) -> dict:
    vals = [ctypes.c_int(0) for _ in range(5)]
    rc = _lib.gemm_f32_tile(_variant(variant), int(config), M, N, K,
                            *[ctypes.byref(v) for v in vals])
    _check(rc, "gemm_f32_tile")
    bm, bn, bk, nt, chosen = (v.value for v in vals)
    return {"BM": bm, "BN": bn, "BK": bk, "threads": nt, "config": chosen}


def gemm_f32_probe_stream(kind, n, x, y, z, stream=0) -> None:
    _check(_lib.gemm_f32_probe_stream(int(kind), int(n), x or None, y or None, z or None,
                                      stream or None), "gemm_f32_probe_stream")


def gemm_f32_probe_mfma(workgroups, iters, out, stream=0) -> None:
    _check(_lib.gemm_f32_probe_mfma(int(workgroups), int(iters), out or None, stream or None),
           "gemm_f32_probe_mfma")


def gemm_f32_probe_mfma_flops(workgroups, iters) -> int:
    return int(_lib.gemm_f32_probe_mfma_flops(int(workgroups), int(iters)))


def gemm_f32_probe_mfma16(shape, workgroups, iters, out, stream=0) -> None:
    _check(_lib.gemm_f32_probe_mfma16(int(shape), int(workgroups), int(iters), out or None,
                                      stream or None), "gemm_f32_probe_mfma16")


def gemm_f32_probe_mfma16_flops(shape, workgroups, iters) -> int:
    return int(_lib.gemm_f32_probe_mfma16_flops(int(shape), int(workgroups), int(iters)))


def gemm_f32_probe_valu(workgroups, iters, out, stream=0) -> None:
    _check(_lib.gemm_f32_probe_valu(int(workgroups), int(iters), out or None, stream or None),
           "gemm_f32_probe_valu")


def gemm_f32_probe_valu_flops(workgroups, iters) -> int:
    return int(_lib.gemm_f32_probe_valu_flops(int(workgroups), int(iters)))


def gemm_f32_probe_lds(workgroups, iters, out, stream=0) -> None:
    _check(_lib.gemm_f32_probe_lds(int(workgroups), int(iters), out or None, stream or None),
           "gemm_f32_probe_lds")


def gemm_f32_probe_lds_bytes(workgroups, iters) -> int:
    return int(_lib.gemm_f32_probe_lds_bytes(int(workgroups), int(iters)))


def gemm_f32_probe_fused(mode, workgroups, trips, out, out_bytes, clocks=0, stream=0) -> None:
    _check(_lib.gemm_f32_probe_fused(int(mode), int(workgroups), int(trips), out or None,
                                     int(out_bytes), clocks or None, stream or None),
           "gemm_f32_probe_fused")


def gemm_f32_probe_fused_flops(mode, workgroups, trips) -> int:
    return int(_lib.gemm_f32_probe_fused_flops(int(mode), int(workgroups), int(trips)))


def gemm_f32_probe_fused_bytes(mode, workgroups, trips) -> int:
    return int(_lib.gemm_f32_probe_fused_bytes(int(mode), int(workgroups), int(trips)))


def gemm_f32_device_props(device: int = 0) -> dict:
    vals = [ctypes.c_int(0) for _ in range(5)]
    _check(_lib.gemm_f32_device_props(int(device), *[ctypes.byref(v) for v in vals]),
           "gemm_f32_device_props")
    cus, clk, lds, wave, l2 = (v.value for v in vals)
    return {"cus": cus, "clock_mhz": clk / 1000.0, "lds_bytes_per_cu": lds, "wave_size": wave,
            "l2_bytes": l2}


def gemm_f32_splitk_plan(M, N, K, config=-1, splits=0) -> dict:
    ints = [ctypes.c_int(0) for _ in range(3)]
    ws = ctypes.c_longlong(0)
    rc = _lib.gemm_f32_splitk_plan(M, N, K, int(config), int(splits),
                                   *[ctypes.byref(v) for v in ints], ctypes.byref(ws))
    _check(rc, "gemm_f32_splitk_plan")
    cfg, used, kc = (v.value for v in ints)
    return {"config": cfg, "splits": used, "kc": kc, "workspace_bytes": ws.value}


def gemm_f32_splitk(M, N, K, A, lda, B, ldb, C, ldc, config, splits, workspace,
                    workspace_bytes, stream=0) -> None:
    rc = _lib.gemm_f32_splitk(M, N, K, A or None, lda, B or None, ldb, C or None, ldc,
                              int(config), int(splits), workspace or None, int(workspace_bytes),
                              stream or None)
    _check(rc, "gemm_f32_splitk")


def gemm_f32_splitk_noalloc(M, N, K, A, lda, B, ldb, C, ldc, config=-1, splits=0,
                            stream=0) -> None:
    rc = _lib.gemm_f32_splitk_noalloc(M, N, K, A or None, lda, B or None, ldb, C or None, ldc,
                                      int(config), int(splits), stream or None)
    _check(rc, "gemm_f32_splitk_noalloc")


def _format(fmt) -> int:
    if isinstance(fmt, str):
        try:
            return MIXED_FORMATS[fmt]
        except KeyError:
            raise ValueError(f"unknown 16-bit format {fmt!r}; one of {sorted(MIXED_FORMATS)}") from None
    return int(fmt)


def gemm_mixed(M, N, K, A, lda, B, ldb, C, ldc, format, config=-1, stream=0) -> None:
    rc = _lib.gemm_mixed(M, N, K, A or None, lda, B or None, ldb, C or None, ldc,
                         _format(format), int(config), stream or None)
    _check(rc, "gemm_mixed")


def gemm_mixed_num_configs() -> int:
    return int(_lib.gemm_mixed_num_configs())


def gemm_mixed_tile(config, M, N, K) -> dict:
    vals = [ctypes.c_int(0) for _ in range(5)]
    rc = _lib.gemm_mixed_tile(int(config), M, N, K, *[ctypes.byref(v) for v in vals])
    _check(rc, "gemm_mixed_tile")
    bm, bn, bk, nt, chosen = (v.value for v in vals)
    return {"BM": bm, "BN": bn, "BK": bk, "threads": nt, "config": chosen}


_INT_MAX = 0x7fffffff


def _fits(*sizes) -> None:
    """Refuses what the C interface's int does not hold (ctypes would cut it)."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX - 1:
        raise ValueError(f"sizes and pitches must be below 2^31, not {max(sizes, key=abs)}")


def _mx_format(fmt) -> int:
    if isinstance(fmt, str):
        try:
            return MX_FORMATS[fmt]
        except KeyError:
            raise ValueError(f"unknown format {fmt!r}; one of {sorted(MX_FORMATS)}") from None
    return int(fmt)


def _along(along) -> int:
    if isinstance(along, str):
        try:
            return MX_ALONG[along]
        except KeyError:
            raise ValueError(f"unknown direction {along!r}; one of {sorted(MX_ALONG)}") from None
    return int(along)


def gemm_mx_code_bytes(K) -> int:
    _fits(int(K))
    return int(_lib.gemm_mx_code_bytes(int(K)))


def gemm_mx_scale_bytes(K) -> int:
    _fits(int(K))
    return int(_lib.gemm_mx_scale_bytes(int(K)))


def gemm_mx_quantize(rows, K, X, ldx, format, along, codes, ld, scales, lds, stream=0) -> None:
    _fits(rows, K, ldx, ld, lds)
    _check(_lib.gemm_mx_quantize(rows, K, X or None, ldx, _mx_format(format), _along(along),
                                 codes or None, ld, scales or None, lds, stream or None),
           "gemm_mx_quantize")


def gemm_mx_dequantize(rows, K, codes, ld, scales, lds, Y, ldy, format, along, stream=0) -> None:
    _fits(rows, K, ld, lds, ldy)
    _check(_lib.gemm_mx_dequantize(rows, K, codes or None, ld, scales or None, lds, Y or None, ldy,
                                   _mx_format(format), _along(along), stream or None),
           "gemm_mx_dequantize")


def gemm_mx(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_format, config=-1,
            stream=0) -> None:
    _fits(M, N, K, lda, ldsa, ldb, ldsb, ldc, int(config))
    _check(_lib.gemm_mx(M, N, K, A or None, lda, SA or None, ldsa, B or None, ldb, SB or None,
                        ldsb, C or None, ldc, _mx_format(c_format), int(config), stream or None),
           "gemm_mx")


def gemm_mx_num_configs() -> int:
    return int(_lib.gemm_mx_num_configs())


def gemm_mx_tile(config, M, N, K) -> dict:
    vals = [ctypes.c_int(0) for _ in range(5)]
    _fits(int(config), M, N, K)
    rc = _lib.gemm_mx_tile(int(config), M, N, K, *[ctypes.byref(v) for v in vals])
    _check(rc, "gemm_mx_tile")
    bm, bn, bk, nt, chosen = (v.value for v in vals)
    return {"BM": bm, "BN": bn, "BK": bk, "threads": nt, "config": chosen}


def gemm_mx_a16(M, N, K, A, lda, a_format, B, ldb, SB, ldsb, C, ldc, c_format, stream=0) -> None:
    _fits(M, N, K, lda, ldb, ldsb, ldc)
    _check(_lib.gemm_mx_a16(M, N, K, A or None, lda, _format(a_format), B or None, ldb,
                            SB or None, ldsb, C or None, ldc, _mx_format(c_format),
                            stream or None),
           "gemm_mx_a16")


def gemm_moe_workspace_bytes(T, E, top, H, I) -> int:
    _fits(int(T), int(E), int(top), int(H), int(I))
    return int(_lib.gemm_moe_workspace_bytes(int(T), int(E), int(top), int(H), int(I)))


def gemm_moe(T, E, top, H, I, X, ldx, R, ldr, format, W1, ld1, S1, lds1, W2, ld2, S2, lds2, weights,
             renormalize, Y, ldy, y_format, ids, gates, workspace, workspace_bytes,
             stream=0) -> None:
    weights = MOE_WEIGHTS[weights] if isinstance(weights, str) else int(weights)
    _fits(T, E, top, H, I, ldx, ldr, ld1, lds1, ld2, lds2, weights, ldy)
    _check(_lib.gemm_moe(T, E, top, H, I, X or None, ldx, R or None, ldr, _format(format),
                         W1 or None, ld1, S1 or None, lds1, W2 or None, ld2, S2 or None, lds2,
                         weights, int(renormalize), Y or None, ldy, _mx_format(y_format),
                         ids or None, gates or None, workspace or None, int(workspace_bytes),
                         stream or None),
           "gemm_moe")


def _named(value, names: dict, what: str) -> int:
    known = names.get(value)
    if known is not None:
        return known
    if isinstance(value, str):
        raise ValueError(f"unknown {what} {value!r}; one of {sorted(names)}")
    return int(value)


def gemm_moe_route(T, E, top, Z, ldz, format, score, bias, groups, top_groups, group_score,
                   renormalize, scale, ids, gates, stream=0) -> None:
    score, group_score = _named(score, ROUTE_SCORES, "score"), _named(group_score, ROUTE_GROUP_SCORES, "group score")
    _fits(T, E, top, ldz, score, groups, top_groups, group_score)
    _check(_lib.gemm_moe_route(T, E, top, Z or None, ldz, _mx_format(format), score, bias or None,
                               groups, top_groups, group_score, int(bool(renormalize)), scale,
                               ids or None, gates or None, stream or None),
           "gemm_moe_route")


def gemm_moe_route_backward(T, E, top, dgates, Z, ldz, format, score, renormalize, scale, ids, dZ,
                            lddz, stream=0) -> None:
    score = _named(score, ROUTE_SCORES, "score")
    _fits(T, E, top, ldz, score, lddz)
    _check(_lib.gemm_moe_route_backward(T, E, top, dgates or None, Z or None, ldz,
                                        _mx_format(format), score, int(bool(renormalize)), scale,
                                        ids or None, dZ or None, lddz, stream or None),
           "gemm_moe_route_backward")


def gemm_experts_workspace_bytes(T, E, top, H, I, backward=0) -> int:
    _fits(int(T), int(E), int(top), int(H), int(I))
    return int(_lib.gemm_experts_workspace_bytes(int(T), int(E), int(top), int(H), int(I),
                                                 int(bool(backward))))


def gemm_experts(T, E, top, H, I, X, ldx, ids, gates, format, W1, ld1, S1, lds1, W2, ld2, S2, lds2,
                 weights, Y, ldy, saved, workspace, workspace_bytes, stream=0) -> None:
    weights = _named(weights, MOE_WEIGHTS, "kind of weights")
    _fits(T, E, top, H, I, ldx, ld1, lds1, ld2, lds2, weights, ldy)
    _check(_lib.gemm_experts(T, E, top, H, I, X or None, ldx, ids or None, gates or None,
                             _format(format), W1 or None, ld1, S1 or None, lds1, W2 or None, ld2,
                             S2 or None, lds2, weights, Y or None, ldy, saved or None,
                             workspace or None, int(workspace_bytes), stream or None),
           "gemm_experts")


def gemm_experts_backward(T, E, top, H, I, dY, lddy, X, ldx, ids, gates, format, W1, ld1, W2, ld2,
                          saved, dX, lddx, dgates, dW1, lddw1, dW2, lddw2, workspace,
                          workspace_bytes, stream=0) -> None:
    _fits(T, E, top, H, I, lddy, ldx, ld1, ld2, lddx, lddw1, lddw2)
    _check(_lib.gemm_experts_backward(T, E, top, H, I, dY or None, lddy, X or None, ldx,
                                      ids or None, gates or None, _format(format), W1 or None, ld1,
                                      W2 or None, ld2, saved or None, dX or None, lddx,
                                      dgates or None, dW1 or None, lddw1, dW2 or None, lddw2,
                                      workspace or None, int(workspace_bytes), stream or None),
           "gemm_experts_backward")


def gemm_adapters_workspace_bytes(T, N, K, R, count) -> int:
    _fits(int(T), int(N), int(K), int(R), int(count))
    return int(_lib.gemm_adapters_workspace_bytes(int(T), int(N), int(K), int(R), int(count)))


def gemm_adapters(T, N, K, R, count, X, ldx, W, ldw, A, lda, B, ldb, ids, scales, format, Y, ldy,
                  workspace, workspace_bytes, stream=0) -> None:
    _fits(T, N, K, R, count, ldx, ldw, lda, ldb, ldy)
    _check(_lib.gemm_adapters(T, N, K, R, count, X or None, ldx, W or None, ldw, A or None, lda,
                              B or None, ldb, ids or None, scales or None, _format(format),
                              Y or None, ldy, workspace or None, int(workspace_bytes),
                              stream or None),
           "gemm_adapters")


def config_name(variant, config: int = -1, M: int = 1, N: int = 1, K: int = 1) -> str:
    """Readable name of a launch-table entry, e.g. "prod#0:128x128x32/256t"."""
    t = gemm_f32_tile(variant, config, M, N, K)
    v = _variant(variant)
    vname = next(k for k, val in VARIANTS.items() if val == v)
    return f"{vname}#{t['config']}:{t['BM']}x{t['BN']}x{t['BK']}/{t['threads']}t"


def mixed_config_name(fmt, config: int = -1, M: int = 1, N: int = 1, K: int = 1) -> str:
    """Readable name of a gemm_mixed entry, e.g. "bf16#0:256x256x64/512t"."""
    t = gemm_mixed_tile(config, M, N, K)
    f = next(k for k, val in MIXED_FORMATS.items() if val == _format(fmt))
    return f"{f}#{t['config']}:{t['BM']}x{t['BN']}x{t['BK']}/{t['threads']}t"


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("the last dimension must be contiguous (stride 1)")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("rows overlap (row stride smaller than the row length)")
    return max(1, t.stride(0) if t.shape[0] > 1 else t.shape[1])


def _empty(device, stream):
    """torch.empty for tensors that belong to ``stream`` (None: the current one).  The
    allocator reuses a tensor's memory in the order of the stream that it belongs to,
    so one that is used on another would be handed out while it is still in use, and
    taken while earlier work still uses it."""
    if stream is None or stream == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty
    owner = (torch.cuda.ExternalStream(stream, device=device) if stream
             else torch.cuda.default_stream(device))

    def empty(*args, **kw):
        with torch.cuda.stream(owner):
            return torch.empty(*args, **kw)

    return empty


def matmul(A, B, out=None, variant="prod", config: int = -1, stream=None):
    """C = A x B on the GPU for float32 tensors (row-major views with unit last stride)."""
    import torch

    for name, t in (("A", A), ("B", B)):
        if t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError(f"{name} must be a float32 CUDA tensor")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if out is None:
        out = _empty(A.device, stream)((M, N), dtype=torch.float32, device=A.device)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M, N) or not out.is_cuda:
        raise TypeError("out must be a float32 CUDA tensor of shape (M, N)")
    if stream is None:
        stream = torch.cuda.current_stream(A.device).cuda_stream
    lda = max(_ld(A), max(1, K))
    ldb = max(_ld(B), max(1, N))
    ldc = max(_ld(out), max(1, N))
    gemm_f32_ex(M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc,
                variant, config, stream)
    return out


def matmul_mixed(A, B, out=None, config: int = -1, stream=None, format=None):
    """C = A x B on the GPU for bfloat16 or float16 tensors, fp32 result.

    A and B must share one 16-bit dtype (or be int16 / uint16 codes with
    ``format`` given) and have unit last stride.
    """
    import torch

    kinds = {torch.bfloat16: "bf16", torch.float16: "f16"}
    if A.dtype != B.dtype:
        raise TypeError("A and B must have the same dtype")
    if A.dtype in kinds:
        fmt = kinds[A.dtype] if format is None else format
        if format is not None and _format(format) != MIXED_FORMATS[kinds[A.dtype]]:
            raise TypeError(f"format {format!r} does not match dtype {A.dtype}")
    elif A.dtype in (torch.int16, torch.uint16) and format is not None:
        fmt = format
    else:
        raise TypeError("A and B must be bfloat16 / float16 tensors (or 16-bit codes with format=)")
    if not (A.is_cuda and B.is_cuda):
        raise TypeError("A and B must be CUDA tensors")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if out is None:
        out = _empty(A.device, stream)((M, N), dtype=torch.float32, device=A.device)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M, N) or not out.is_cuda:
        raise TypeError("out must be a float32 CUDA tensor of shape (M, N)")
    if stream is None:
        stream = torch.cuda.current_stream(A.device).cuda_stream
    lda = max(_ld(A), max(1, K))
    ldb = max(_ld(B), max(1, N))
    ldc = max(_ld(out), max(1, N))
    gemm_mixed(M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc, fmt,
               config, stream)
    return out


def matmul_splitk(A, B, out=None, config: int = -1, splits: int = 0, workspace=None, stream=None):
    """C = A x B through the split-K plan, for float32 CUDA tensors.

    ``workspace`` is a CUDA tensor of at least the plan's workspace bytes; when
    None, one is allocated with torch for this call.
    """
    import torch

    for name, t in (("A", A), ("B", B)):
        if t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError(f"{name} must be a float32 CUDA tensor")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if out is None:
        out = _empty(A.device, stream)((M, N), dtype=torch.float32, device=A.device)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M, N) or not out.is_cuda:
        raise TypeError("out must be a float32 CUDA tensor of shape (M, N)")
    plan = gemm_f32_splitk_plan(M, N, K, config, splits)
    if workspace is None and plan["workspace_bytes"] > 0:
        workspace = _empty(A.device, stream)(plan["workspace_bytes"] // 4, dtype=torch.float32,
                                             device=A.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(A.device).cuda_stream
    lda = max(_ld(A), max(1, K))
    ldb = max(_ld(B), max(1, N))
    ldc = max(_ld(out), max(1, N))
    gemm_f32_splitk(M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc, config,
                    splits, ws_ptr, ws_bytes, stream)
    return out


class MxTensor:
    """A matrix in 4-bit microscaled form (include/gemm_mx.h): ``codes`` and
    ``scales`` are uint8 tensors of ``rows`` rows (more leading dimensions for a
    stack of matrices), each row 16 ceil(K / 32) bytes of codes and
    16 ceil(K / 512) bytes of scales."""

    __slots__ = ("codes", "scales", "K")

    def __init__(self, codes, scales, K: int):
        K = int(K)
        if K < 0:
            raise ValueError("K must be >= 0")
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        c, s = codes.shape, scales.shape
        for name, shape, need in (("codes", c, (K + 31) // 32 * 16), ("scales", s, (K + 511) // 512 * 16)):
            if len(shape) < 2 or shape[-1] < need:
                raise ValueError(f"{name} must have rows of at least {need} bytes for K = {K}")
        if c[0] != s[0] or (len(c) != 2 or len(s) != 2) and c[:-1] != s[:-1]:
            raise ValueError("codes and scales must have the same rows")
        self.codes, self.scales, self.K = codes, scales, K

    @property
    def shape(self):
        """(rows, K), after any leading dimensions."""
        return (*self.codes.shape[:-1], self.K)

    @classmethod
    def empty(cls, rows: int, K: int, device) -> "MxTensor":
        blocks = (K + 31) // 32
        return cls(torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=device),
                   torch.empty((rows, (blocks + 15) // 16 * 16), dtype=torch.uint8, device=device), K)


def _row_pitch(t) -> int:
    """Row pitch in bytes of a 2-D uint8 tensor with contiguous rows, at least 16."""
    rows, width = t.shape
    if width > 0 and width % 16 == 0 and t.is_contiguous():
        return width
    if width > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (last stride 1)")
    if rows > 1:
        if t.stride(0) < width:
            raise ValueError("rows overlap (row stride smaller than the row length)")
        return max(16, t.stride(0))
    return max(16, (width + 15) // 16 * 16)


def _mx_args(q, name: str, device):
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name} must be an MxTensor")
    codes, scales = q.codes, q.scales
    if len(codes.shape) != 2:
        raise ValueError(f"{name} must be one matrix (2-D codes and scales)")
    if not codes.is_cuda or codes.device != device or scales.device != device:
        raise TypeError(f"{name} must be on {device} like the other operands")
    return codes.data_ptr(), _row_pitch(codes), scales.data_ptr(), _row_pitch(scales)


def _pitch(t) -> int:
    """_ld, without its checks where a matrix is contiguous."""
    if t.dim() == 2 and t.is_contiguous():
        return t.shape[1] or 1
    return _ld(t)


def _launch(fn, where: str, device, stream, args) -> None:
    """Calls an entry of the library with `device` current, on `stream` or, when
    it is None, on the device's current stream."""
    index = device.index
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():  # CUDA tensors exist, so torch's state does
        rc = fn(*args, stream or None)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream or None)
    if rc != 0:
        raise GemmError(rc, where)


def _mx_out(out, shape, dtype, device, stream):
    if out is None:
        return _empty(device, stream)(shape, dtype=dtype, device=device)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or out.device != device:
        raise TypeError(f"out must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def mx_quantize(X, along: str = "rows", out=None, stream=None):
    """The MX form of a float32, bfloat16 or float16 CUDA matrix with unit last
    stride: of its rows, or (``along="columns"``) of its columns."""
    fmt = _MX_DTYPES.get(X.dtype)
    if fmt is None or not X.is_cuda:
        raise TypeError("X must be a float32, bfloat16 or float16 CUDA tensor")
    ldx, device, way = _pitch(X), X.device, _along(along)
    rows, K = X.shape
    if way == 1:
        rows, K = K, rows
    if max(rows, K, ldx) > _INT_MAX:
        _fits(rows, K, ldx)
    if out is None:
        c, s = (K + 31) // 32 * 16, (K + 511) // 512 * 16
        empty = _empty(device, stream)
        codes = empty((rows, c), dtype=torch.uint8, device=device)
        scales = empty((rows, s), dtype=torch.uint8, device=device)
        out = MxTensor(codes, scales, K)
        args = codes.data_ptr(), c or 16, scales.data_ptr(), s or 16
    else:
        args = _mx_args(out, "out", device)
        if out.shape != (rows, K):
            raise ValueError(f"out must be an MxTensor of shape {(rows, K)}")
        _fits(args[1], args[3])
    _launch(_lib.gemm_mx_quantize, "gemm_mx_quantize", device, stream,
            (rows, K, X.data_ptr(), ldx, fmt, way, *args))
    return out


def mx_dequantize(q, dtype=torch.float32, along: str = "rows", out=None, stream=None):
    """The values of an MxTensor as a matrix of ``dtype``: its rows as rows, or
    (``along="columns"``) as columns."""
    fmt = _MX_DTYPES.get(dtype)
    if fmt is None:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    if not isinstance(q, MxTensor):
        raise TypeError("q must be an MxTensor")
    device, way = q.codes.device, _along(along)
    args = _mx_args(q, "q", device)
    rows, K = q.codes.shape[0], q.K
    out = _mx_out(out, (rows, K) if way == 0 else (K, rows), dtype, device, stream)
    ldy = _pitch(out)
    if max(rows, K, args[1], args[3], ldy) > _INT_MAX:
        _fits(rows, K, args[1], args[3], ldy)
    _launch(_lib.gemm_mx_dequantize, "gemm_mx_dequantize", device, stream,
            (rows, K, *args, out.data_ptr(), ldy, fmt, way))
    return out


def matmul_mx(A, B, dtype=torch.float32, out=None, config: int = -1, stream=None):
    """C[i][j] = sum_k A[i][k] B[j][k] for the rows of A and of the MxTensor B.

    A is an MxTensor, or a bfloat16 or float16 CUDA matrix with unit last
    stride (whose values enter as they are; ``config`` is then not taken).
    ``dtype`` is the result's: float32, bfloat16 or float16.
    """
    fmt = _MX_DTYPES.get(dtype)
    if fmt is None:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    if not isinstance(B, MxTensor):
        raise TypeError("B must be an MxTensor")
    device = B.codes.device
    b = _mx_args(B, "B", device)
    N, K = B.codes.shape[0], B.K
    mx = isinstance(A, MxTensor)
    if mx:
        a = _mx_args(A, "A", device)
        M, K2 = A.codes.shape[0], A.K
    else:
        if A.dtype not in (torch.bfloat16, torch.float16) or A.device != device:
            raise TypeError(f"A must be an MxTensor, or a bfloat16 or float16 tensor on {device}")
        if config != -1:
            raise ValueError("config is for products of two MxTensors")
        a = A.data_ptr(), _pitch(A), _MX_DTYPES[A.dtype]
        M, K2 = A.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} and {tuple(B.shape)}")
    if max(M, N, K, config, a[1], b[1], b[3], a[3] if mx else 0) > _INT_MAX:
        _fits(M, N, K, config, a[1], b[1], b[3], a[3] if mx else 0)
    if out is None:
        out = _empty(device, stream)((M, N), dtype=dtype, device=device)
        ldc = N or 1
    else:
        _mx_out(out, (M, N), dtype, device, stream)
        ldc = _pitch(out)
        _fits(ldc)
    if mx:
        _launch(_lib.gemm_mx, "gemm_mx", device, stream,
                (M, N, K, *a, *b, out.data_ptr(), ldc, fmt, config))
    else:
        _launch(_lib.gemm_mx_a16, "gemm_mx_a16", device, stream,
                (M, N, K, *a, *b, out.data_ptr(), ldc, fmt))
    return out


def _expert_rows(w, name: str, dtype, device, E: int, rows: int, K: int):
    """Pointers and pitches of stacked expert matrices (E, rows, K): (weights,
    pitch, scales, scale pitch), the experts' rows following one another."""
    def pitch(t, width, what):
        shape = t.shape
        if len(shape) != 3 or t.device != device:
            raise TypeError(f"{what} must be a 3-D tensor on {device}")
        if shape[0] != E or shape[1] != rows:
            raise ValueError(f"{what} must have {E} experts of {rows} rows, not {tuple(shape)}")
        if E * rows > 1 and t.is_contiguous():
            return shape[2]
        if t.shape[2] > 1 and t.stride(2) != 1:
            raise ValueError(f"{what} must have contiguous rows (last stride 1)")
        if rows > 1 and t.stride(1) < t.shape[2]:
            raise ValueError(f"{what}: rows overlap")
        step = t.stride(1) if rows > 1 else (t.stride(0) if E > 1 else width)
        if E > 1 and t.stride(0) != rows * step:
            raise ValueError(f"{what}: experts must follow one another (stride {rows * step})")
        return step

    if isinstance(w, MxTensor):
        if w.K != K:
            raise ValueError(f"{name} must have rows of {K} values, not {w.K}")
        c = pitch(w.codes, (K + 31) // 32 * 16, name + ".codes")
        s = pitch(w.scales, (K + 511) // 512 * 16, name + ".scales")
        return w.codes.data_ptr(), c, w.scales.data_ptr(), s
    if w.dtype != dtype:
        raise TypeError(f"{name} must be an MxTensor, or {dtype} like the tokens")
    if w.dim() == 3 and w.shape[2] != K:
        raise ValueError(f"{name} must have rows of {K} values, not {w.shape[2]}")
    return w.data_ptr(), pitch(w, K, name), 0, 0


def moe_layer(X, router, w1, w2, top: int, renormalize: bool = True, dtype=None, out=None,
              workspace=None, stream=None):
    """A mixture-of-experts layer for a few tokens (include/gemm_moe.h): (Y, ids, gates).

    X is (T, H), router (E, H), both bfloat16 or float16; w1 is (E, 2 I, H) with
    each expert's gate rows first and w2 (E, H, I), tensors of the same dtype or
    stacks of MX matrices (MxTensor with 3-D codes and scales).  Y is (T, H) in
    ``dtype`` (X's, or float32), ids (T, top) int32 and gates (T, top) float32.
    ``workspace`` is a uint8 CUDA tensor of at least gemm_moe_workspace_bytes;
    when None, one is allocated with torch for this call.
    """
    if X.dtype not in (torch.bfloat16, torch.float16) or not X.is_cuda:
        raise TypeError("X must be a bfloat16 or float16 CUDA tensor")
    device = X.device
    if router.dtype != X.dtype or router.device != device:
        raise TypeError(f"router must be a {X.dtype} tensor on {device}")
    ldx, ldr = _pitch(X), _pitch(router)
    T, H = X.shape
    E = router.shape[0]
    if router.shape[1] != H:
        raise ValueError(f"router must have rows of {H} values, not {router.shape[1]}")
    if isinstance(w1, MxTensor) != isinstance(w2, MxTensor):
        raise TypeError("w1 and w2 must both be MxTensors or both tensors")
    mx = isinstance(w2, MxTensor)
    I = w2.K if mx else w2.shape[-1]
    a1 = _expert_rows(w1, "w1", X.dtype, device, E, 2 * I, H)
    a2 = _expert_rows(w2, "w2", X.dtype, device, E, H, I)
    dtype = X.dtype if dtype is None else dtype
    if dtype not in (X.dtype, torch.float32):
        raise TypeError(f"dtype must be {X.dtype} or float32")
    top = int(top)
    if max(T, E, top, H, I, ldx, ldr, a1[1], a1[3], a2[1], a2[3]) > _INT_MAX:
        _fits(T, E, top, H, I, ldx, ldr, a1[1], a1[3], a2[1], a2[3])
    need = _lib.gemm_moe_workspace_bytes(T, E, top, H, I)
    if need < 0:
        raise ValueError(f"sizes outside the layer's bounds: {T} tokens, {E} experts, top {top}, "
                         f"widths {H} and {I}")
    empty = _empty(device, stream)
    if out is None:
        out = empty((T, H), dtype=dtype, device=device)
        ldy = H
    else:
        _mx_out(out, (T, H), dtype, device, stream)
        ldy = _pitch(out)
        _fits(ldy)
    ids = empty((T, top), dtype=torch.int32, device=device)
    gates = empty((T, top), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise TypeError(f"workspace must be a contiguous tensor on {device}")
    _launch(_lib.gemm_moe, "gemm_moe", device, stream,
            (T, E, top, H, I, X.data_ptr(), ldx, router.data_ptr(), ldr, _MX_DTYPES[X.dtype],
             *a1, *a2, int(mx), int(renormalize), out.data_ptr(), ldy, _MX_DTYPES[dtype],
             ids.data_ptr(), gates.data_ptr(), workspace.data_ptr(),
             workspace.numel() * workspace.element_size()))
    return out, ids, gates


def _choices(ids, gates, name: str, device):
    """Checks a contiguous (T, top) int32 tensor of ids and its float32 companion."""
    if ids.dtype != torch.int32 or ids.device != device or ids.dim() != 2 or not ids.is_contiguous():
        raise TypeError(f"ids must be a contiguous 2-D int32 tensor on {device}")
    if gates.dtype != torch.float32 or gates.device != device or not gates.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor on {device}")
    if gates.shape != ids.shape:
        raise ValueError(f"{name} must have the shape of ids, {tuple(ids.shape)}")


def _logits(logits):
    fmt = _MX_DTYPES.get(logits.dtype)
    if fmt is None or not logits.is_cuda:
        raise TypeError("logits must be a float32, bfloat16 or float16 CUDA tensor")
    return fmt, _pitch(logits)


def moe_route(logits, top: int, score="softmax", bias=None, groups: int = 1, top_groups: int = 1,
              group_score="max", renormalize: bool = True, scale: float = 1.0, stream=None):
    """Chosen experts and their gates from logits (T, E) (include/gemm_route.h): (ids, gates).

    ``score`` is "softmax" or "sigmoid"; ``bias`` (E float32) is added to the scores
    for the choice alone.  The experts are ``groups`` runs; where ``top_groups`` is
    less, only experts of that many groups can be chosen, by the largest key in a
    group (``group_score="max"``) or the sum of its two largest ("top2").  With
    ``renormalize`` a token's gates add up to ``scale``.  ids are (T, top) int32,
    gates (T, top) float32.
    """
    fmt, ldz = _logits(logits)
    device = logits.device
    T, E = logits.shape
    if bias is not None:
        if bias.dtype != torch.float32 or bias.device != device or not bias.is_contiguous():
            raise TypeError(f"bias must be a contiguous float32 tensor on {device}")
        if tuple(bias.shape) != (E,):
            raise ValueError(f"bias must have {E} values")
    top, groups, top_groups = int(top), int(groups), int(top_groups)
    score = _named(score, ROUTE_SCORES, "score")
    group_score = _named(group_score, ROUTE_GROUP_SCORES, "group score")
    if max(T, E, top, ldz, score, groups, top_groups, group_score) > _INT_MAX or min(
            top, score, groups, top_groups, group_score) < 0:
        _fits(T, E, top, ldz, score, groups, top_groups, group_score)
        raise ValueError("top, groups and top_groups must not be negative")
    empty = _empty(device, stream)
    ids = empty(T, top, dtype=torch.int32, device=device)
    gates = empty(T, top, dtype=torch.float32, device=device)
    _launch(_lib.gemm_moe_route, "gemm_moe_route", device, stream,
            (T, E, top, logits.data_ptr(), ldz, fmt, score,
             bias.data_ptr() if bias is not None else None, groups, top_groups, group_score,
             int(bool(renormalize)), float(scale), ids.data_ptr(), gates.data_ptr()))
    return ids, gates


def moe_route_backward(dgates, logits, ids, score="softmax", renormalize: bool = True,
                       scale: float = 1.0, out=None, stream=None):
    """The gradient of moe_route's logits, in their dtype, from that of its gates
    (T, top): for the ids that it gave and the same score, renormalize and scale."""
    fmt, ldz = _logits(logits)
    device = logits.device
    _choices(ids, dgates, "dgates", device)
    T, E = logits.shape
    if ids.shape[0] != T:
        raise ValueError(f"ids must have {T} rows, not {ids.shape[0]}")
    score = _named(score, ROUTE_SCORES, "score")
    if out is None:
        out, lddz = _empty(device, stream)(T, E, dtype=logits.dtype, device=device), E or 1
    else:
        lddz = _pitch(_mx_out(out, (T, E), logits.dtype, device, stream))
    top = ids.shape[1]
    if max(T, E, top, ldz, lddz, score) > _INT_MAX:
        _fits(T, E, top, ldz, lddz, score)
    _launch(_lib.gemm_moe_route_backward, "gemm_moe_route_backward", device, stream,
            (T, E, top, dgates.data_ptr(), logits.data_ptr(), ldz, fmt, score,
             int(bool(renormalize)), float(scale), ids.data_ptr(), out.data_ptr(), lddz))
    return out


def _workspace(workspace, need: int, empty, device):
    if workspace is None:
        return empty(need, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise TypeError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _experts_sizes(X, ids, gates, w1, w2):
    if X.dtype not in (torch.bfloat16, torch.float16) or not X.is_cuda:
        raise TypeError("X must be a bfloat16 or float16 CUDA tensor")
    device = X.device
    ldx = _pitch(X)
    T, H = X.shape
    _choices(ids, gates, "gates", device)
    if ids.shape[0] != T:
        raise ValueError(f"ids must have {T} rows, not {ids.shape[0]}")
    if isinstance(w1, MxTensor) != isinstance(w2, MxTensor):
        raise TypeError("w1 and w2 must both be MxTensors or both tensors")
    if len(w2.shape) != 3:
        raise ValueError("w2 must have three dimensions: experts, rows, values")
    E, I = w2.shape[0], w2.shape[2]
    a1 = _expert_rows(w1, "w1", X.dtype, device, E, 2 * I, H)
    a2 = _expert_rows(w2, "w2", X.dtype, device, E, H, I)
    top = ids.shape[1]
    if max(T, E, top, H, I, ldx, a1[1], a1[3], a2[1], a2[3]) > _INT_MAX:
        _fits(T, E, top, H, I, ldx, a1[1], a1[3], a2[1], a2[3])
    return device, T, E, top, H, I, ldx, a1, a2


def _experts_bytes(T, E, top, H, I, backward: int) -> int:
    need = _lib.gemm_experts_workspace_bytes(T, E, top, H, I, backward)
    if need < 0:
        raise ValueError(f"sizes outside the products' bounds: {T} tokens, {E} experts, top {top}, "
                         f"widths {H} and {I}")
    return need


def moe_experts(X, ids, gates, w1, w2, save: bool = False, out=None, workspace=None, stream=None):
    """The experts' products for a choice made before (include/gemm_experts.h), y[t] =
    sum_s gates[t][s] w2[e] u, u = silu(w1[e][:I] x[t]) * (w1[e][I:] x[t]), e = ids[t][s].

    X is (T, H), bfloat16 or float16; ids (T, top) int32, where an id outside 0 .. E - 1
    is a dropped choice, gates (T, top) float32; w1 is (E, 2 I, H) and w2 (E, H, I),
    tensors of X's dtype or, up to 256 tokens and without ``save``, stacks of MX matrices.
    Returns Y, (T, H) in X's dtype; with ``save`` (Y, saved), the second for
    moe_experts_backward.  u is kept in X's dtype (in float16 infinite past 65,504) but for a
    few tokens without ``save`` (T top <= 6 E, T <= 256), where it is kept in float32.
    ``workspace`` is a uint8 CUDA tensor of at least
    gemm_experts_workspace_bytes; when None, one is allocated with torch for this call.
    """
    device, T, E, top, H, I, ldx, a1, a2 = _experts_sizes(X, ids, gates, w1, w2)
    mx = isinstance(w2, MxTensor)
    if mx and (save or T > 256):
        raise ValueError("MX weights are for up to 256 tokens, without save")
    need = _experts_bytes(T, E, top, H, I, 0)
    empty = _empty(device, stream)
    if out is None:
        out, ldy = empty(T, H, dtype=X.dtype, device=device), H
    else:
        ldy = _pitch(_mx_out(out, (T, H), X.dtype, device, stream))
        _fits(ldy)
    saved = empty(T * top, 2 * I, dtype=torch.float32, device=device) if save else None
    workspace = _workspace(workspace, need, empty, device)
    _launch(_lib.gemm_experts, "gemm_experts", device, stream,
            (T, E, top, H, I, X.data_ptr(), ldx, ids.data_ptr(), gates.data_ptr(),
             _MX_DTYPES[X.dtype], *a1, *a2, int(mx), out.data_ptr(), ldy,
             saved.data_ptr() if save else None, workspace.data_ptr(),
             workspace.numel() * workspace.element_size()))
    return (out, saved) if save else out


def moe_experts_backward(dY, X, ids, gates, w1, w2, saved, weights: bool = True, workspace=None,
                         stream=None):
    """The gradients (dX, dgates, dw1, dw2) of moe_experts from that of its result, with
    the ``saved`` of the same call; without ``weights`` (dX, dgates) alone."""
    device, T, E, top, H, I, ldx, a1, a2 = _experts_sizes(X, ids, gates, w1, w2)
    if isinstance(w2, MxTensor):
        raise TypeError("w1 and w2 must be tensors")
    if dY.dtype != X.dtype or dY.device != device or tuple(dY.shape) != (T, H):
        raise TypeError(f"dY must be a {X.dtype} tensor of shape {(T, H)} on {device}")
    lddy = _pitch(dY)
    _fits(lddy)
    if (saved.dtype != torch.float32 or saved.device != device or not saved.is_contiguous()
            or tuple(saved.shape) != (T * top, 2 * I)):
        raise TypeError(f"saved must be a contiguous float32 tensor of shape {(T * top, 2 * I)} on {device}")
    need = _experts_bytes(T, E, top, H, I, 1)
    empty = _empty(device, stream)
    dX = empty(T, H, dtype=X.dtype, device=device)
    dgates = empty(T, top, dtype=torch.float32, device=device)
    dw1 = empty(E, 2 * I, H, dtype=X.dtype, device=device) if weights else None
    dw2 = empty(E, H, I, dtype=X.dtype, device=device) if weights else None
    workspace = _workspace(workspace, need, empty, device)
    _launch(_lib.gemm_experts_backward, "gemm_experts_backward", device, stream,
            (T, E, top, H, I, dY.data_ptr(), lddy, X.data_ptr(), ldx, ids.data_ptr(),
             gates.data_ptr(), _MX_DTYPES[X.dtype], a1[0], a1[1], a2[0], a2[1], saved.data_ptr(),
             dX.data_ptr(), H, dgates.data_ptr(), dw1.data_ptr() if weights else None, H,
             dw2.data_ptr() if weights else None, I, workspace.data_ptr(),
             workspace.numel() * workspace.element_size()))
    return (dX, dgates, dw1, dw2) if weights else (dX, dgates)


def matmul_adapters(X, w, a, b, ids, scales=None, out=None, workspace=None, stream=None):
    """A shared projection with low-rank adapters (include/gemm_adapters.h), y[t] = w x[t] +
    scales[r] b[r] (a[r] x[t]), r = ids[t]; a row whose id is outside 0 .. count - 1 has no
    adapter.

    X is (T, K) and w (N, K), both bfloat16 or float16; a is (count, R, K) and b (count, N, R)
    of the same dtype; ids (T,) int32; scales (count,) float32, or None for 1 each.  Returns
    (T, N) in X's dtype.  ``workspace`` is a uint8 CUDA tensor of at least
    gemm_adapters_workspace_bytes; when None, one is allocated with torch for this call.
    """
    if X.dtype not in (torch.bfloat16, torch.float16) or not X.is_cuda:
        raise TypeError("X must be a bfloat16 or float16 CUDA tensor")
    device = X.device
    if w.dtype != X.dtype or w.device != device:
        raise TypeError(f"w must be a {X.dtype} tensor on {device}")
    ldx, ldw = _pitch(X), _pitch(w)
    T, K = X.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w must have rows of {K} values, not {w.shape[1]}")
    if isinstance(a, MxTensor) or isinstance(b, MxTensor):
        raise TypeError("a and b must be tensors")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must have three dimensions: adapters, rows, values")
    count, R = a.shape[0], a.shape[1]
    pa = _expert_rows(a, "a", X.dtype, device, count, R, K)
    pb = _expert_rows(b, "b", X.dtype, device, count, N, R)
    if ids.dtype != torch.int32 or ids.device != device or not ids.is_contiguous():
        raise TypeError(f"ids must be a contiguous int32 tensor on {device}")
    if tuple(ids.shape) != (T,):
        raise ValueError(f"ids must have {T} values")
    if scales is not None:
        if scales.dtype != torch.float32 or scales.device != device or not scales.is_contiguous():
            raise TypeError(f"scales must be a contiguous float32 tensor on {device}")
        if tuple(scales.shape) != (count,):
            raise ValueError(f"scales must have {count} values")
    if max(T, N, K, R, count, ldx, ldw, pa[1], pb[1]) > _INT_MAX:
        _fits(T, N, K, R, count, ldx, ldw, pa[1], pb[1])
    need = _lib.gemm_adapters_workspace_bytes(T, N, K, R, count)
    if need < 0:
        raise ValueError(f"sizes outside the product's bounds: {T} rows, {N} x {K}, {count} adapters "
                         f"of rank {R}")
    empty = _empty(device, stream)
    if out is None:
        out, ldy = empty(T, N, dtype=X.dtype, device=device), N
    else:
        ldy = _pitch(_mx_out(out, (T, N), X.dtype, device, stream))
        _fits(ldy)
    workspace = _workspace(workspace, need, empty, device)
    _launch(_lib.gemm_adapters, "gemm_adapters", device, stream,
            (T, N, K, R, count, X.data_ptr(), ldx, w.data_ptr(), ldw, pa[0], pa[1], pb[0], pb[1],
             ids.data_ptr(), scales.data_ptr() if scales is not None else None,
             _MX_DTYPES[X.dtype], out.data_ptr(), ldy, workspace.data_ptr(),
             workspace.numel() * workspace.element_size()))
    return out
