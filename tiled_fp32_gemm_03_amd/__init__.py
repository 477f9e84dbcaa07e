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
