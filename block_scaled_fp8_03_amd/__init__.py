"""Block-scaled FP8 linear for AMD MI355X (gfx950): Python binding.

This module only marshals torch tensors into the C ABI of ``libfp8bs.so``
(declared in ``include/fp8bs.h``); every step of the computation runs in the
library's HIP kernels.  PyTorch provides device memory and streams.

Raw entry points carry the C names and take caller-allocated outputs:
``fp8bs_act_quant``, ``fp8bs_weight_quant``, ``fp8bs_weight_dequant``,
``fp8bs_gemm``, ``fp8bs_moe_gemm``, the BF16 path ``fp8bs_w8a16_gemm`` and
the MoE dispatch/combine steps
``fp8bs_moe_route``, ``fp8bs_moe_quant_scatter``, ``fp8bs_moe_combine``, the
absorb attention over a paged latent cache ``fp8bs_mla_attention`` between
``fp8bs_mla_absorb_key`` and ``fp8bs_mla_absorb_value``, and that cache's
``fp8bs_mla_cache_write``, ``fp8bs_cache_update``, ``fp8bs_cache_compact``.
Allocating conveniences: ``act_quant``, ``weight_quant``, ``weight_dequant``,
``fp8_gemm``, ``moe_gemm``, ``linear``, ``w8a16_gemm``, ``moe_route``,
``moe_quant_scatter``, ``moe_combine``, ``mla_absorb_key``, ``mla_absorb_value``,
``mla_cache_alloc``, ``mla_cache_write``, ``mla_attention``, ``cache_update``,
``cache_compact``.

The operations follow the DeepSeek-V3 inference pages ("DeepSeek-V3
Administrator & Developer Guide", sections 6.3, 6.4, 8.5.1-8.5.3; "DeepSeek-V3
User Guide", FAQ on scale_fmt ue8m0).  If the library has not been built the
calls raise; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

__all__ = [
    "SCALE_FP32", "SCALE_UE8M0", "OUT_BF16", "OUT_F32", "Fp8bsError", "library_path", "lib",
    "fp8bs_act_quant", "fp8bs_weight_quant", "fp8bs_weight_dequant", "fp8bs_gemm",
    "fp8bs_moe_gemm", "fp8bs_w8a16_gemm", "fp8bs_moe_route", "fp8bs_moe_quant_scatter",
    "fp8bs_moe_combine", "w8a16_gemm", "fp8bs_gemm_ue8m0", "fp8bs_weight_quant_ue8m0",
    "fp8_gemm_ue8m0", "fp8bs_mla_absorb_key", "fp8bs_mla_absorb_value", "mla_absorb_key",
    "mla_absorb_value", "act_quant", "weight_quant", "weight_dequant", "fp8_gemm", "moe_gemm", "linear", "moe_route",
    "moe_quant_scatter", "moe_combine", "MlaCache", "mla_cache_alloc", "fp8bs_mla_cache_write", "mla_cache_write",
    "fp8bs_mla_attention", "mla_attention", "fp8bs_cache_update", "cache_update", "fp8bs_cache_compact",
    "cache_compact",
]

SCALE_FP32 = 0
SCALE_UE8M0 = 1
OUT_BF16 = 0
OUT_F32 = 1
CACHE_BF16 = 0
CACHE_FP8 = 1
BLOCK = 128
MLA_RANK = 512      # latent width of the MLA cache
MLA_ROPE = 64       # its rotated width

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8bs.so")
_lib = None


class Fp8bsError(RuntimeError):
    """A non-zero status returned by the C ABI."""

    def __init__(self, fn: str, status: int):
        msg = lib().fp8bs_status_string(status).decode()
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded ``libfp8bs.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is missing: build it with "
                           "`python -m block_scaled_fp8_03_amd.build`")
    L = ctypes.CDLL(library_path)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.fp8bs_status_string.argtypes = [I]
    L.fp8bs_status_string.restype = ctypes.c_char_p
    L.fp8bs_version.restype = I
    L.fp8bs_act_quant.argtypes = [P, P, P, I64, I64, I, P]
    L.fp8bs_e4m3_encode.argtypes = [P, P, I64, P]
    L.fp8bs_weight_quant.argtypes = [P, P, P, I64, I64, P]
    L.fp8bs_weight_dequant.argtypes = [P, P, P, I64, I64, P]
    L.fp8bs_gemm.argtypes = [P, P, P, P, P, I64, I64, I64, I, P]
    L.fp8bs_moe_gemm.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, I, P]
    L.fp8bs_w8a16_gemm.argtypes = [P, P, P, P, I64, I64, I64, I, P]
    L.fp8bs_gemm_ue8m0.argtypes = [P, P, P, P, P, I64, I64, I64, I, P]
    L.fp8bs_weight_quant_ue8m0.argtypes = [P, P, P, I64, I64, P]
    L.fp8bs_moe_route_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_moe_route_workspace_size.restype = I64
    L.fp8bs_moe_route.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P]
    L.fp8bs_moe_route_noalloc.argtypes = [P, I64, I64, I64, P, P, P, P]
    L.fp8bs_moe_quant_scatter.argtypes = [P, P, P, P, I64, I64, I64, I64, I, P]
    L.fp8bs_moe_combine.argtypes = [P, P, P, P, I64, I64, I64, I64, I, P]
    L.fp8bs_mla_absorb_key.argtypes = [P, I64, I64, P, P, P, I64, I64, I64, I64, I64, I, P]
    L.fp8bs_mla_absorb_value.argtypes = [P, I64, I64, P, P, P, I64, I64, I64, I64, I64, I, P]
    F = ctypes.c_float
    L.fp8bs_mla_cache_write.argtypes = [P, I64, I64, P, I64, P, I, F, P, I64, P, P, P, P, I, P, P, P,
                                        I64, I64, I64, I64, I64, I64, I64, I64, P]
    L.fp8bs_mla_attention_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_mla_attention.argtypes = [P, I64, I64, P, I64, I64, P, P, P, I, P, P, P, F, I, P, I, P,
                                      I64, I64, I64, I64, I64, I64, I64, I64, P, I64, P]
    L.fp8bs_cache_update_workspace_size.argtypes = [I64, I64, I64, I64]
    L.fp8bs_cache_update.argtypes = [P, P, P, I, P, P, P, P, P, P, I64, I64, I64, I64, I64, I64, I64, P, I64, P]
    L.fp8bs_cache_compact_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_cache_compact.argtypes = [P, P, P, I, P, P, P, P, I64, I64, I64, I64, I64, I64, P, I64, P]
    for fn in ("fp8bs_mla_attention_workspace_size", "fp8bs_cache_update_workspace_size",
               "fp8bs_cache_compact_workspace_size"):
        getattr(L, fn).restype = I64
    for fn in ("fp8bs_mla_cache_write", "fp8bs_mla_attention", "fp8bs_cache_update", "fp8bs_cache_compact",
               "fp8bs_act_quant", "fp8bs_weight_quant", "fp8bs_weight_dequant", "fp8bs_gemm",
               "fp8bs_moe_gemm", "fp8bs_w8a16_gemm", "fp8bs_moe_route", "fp8bs_moe_quant_scatter",
               "fp8bs_moe_combine", "fp8bs_gemm_ue8m0", "fp8bs_weight_quant_ue8m0",
               "fp8bs_mla_absorb_key", "fp8bs_mla_absorb_value"):
        getattr(L, fn).restype = I
    _lib = L
    return L


# ---------------------------------------------------------------- marshalling

_F8 = (torch.float8_e4m3fn, torch.uint8)


def _need(t: torch.Tensor, dtypes, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _call(fn: str, *args) -> None:
    st = getattr(lib(), fn)(*args)
    if st != 0:
        raise Fp8bsError(fn, st)


def _fmt(scale_fmt) -> int:
    if scale_fmt in (SCALE_FP32, "fp32", None):
        return SCALE_FP32
    if scale_fmt in (SCALE_UE8M0, "ue8m0"):
        return SCALE_UE8M0
    raise ValueError(f"unknown scale_fmt {scale_fmt!r}")


def _out_code(c: torch.Tensor) -> int:
    if c.dtype == torch.bfloat16:
        return OUT_BF16
    if c.dtype == torch.float32:
        return OUT_F32
    raise TypeError(f"output dtype {c.dtype} is neither bfloat16 nor float32")


# ------------------------------------------------------- raw C-named wrappers

def fp8bs_act_quant(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, scale_fmt=SCALE_FP32) -> None:
    """x bf16 [M, K] -> q e4m3 [M, K], s float32 [M, K/128] (outputs preallocated)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    if tuple(q.shape) != (M, K) or tuple(s.shape) != (M, K // BLOCK if K % BLOCK == 0 else -1):
        raise ValueError("q must be [M, K] and s [M, K/128]")
    _call("fp8bs_act_quant", _need(x, (torch.bfloat16,), "x"), _need(q, _F8, "q"),
          _need(s, (torch.float32,), "s"), M, K, _fmt(scale_fmt), _stream(x))


def fp8bs_weight_quant(w: torch.Tensor, q: torch.Tensor, s: torch.Tensor, scale_fmt=SCALE_FP32) -> None:
    """w bf16 [N, K] -> q e4m3 [N, K], s float32 [ceil(N/128), ceil(K/128)]
    (scale_fmt "ue8m0": power-of-two block scales)."""
    N, K = w.shape
    if tuple(q.shape) != (N, K) or tuple(s.shape) != (-(-N // BLOCK), -(-K // BLOCK)):
        raise ValueError("q must be [N, K] and s [ceil(N/128), ceil(K/128)]")
    fn = "fp8bs_weight_quant_ue8m0" if _fmt(scale_fmt) == SCALE_UE8M0 else "fp8bs_weight_quant"
    _call(fn, _need(w, (torch.bfloat16,), "w"), _need(q, _F8, "q"), _need(s, (torch.float32,), "s"),
          N, K, _stream(w))


def fp8bs_weight_dequant(w: torch.Tensor, s: torch.Tensor, y: torch.Tensor) -> None:
    """w e4m3 [N, K], s float32 [ceil(N/128), ceil(K/128)] -> y bf16 [N, K]."""
    N, K = w.shape
    if tuple(s.shape) != (-(-N // BLOCK), -(-K // BLOCK)) or tuple(y.shape) != (N, K):
        raise ValueError("s must be [ceil(N/128), ceil(K/128)] and y [N, K]")
    _call("fp8bs_weight_dequant", _need(w, _F8, "w"), _need(s, (torch.float32,), "s"),
          _need(y, (torch.bfloat16,), "y"), N, K, _stream(w))


def fp8bs_gemm(a: torch.Tensor, a_s: torch.Tensor, b: torch.Tensor, b_s: torch.Tensor,
               c: torch.Tensor, ue8m0: bool = False) -> None:
    """C [M, N] (bf16 or float32, by c.dtype) = block-scaled A [M, K] . B [N, K]^T.
    ue8m0=True calls fp8bs_gemm_ue8m0 (all scales must be powers of two)."""
    M, K = a.shape
    N, K2 = b.shape
    if K != K2 or K % BLOCK:
        raise ValueError("A and B need the same K, a multiple of 128")
    if (tuple(a_s.shape) != (M, K // BLOCK) or tuple(b_s.shape) != (-(-N // BLOCK), K // BLOCK)
            or tuple(c.shape) != (M, N)):
        raise ValueError("scale or output shape mismatch")
    _call("fp8bs_gemm_ue8m0" if ue8m0 else "fp8bs_gemm", _need(a, _F8, "a"),
          _need(a_s, (torch.float32,), "a_s"),
          _need(b, _F8, "b"), _need(b_s, (torch.float32,), "b_s"),
          _need(c, (torch.bfloat16, torch.float32), "c"), M, N, K, _out_code(c), _stream(a))


def fp8bs_moe_gemm(a: torch.Tensor, a_s: torch.Tensor, b: torch.Tensor, b_s: torch.Tensor,
                   offsets: torch.Tensor, c: torch.Tensor) -> None:
    """Grouped GEMM: rows [offsets[e], offsets[e+1]) of A use expert e's B[e]."""
    R, K = a.shape
    E, N, K2 = b.shape
    if K != K2 or K % BLOCK:
        raise ValueError("A and B need the same K, a multiple of 128")
    if (tuple(a_s.shape) != (R, K // BLOCK) or tuple(b_s.shape) != (E, -(-N // BLOCK), K // BLOCK)
            or tuple(offsets.shape) != (E + 1,) or tuple(c.shape) != (R, N)):
        raise ValueError("scale, offsets or output shape mismatch")
    _call("fp8bs_moe_gemm", _need(a, _F8, "a"), _need(a_s, (torch.float32,), "a_s"),
          _need(b, _F8, "b"), _need(b_s, (torch.float32,), "b_s"),
          _need(offsets, (torch.int32,), "offsets"),
          _need(c, (torch.bfloat16, torch.float32), "c"), R, E, N, K, _out_code(c), _stream(a))


def fp8bs_w8a16_gemm(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, c: torch.Tensor) -> None:
    """The BF16 path: C [M, N] = x bf16 [M, K] . weight_dequant(w e4m3 [N, K], w_s)^T."""
    M, K = x.shape
    N, K2 = w.shape
    if K != K2 or K % BLOCK:
        raise ValueError("x and w need the same K, a multiple of 128")
    if tuple(w_s.shape) != (-(-N // BLOCK), K // BLOCK) or tuple(c.shape) != (M, N):
        raise ValueError("scale or output shape mismatch")
    _call("fp8bs_w8a16_gemm", _need(x, (torch.bfloat16,), "x"), _need(w, _F8, "w"),
          _need(w_s, (torch.float32,), "w_s"), _need(c, (torch.bfloat16, torch.float32), "c"),
          M, N, K, _out_code(c), _stream(x))


def fp8bs_moe_route(indices: torch.Tensor, E: int, offsets: torch.Tensor, row_token: torch.Tensor,
                    row_of: torch.Tensor, workspace: torch.Tensor) -> None:
    """Stable counting sort of routed expert ids int32 [T, topk] by expert:
    offsets [E+1], row_token [T*topk], row_of [T, topk] (see fp8bs.h)."""
    if indices.dim() != 2:
        raise ValueError("indices must be [T, topk]")
    T, topk = indices.shape
    need = lib().fp8bs_moe_route_workspace_size(T, topk, E)
    if need < 0:
        raise ValueError("sizes out of range")
    if (tuple(offsets.shape) != (E + 1,) or tuple(row_token.shape) != (T * topk,)
            or tuple(row_of.shape) != (T, topk)):
        raise ValueError("offsets must be [E+1], row_token [T*topk] and row_of [T, topk]")
    nbytes = workspace.numel() * workspace.element_size()
    ws = _need(workspace, (torch.uint8, torch.int32), "workspace") if nbytes else None
    _call("fp8bs_moe_route", _need(indices, (torch.int32,), "indices"), T, topk, E,
          _need(offsets, (torch.int32,), "offsets"), _need(row_token, (torch.int32,), "row_token"),
          _need(row_of, (torch.int32,), "row_of"), ws, nbytes, _stream(indices))


def fp8bs_e4m3_encode(x: torch.Tensor, q: torch.Tensor) -> None:
    """The float32 -> e4m3 conversion act_quant uses (RNE, saturating at 448):
    q e4m3 [n] from x float32 [n]."""
    if x.numel() != q.numel():
        raise ValueError("x and q need the same number of elements")
    _call("fp8bs_e4m3_encode", _need(x, (torch.float32,), "x"), _need(q, _F8, "q"),
          x.numel(), _stream(x))


def fp8bs_moe_route_noalloc(indices: torch.Tensor, E: int, offsets: torch.Tensor,
                            row_token: torch.Tensor, row_of: torch.Tensor) -> None:
    """fp8bs_moe_route without a workspace: the library's own device table
    (no allocation; calls overlapping on one GPU race, see fp8bs.h)."""
    if indices.dim() != 2:
        raise ValueError("indices must be [T, topk]")
    T, topk = indices.shape
    if (tuple(offsets.shape) != (E + 1,) or tuple(row_token.shape) != (T * topk,)
            or tuple(row_of.shape) != (T, topk)):
        raise ValueError("offsets must be [E+1], row_token [T*topk] and row_of [T, topk]")
    _call("fp8bs_moe_route_noalloc", _need(indices, (torch.int32,), "indices"), T, topk, E,
          _need(offsets, (torch.int32,), "offsets"), _need(row_token, (torch.int32,), "row_token"),
          _need(row_of, (torch.int32,), "row_of"), _stream(indices))


def fp8bs_moe_quant_scatter(x: torch.Tensor, row_of: torch.Tensor, q: torch.Tensor, s: torch.Tensor,
                            scale_fmt=SCALE_FP32) -> None:
    """act_quant of each token row of x bf16 [T, K] written to its routed rows
    of q e4m3 [R, K] and s float32 [R, K/128]."""
    T, K = x.shape
    R = q.shape[0]
    if row_of.dim() != 2 or row_of.shape[0] != T:
        raise ValueError("row_of must be [T, topk]")
    if tuple(q.shape) != (R, K) or K % BLOCK or tuple(s.shape) != (R, K // BLOCK):
        raise ValueError("q must be [R, K] and s [R, K/128], K a multiple of 128")
    _call("fp8bs_moe_quant_scatter", _need(x, (torch.bfloat16,), "x"),
          _need(row_of, (torch.int32,), "row_of"), _need(q, _F8, "q"),
          _need(s, (torch.float32,), "s"), T, row_of.shape[1], R, K, _fmt(scale_fmt), _stream(x))


def fp8bs_moe_combine(out: torch.Tensor, w: torch.Tensor, row_of: torch.Tensor, y: torch.Tensor) -> None:
    """y [T, N] = sum_k w[t, k] * out[row_of[t, k]] (out bf16 [R, N], y bf16 or float32)."""
    R, N = out.shape
    T, topk = w.shape
    if tuple(row_of.shape) != (T, topk) or tuple(y.shape) != (T, N):
        raise ValueError("row_of must be [T, topk] like w, and y [T, N]")
    _call("fp8bs_moe_combine", _need(out, (torch.bfloat16,), "out"), _need(w, (torch.float32,), "w"),
          _need(row_of, (torch.int32,), "row_of"), _need(y, (torch.bfloat16, torch.float32), "y"),
          T, topk, R, N, _out_code(y), _stream(out))


# ------------------------------------------------------ allocating wrappers

def act_quant(x: torch.Tensor, scale_fmt="fp32"):
    """x bf16 [..., K] -> (e4m3 [..., K], float32 [..., K/128])."""
    K = x.shape[-1]
    x2 = x.reshape(-1, K)
    q = torch.empty(x2.shape, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty((x2.shape[0], K // BLOCK), dtype=torch.float32, device=x.device)
    fp8bs_act_quant(x2, q, s, scale_fmt)
    return q.view(x.shape), s.view(*x.shape[:-1], K // BLOCK)


def weight_quant(w: torch.Tensor, scale_fmt="fp32"):
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty((-(-N // BLOCK), -(-K // BLOCK)), dtype=torch.float32, device=w.device)
    fp8bs_weight_quant(w, q, s, scale_fmt)
    return q, s


def weight_dequant(w: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    y = torch.empty(w.shape, dtype=torch.bfloat16, device=w.device)
    fp8bs_weight_dequant(w, s, y)
    return y


def fp8_gemm(a, a_s, b, b_s, out_dtype=torch.bfloat16) -> torch.Tensor:
    c = torch.empty((a.shape[0], b.shape[0]), dtype=out_dtype, device=a.device)
    fp8bs_gemm(a, a_s, b, b_s, c)
    return c


def fp8_gemm_ue8m0(a, a_s, b, b_s, out_dtype=torch.bfloat16) -> torch.Tensor:
    """fp8_gemm for power-of-two scales, the scales applied by the MFMA."""
    c = torch.empty((a.shape[0], b.shape[0]), dtype=out_dtype, device=a.device)
    fp8bs_gemm(a, a_s, b, b_s, c, ue8m0=True)
    return c


def moe_gemm(a, a_s, b, b_s, offsets, out_dtype=torch.bfloat16) -> torch.Tensor:
    c = torch.empty((a.shape[0], b.shape[1]), dtype=out_dtype, device=a.device)
    fp8bs_moe_gemm(a, a_s, b, b_s, offsets, c)
    return c


def linear(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, scale_fmt="fp32",
           out_dtype=torch.bfloat16) -> torch.Tensor:
    """The FP8 linear: act_quant(x) then the block-scaled GEMM with W (Admin
    guide 6.3, gemm_impl = "fp8")."""
    K = x.shape[-1]
    q, s = act_quant(x.reshape(-1, K), scale_fmt)
    y = fp8_gemm(q, s, w, w_s, out_dtype)
    return y.view(*x.shape[:-1], w.shape[0])


def moe_route(indices: torch.Tensor, E: int):
    """Routed expert ids int32 [T, topk] -> (offsets [E+1], row_token [T*topk],
    row_of [T, topk]), all int32 on the device; no host synchronisation."""
    T, topk = indices.shape
    dev = indices.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * topk, dtype=torch.int32, device=dev)
    row_of = torch.empty((T, topk), dtype=torch.int32, device=dev)
    need = lib().fp8bs_moe_route_workspace_size(T, topk, E)
    if need < 0:
        raise ValueError("sizes out of range")
    ws = torch.empty(max(need, 0), dtype=torch.uint8, device=dev)
    fp8bs_moe_route(indices, E, offsets, row_token, row_of, ws)
    return offsets, row_token, row_of


def moe_quant_scatter(x: torch.Tensor, row_of: torch.Tensor, R: int, scale_fmt="fp32"):
    """The expert inputs: (q e4m3 [R, K], s float32 [R, K/128])."""
    K = x.shape[-1]
    q = torch.empty((R, K), dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty((R, K // BLOCK), dtype=torch.float32, device=x.device)
    fp8bs_moe_quant_scatter(x, row_of, q, s, scale_fmt)
    return q, s


def moe_combine(out: torch.Tensor, w: torch.Tensor, row_of: torch.Tensor,
                out_dtype=torch.bfloat16) -> torch.Tensor:
    y = torch.empty((w.shape[0], out.shape[1]), dtype=out_dtype, device=out.device)
    fp8bs_moe_combine(out, w, row_of, y)
    return y


def _fp8bs_mla(fn: str, inp: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, out: torch.Tensor,
               dn: int, dv: int, value_side: bool) -> None:
    if inp.dim() != 3 or w.dim() != 2:
        raise ValueError("input must be [T, H, width] and wkv_b [H*(dn+dv), R]")
    T, H, width = inp.shape
    R = w.shape[1]
    if w.shape[0] != H * (dn + dv) or width != (R if value_side else dn):
        raise ValueError("wkv_b must be [H*(dn+dv), R]; q [T, H, dn] or x [T, H, R]")
    if tuple(w_s.shape) != (-(-w.shape[0] // BLOCK), -(-R // BLOCK)):
        raise ValueError("wkv_b_s must be [H*(dn+dv)/128, R/128]")
    if tuple(out.shape) != (T, H, dv if value_side else R):
        raise ValueError("out shape mismatch")
    if inp.dtype != torch.bfloat16 or not inp.is_cuda or (width > 1 and inp.stride(2) != 1):
        raise ValueError("input must be a bf16 device tensor with a contiguous last dimension")
    _call(fn, inp.data_ptr(), inp.stride(0), inp.stride(1), _need(w, _F8, "wkv_b"),
          _need(w_s, (torch.float32,), "wkv_b_s"), _need(out, (torch.bfloat16, torch.float32), "out"),
          T, H, dn, dv, R, _out_code(out), _stream(inp))


def fp8bs_mla_absorb_key(q: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, out: torch.Tensor,
                         dn: int, dv: int) -> None:
    """q bf16 [T, H, dn] (strided token/head dims allowed, e.g. the q_nope
    slice of q) -> out [T, H, R] = q_nope absorbed through the key rows of
    the FP8 wkv_b [H*(dn+dv), R]."""
    _fp8bs_mla("fp8bs_mla_absorb_key", q, w, w_s, out, dn, dv, False)


def fp8bs_mla_absorb_value(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, out: torch.Tensor,
                           dn: int, dv: int) -> None:
    """x bf16 [T, H, R] (the attention-weighted latent) -> out [T, H, dv]
    through the value rows of the FP8 wkv_b [H*(dn+dv), R]."""
    _fp8bs_mla("fp8bs_mla_absorb_value", x, w, w_s, out, dn, dv, True)


def mla_absorb_key(q, w, w_s, dn: int, dv: int, out_dtype=torch.bfloat16) -> torch.Tensor:
    out = torch.empty((q.shape[0], q.shape[1], w.shape[1]), dtype=out_dtype, device=q.device)
    fp8bs_mla_absorb_key(q, w, w_s, out, dn, dv)
    return out


def mla_absorb_value(x, w, w_s, dn: int, dv: int, out_dtype=torch.bfloat16) -> torch.Tensor:
    out = torch.empty((x.shape[0], x.shape[1], dv), dtype=out_dtype, device=x.device)
    fp8bs_mla_absorb_value(x, w, w_s, out, dn, dv)
    return out


def w8a16_gemm(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, out_dtype=torch.bfloat16) -> torch.Tensor:
    """x bf16 [..., K] times the dequantised FP8 weight [N, K]^T -> [..., N]."""
    K = x.shape[-1]
    x2 = x.reshape(-1, K)
    c = torch.empty((x2.shape[0], w.shape[0]), dtype=out_dtype, device=x.device)
    fp8bs_w8a16_gemm(x2, w, w_s, c)
    return c.view(*x.shape[:-1], w.shape[0])


# ------------------------------------------------------ the paged MLA cache

class MlaCache(NamedTuple):
    """A paged cache of MLA latents: ``latent`` [P, ps, 512] (bfloat16, or
    float8_e4m3fn codes), ``rope`` bfloat16 [P, ps, 64], and for codes ``scale``
    float32 [P, ps, 4], powers of two."""
    latent: torch.Tensor
    rope: torch.Tensor
    scale: Optional[torch.Tensor] = None


def mla_cache_alloc(pages: int, page_size: int, device, dtype=torch.bfloat16) -> MlaCache:
    """An empty cache of ``pages`` pages of ``page_size`` tokens (``dtype``
    torch.bfloat16 or torch.float8_e4m3fn); its contents are not initialised."""
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"cache dtype {dtype} is neither bfloat16 nor float8_e4m3fn")
    latent = torch.empty((pages, page_size, MLA_RANK), dtype=dtype, device=device)
    rope = torch.empty((pages, page_size, MLA_ROPE), dtype=torch.bfloat16, device=device)
    scale = None
    if dtype == torch.float8_e4m3fn:
        scale = torch.empty((pages, page_size, MLA_RANK // BLOCK), dtype=torch.float32, device=device)
    return MlaCache(latent, rope, scale)


_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_LATENT = (torch.bfloat16, *_F8)


def _ptr(t: torch.Tensor, name: str, dtypes, shape, dev) -> int:
    """The address of a contiguous tensor of one of `dtypes`, of `shape`, on device `dev`."""
    if getattr(t, "dtype", None) in dtypes and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.device != dev:
        raise ValueError(f"{name} lies on {t.device}, other tensors on {dev}")
    raise ValueError(f"{name} must be contiguous")


def _misfit(message: str, **tensors) -> Exception:
    """What to raise for arguments without the dimensions that `message` asks for."""
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            return TypeError(f"{name} must be a torch.Tensor")
    return ValueError(message)


def _rows3(t: torch.Tensor, name: str, shape, dev):
    """A bf16 [T, H, width] view with a dense last dimension: (pointer, token stride, head stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected bfloat16")
    if t.device != dev:
        raise ValueError(f"{name} lies on {t.device}, other tensors on {dev}")
    st, sh, sw = t.stride()
    T, H, _ = shape
    if sw != 1 and T * H > 0:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t.data_ptr(), (st if T > 1 else 0), (sh if H > 1 else 0)


def _cache_args(cache: MlaCache):
    """(device, latent, scale, rope, format, P, ps), checked but for the device's kind (_call_on)."""
    try:
        lat, rope, scale = cache
    except (TypeError, ValueError):
        raise TypeError("cache must be an MlaCache") from None
    try:
        dev = lat.device
        P, ps, _ = lat.shape
    except (AttributeError, ValueError):
        raise _misfit(f"cache.latent must be [P, ps, {MLA_RANK}]", **{"cache.latent": lat}) from None
    bf16 = lat.dtype == torch.bfloat16
    if bf16 != (scale is None):
        raise ValueError("cache.scale goes with a float8_e4m3fn cache, and only with one")
    return (dev, _ptr(lat, "cache.latent", _LATENT, (P, ps, MLA_RANK), dev),
            None if bf16 else _ptr(scale, "cache.scale", _F32, (P, ps, MLA_RANK // BLOCK), dev),
            _ptr(rope, "cache.rope", _BF16, (P, ps, MLA_ROPE), dev), CACHE_BF16 if bf16 else CACHE_FP8, P, ps)


def _scratch(workspace: Optional[torch.Tensor], dev):
    """(pointer, bytes) of a workspace."""
    n = 0 if workspace is None else workspace.numel()
    if not n:
        return None, 0
    return (_ptr(workspace, "workspace", (torch.uint8, torch.int32, torch.float32), workspace.shape, dev),
            n * workspace.element_size())


# the current stream's handle without the Stream object around it (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call_on(dev, fn: str, *args) -> None:
    """fn(*args, the current stream of device `dev`), with that device current."""
    if dev.type != "cuda":
        raise ValueError("cache.latent must be a device tensor")
    stream = _raw_stream(dev.index)
    if torch.cuda.current_device() == dev.index:
        _call(fn, *args, stream)
    else:
        with torch.cuda.device(dev):
            _call(fn, *args, stream)


def fp8bs_mla_cache_write(q_rope: torch.Tensor, kv: torch.Tensor, norm_w: torch.Tensor, eps: float,
                          rope_cs: torch.Tensor, q_out: torch.Tensor, cache: MlaCache, table: torch.Tensor,
                          cu_q: torch.Tensor, lens: torch.Tensor) -> None:
    """New tokens into the cache: kv bf16 [T, 576] (token stride free) normalised
    (norm_w [512] bf16 or float32), rotated and stored at the last positions of
    their sequences; q_rope bf16 [T, H, 64] (a slice of q may be passed) rotated
    into q_out bf16 [T, H, 64].  rope_cs float32 [n_pos, 32, 2] holds (cos, sin)."""
    try:
        (T, H, _), (_, _), (B, W), (n_pos, _, _) = q_rope.shape, kv.shape, table.shape, rope_cs.shape
    except (AttributeError, TypeError, ValueError):
        raise _misfit("q_rope must be [T, H, 64], kv [T, 576], table [B, W] and rope_cs [n_pos, 32, 2]",
                      q_rope=q_rope, kv=kv, table=table, rope_cs=rope_cs) from None
    dev, lat, scale, rope, fmt, P, ps = _cache_args(cache)
    qp, ldt, ldh = _rows3(q_rope, "q_rope", (T, H, MLA_ROPE), dev)
    if not isinstance(kv, torch.Tensor):
        raise TypeError("kv must be a torch.Tensor")
    if kv.shape != (T, MLA_RANK + MLA_ROPE) or kv.dtype != torch.bfloat16 or kv.device != dev or (T and kv.stride(1) != 1):
        raise ValueError(f"kv must be bfloat16 [{T}, {MLA_RANK + MLA_ROPE}] on {dev} with a contiguous last dimension")
    kp, ldk = kv.data_ptr(), (kv.stride(0) if T > 1 else 0)
    _call_on(dev, "fp8bs_mla_cache_write", qp, ldt, ldh, kp, ldk,
             _ptr(norm_w, "norm_w", (torch.bfloat16, torch.float32), (MLA_RANK,), dev), norm_w.dtype == torch.float32,
             eps, _ptr(rope_cs, "rope_cs", _F32, (n_pos, MLA_ROPE // 2, 2), dev), n_pos,
             _ptr(q_out, "q_out", _BF16, (T, H, MLA_ROPE), dev), lat, scale, rope, fmt,
             _ptr(table, "table", _I32, (B, W), dev), _ptr(cu_q, "cu_q", _I32, (B + 1,), dev),
             _ptr(lens, "lens", _I32, (B,), dev), T, H, B, W, P, ps, MLA_RANK, MLA_ROPE)


def mla_cache_write(q_rope, kv, norm_w, eps, rope_cs, cache: MlaCache, table, cu_q, lens) -> torch.Tensor:
    """fp8bs_mla_cache_write; returns the rotated queries [T, H, 64] (not
    initialised where the call writes none: tokens without a position)."""
    if not isinstance(q_rope, torch.Tensor):
        raise TypeError("q_rope must be a torch.Tensor")
    q_out = q_rope.new_empty(q_rope.shape)
    fp8bs_mla_cache_write(q_rope, kv, norm_w, eps, rope_cs, q_out, cache, table, cu_q, lens)
    return q_out


def fp8bs_mla_attention(q_lat: torch.Tensor, q_rope: torch.Tensor, cache: MlaCache, table: torch.Tensor,
                        cu_q: torch.Tensor, lens: torch.Tensor, scale: float, out: torch.Tensor,
                        lse: Optional[torch.Tensor], workspace: torch.Tensor, causal: bool = True) -> None:
    """The new tokens' attention over the cache: q_lat bf16 [T, H, 512] (from
    mla_absorb_key) and q_rope bf16 [T, H, 64] (from mla_cache_write), any token
    and head strides; out [T, H, 512] bf16 or float32, lse float32 [T, H] or None."""
    try:
        (T, H, _), (B, W) = q_lat.shape, table.shape
    except (AttributeError, TypeError, ValueError):
        raise _misfit(f"q_lat must be [T, H, {MLA_RANK}] and table [B, W]", q_lat=q_lat, table=table) from None
    dev, lat, sc, rope, fmt, P, ps = _cache_args(cache)
    qp, ldt, ldh = _rows3(q_lat, "q_lat", (T, H, MLA_RANK), dev)
    rp, ldrt, ldrh = _rows3(q_rope, "q_rope", (T, H, MLA_ROPE), dev)
    ws, nbytes = _scratch(workspace, dev)
    _call_on(dev, "fp8bs_mla_attention", qp, ldt, ldh, rp, ldrt, ldrh, lat, sc, rope, fmt,
             _ptr(table, "table", _I32, (B, W), dev), _ptr(cu_q, "cu_q", _I32, (B + 1,), dev),
             _ptr(lens, "lens", _I32, (B,), dev), scale, causal,
             _ptr(out, "out", (torch.bfloat16, torch.float32), (T, H, MLA_RANK), dev), _out_code(out),
             None if lse is None else _ptr(lse, "lse", _F32, (T, H), dev), T, H, B, W, P, ps, MLA_RANK, MLA_ROPE,
             ws, nbytes)


def mla_attention(q_lat, q_rope, cache: MlaCache, table, cu_q, lens, scale: float, causal: bool = True,
                  return_lse: bool = False, out_dtype=torch.bfloat16):
    """fp8bs_mla_attention: out [T, H, 512], with return_lse (out, lse); not
    initialised in rows behind the last sequence."""
    try:
        (T, H, _), (B, _) = q_lat.shape, table.shape
        new_empty = q_lat.new_empty
    except (AttributeError, TypeError, ValueError):
        raise _misfit(f"q_lat must be [T, H, {MLA_RANK}] and table [B, W]", q_lat=q_lat, table=table) from None
    need = lib().fp8bs_mla_attention_workspace_size(T, H, B)
    if need < 0:
        raise ValueError("sizes out of range")
    out = new_empty((T, H, MLA_RANK), dtype=out_dtype)
    lse = new_empty((T, H), dtype=torch.float32) if return_lse else None
    ws = new_empty(need, dtype=torch.uint8)
    fp8bs_mla_attention(q_lat, q_rope, cache, table, cu_q, lens, scale, out, lse, ws, causal)
    return (out, lse) if return_lse else out


def fp8bs_cache_update(cache: MlaCache, table: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor,
                       new_lens: torch.Tensor, table_out: torch.Tensor, lens_out: torch.Tensor,
                       workspace: Optional[torch.Tensor]) -> None:
    """The next step's rows: row i continues old row parent[i] (else it is
    empty) and is to hold new_lens[i] tokens; table_out [N, W], lens_out [N].
    Forks, frees, truncates, grows and copies on write (see fp8bs.h)."""
    try:
        (B, W), (N,) = table.shape, parent.shape
    except (AttributeError, TypeError, ValueError):
        raise _misfit("table must be [B, W] and parent [N]", table=table, parent=parent) from None
    dev, lat, sc, rope, fmt, P, ps = _cache_args(cache)
    ws, nbytes = _scratch(workspace, dev)
    _call_on(dev, "fp8bs_cache_update", lat, sc, rope, fmt, _ptr(table, "table", _I32, (B, W), dev),
             _ptr(lens, "lens", _I32, (B,), dev), _ptr(parent, "parent", _I32, (N,), dev),
             _ptr(new_lens, "new_lens", _I32, (N,), dev), _ptr(table_out, "table_out", _I32, (N, W), dev),
             _ptr(lens_out, "lens_out", _I32, (N,), dev), B, N, W, P, ps, MLA_RANK, MLA_ROPE, ws, nbytes)


def cache_update(cache: MlaCache, table, lens, parent, new_lens):
    """fp8bs_cache_update: (table_out [N, W], lens_out [N])."""
    try:
        (B, W), (N,), P = table.shape, parent.shape, cache[0].shape[0]
        new_empty = table.new_empty
    except (AttributeError, IndexError, TypeError, ValueError):
        _cache_args(cache)
        raise _misfit("table must be [B, W] and parent [N]", table=table, parent=parent) from None
    need = lib().fp8bs_cache_update_workspace_size(B, N, W, P)
    if need < 0:
        raise ValueError("sizes out of range")
    table_out, lens_out = new_empty((N, W)), new_empty(N)
    ws = new_empty((need + 3) // 4) if need else None
    fp8bs_cache_update(cache, table, lens, parent, new_lens, table_out, lens_out, ws)
    return table_out, lens_out


def fp8bs_cache_compact(cache: MlaCache, table: torch.Tensor, lens: torch.Tensor, table_out: torch.Tensor,
                        count: torch.Tensor, workspace: Optional[torch.Tensor]) -> None:
    """The pages that the rows use moved to the lowest indices; table_out
    [B, W] holds the new ones, count [1] (or a 0-d tensor) how many."""
    try:
        B, W = table.shape
        one = count.numel() == 1
    except (AttributeError, TypeError, ValueError):
        raise _misfit("table must be [B, W]", table=table, count=count) from None
    if not one:
        raise ValueError("count must hold one value")
    dev, lat, sc, rope, fmt, P, ps = _cache_args(cache)
    ws, nbytes = _scratch(workspace, dev)
    _call_on(dev, "fp8bs_cache_compact", lat, sc, rope, fmt, _ptr(table, "table", _I32, (B, W), dev),
             _ptr(lens, "lens", _I32, (B,), dev), _ptr(table_out, "table_out", _I32, (B, W), dev),
             _ptr(count, "count", _I32, count.shape, dev), B, W, P, ps, MLA_RANK, MLA_ROPE, ws, nbytes)


def cache_compact(cache: MlaCache, table, lens):
    """fp8bs_cache_compact: (table_out [B, W], count, a 0-d tensor)."""
    try:
        (B, W), P = table.shape, cache[0].shape[0]
        new_empty = table.new_empty
    except (AttributeError, IndexError, TypeError, ValueError):
        _cache_args(cache)
        raise _misfit("table must be [B, W]", table=table) from None
    need = lib().fp8bs_cache_compact_workspace_size(B, W, P)
    if need < 0:
        raise ValueError("sizes out of range")
    table_out, count = new_empty((B, W)), new_empty(())
    ws = new_empty((need + 3) // 4) if need else None
    fp8bs_cache_compact(cache, table, lens, table_out, count, ws)
    return table_out, count
