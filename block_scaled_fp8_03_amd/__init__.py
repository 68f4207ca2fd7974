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
``fp8bs_mla_cache_write``, ``fp8bs_cache_update``, ``fp8bs_cache_compact``, and
what stands between the FP8 products of a block with experts:
``fp8bs_rmsnorm``, ``fp8bs_moe_gate``, ``fp8bs_moe_balance``, ``fp8bs_swiglu``
with their gradients ``fp8bs_rmsnorm_bwd``, ``fp8bs_moe_gate_bwd``,
``fp8bs_swiglu_bwd`` and ``fp8bs_moe_combine_bwd``.
Allocating conveniences: ``act_quant``, ``weight_quant``, ``weight_dequant``,
``fp8_gemm``, ``moe_gemm``, ``linear``, ``w8a16_gemm``, ``moe_route``,
``moe_quant_scatter``, ``moe_combine``, ``mla_absorb_key``, ``mla_absorb_value``,
``mla_cache_alloc``, ``mla_cache_write``, ``mla_attention``, ``cache_update``,
``cache_compact``, ``rmsnorm``, ``rmsnorm_quant``, ``rmsnorm_bwd``, ``moe_gate``,
``moe_balance``, ``moe_gate_bwd``, ``swiglu``, ``swiglu_quant``, ``swiglu_bwd``,
``moe_combine_bwd``.

The operations follow the DeepSeek-V3 inference pages ("DeepSeek-V3
Administrator & Developer Guide", sections 6.3, 6.4, 8.5.1-8.5.3; "DeepSeek-V3
User Guide", FAQ on scale_fmt ue8m0).  Gradients are calls of their own (``*_bwd``):
no operator takes part in autograd, and what comes of a tensor that requires a
gradient is detached from it.  If the library has not been built the
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
    "cache_compact", "SCORE_SIGMOID", "SCORE_SOFTMAX", "fp8bs_rmsnorm", "rmsnorm", "rmsnorm_quant",
    "fp8bs_rmsnorm_bwd", "rmsnorm_bwd", "fp8bs_moe_gate", "moe_gate", "fp8bs_moe_balance", "moe_balance",
    "fp8bs_moe_gate_bwd", "moe_gate_bwd", "fp8bs_swiglu", "swiglu", "swiglu_quant", "fp8bs_swiglu_bwd", "swiglu_bwd",
    "fp8bs_moe_combine_bwd", "moe_combine_bwd",
]

SCALE_FP32 = 0
SCALE_UE8M0 = 1
OUT_BF16 = 0
OUT_F32 = 1
SCORE_SIGMOID = 0
SCORE_SOFTMAX = 1
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
    L.fp8bs_rmsnorm.argtypes = [P, I64, P, P, I, P, I, F, P, P, P, I, I64, I64, P]
    L.fp8bs_rmsnorm_bwd_workspace_size.argtypes = [I64, I64]
    L.fp8bs_rmsnorm_bwd.argtypes = [P, P, I64, I, P, I, F, P, P, P, I64, I64, P, I64, P]
    L.fp8bs_moe_gate.argtypes = [P, I64, I, P, I64, I64, I64, I64, I64, I, I, F, P, P, P]
    L.fp8bs_moe_balance_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_moe_balance.argtypes = [P, I64, I, P, P, I64, I64, I64, I64, I, P, P, P, P, I64, P]
    L.fp8bs_moe_gate_bwd.argtypes = [P, I64, I, P, P, I, I, F, P, P, P, I64, I64, I64, I64, P, I, P]
    L.fp8bs_swiglu.argtypes = [P, I64, P, I64, P, P, P, P, I, I64, I64, P]
    L.fp8bs_swiglu_bwd.argtypes = [P, P, I64, P, I64, P, P, I64, P, I64, I64, I64, P]
    L.fp8bs_moe_combine_bwd.argtypes = [P, I, P, P, P, P, P, I64, I64, I64, I64, P]
    L.fp8bs_mla_attention_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_mla_attention.argtypes = [P, I64, I64, P, I64, I64, P, P, P, I, P, P, P, F, I, P, I, P,
                                      I64, I64, I64, I64, I64, I64, I64, I64, P, I64, P]
    L.fp8bs_cache_update_workspace_size.argtypes = [I64, I64, I64, I64]
    L.fp8bs_cache_update.argtypes = [P, P, P, I, P, P, P, P, P, P, I64, I64, I64, I64, I64, I64, I64, P, I64, P]
    L.fp8bs_cache_compact_workspace_size.argtypes = [I64, I64, I64]
    L.fp8bs_cache_compact.argtypes = [P, P, P, I, P, P, P, P, I64, I64, I64, I64, I64, I64, P, I64, P]
    for fn in ("fp8bs_mla_attention_workspace_size", "fp8bs_cache_update_workspace_size",
               "fp8bs_cache_compact_workspace_size", "fp8bs_rmsnorm_bwd_workspace_size",
               "fp8bs_moe_balance_workspace_size"):
        getattr(L, fn).restype = I64
    for fn in ("fp8bs_mla_cache_write", "fp8bs_mla_attention", "fp8bs_cache_update", "fp8bs_cache_compact",
               "fp8bs_act_quant", "fp8bs_weight_quant", "fp8bs_weight_dequant", "fp8bs_gemm",
               "fp8bs_moe_gemm", "fp8bs_w8a16_gemm", "fp8bs_moe_route", "fp8bs_moe_quant_scatter",
               "fp8bs_moe_combine", "fp8bs_gemm_ue8m0", "fp8bs_weight_quant_ue8m0",
               "fp8bs_mla_absorb_key", "fp8bs_mla_absorb_value", "fp8bs_rmsnorm", "fp8bs_rmsnorm_bwd",
               "fp8bs_moe_gate", "fp8bs_moe_balance", "fp8bs_moe_gate_bwd", "fp8bs_swiglu", "fp8bs_swiglu_bwd",
               "fp8bs_moe_combine_bwd"):
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


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call_on(dev, fn: str, *args) -> None:
    """fn(*args, the current stream of device `dev`), with that device current."""
    if dev.type != "cuda":
        raise ValueError("cache.latent must be a device tensor")
    stream = _raw_stream(dev.index)
    if _current_device() == dev.index:
        st = getattr(lib(), fn)(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = getattr(lib(), fn)(*args, stream)
    if st != 0:
        raise Fp8bsError(fn, st)


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


# ------------------------------------------- what stands between the products
#
# Each operator's raw form checks its outputs and the allocating one makes them;
# both hand their addresses to one function that checks the inputs and calls (the
# checks of a tensor cost as much as its allocation: 1 us).

_FLOATS = (torch.bfloat16, torch.float32)
_EMPTY, _ONE = torch.Size([]), torch.Size([1])


def _rows2(t: torch.Tensor, name: str, dtypes, shape, dev):
    """A [M, width] view with a dense last dimension: (pointer, row stride)."""
    if getattr(t, "dtype", None) in dtypes and t.shape == shape and t.device == dev:
        sm, sw = t.stride()
        M, width = shape
        if sw == 1 or M == 0 or width <= 1:
            return t.data_ptr(), (sm if M > 1 else 0)
        raise ValueError(f"{name} must have a contiguous last dimension")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} lies on {t.device}, other tensors on {dev}")


def _opt(t: Optional[torch.Tensor], name: str, dtypes, shape, dev) -> Optional[int]:
    return None if t is None else _ptr(t, name, dtypes, shape, dev)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    """The address of a tensor that was made here."""
    return None if t is None else t.data_ptr()


def _count(n_rows: Optional[torch.Tensor], dev) -> Optional[int]:
    """The address of a count of rows on the device: one int32."""
    if n_rows is None:
        return None
    return _ptr(n_rows, "n_rows", _I32, _EMPTY if getattr(n_rows, "shape", None) == _EMPTY else _ONE, dev)


def _score(score) -> int:
    if score in (SCORE_SIGMOID, "sigmoid"):
        return SCORE_SIGMOID
    if score in (SCORE_SOFTMAX, "softmax"):
        return SCORE_SOFTMAX
    raise ValueError(f"unknown score {score!r}")


def _shape2(t, message: str, name: str):
    """The two sizes of a 2-D tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise _misfit(message, **{name: t})
    return t.shape


def _main2(t: torch.Tensor, name: str, dtypes, sizes: str):
    """The tensor that the others go by, a [M, width] view with a dense last
    dimension: (M, width, device, pointer, row stride)."""
    try:
        M, width = t.shape
        sm, sw = t.stride()
        dev = t.device
        fits = t.dtype in dtypes
    except (AttributeError, TypeError, ValueError):
        raise _misfit(f"{name} must be [{sizes}]", **{name: t}) from None
    if not fits:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if sw != 1 and M > 0 and width > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return M, width, dev, t.data_ptr(), (sm if M > 1 else 0)


def _launch(first: str, dev, fn, *args) -> None:
    """fn(*args, the current stream of `dev`), with that device current; `first` names the tensor that lies there."""
    index = dev.index
    if index is None:                                # what is not on a device has none
        raise ValueError(f"{first} must be a device tensor")
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        raise Fp8bsError(fn.__name__, st)


def _rmsnorm(dev, xp, ld, M, K, res, norm_w, eps, res_out, y, q, s, scale_fmt) -> None:
    """fp8bs_rmsnorm of x and outputs given by their addresses."""
    res_f32 = res is not None and getattr(res, "dtype", None) == torch.float32
    _launch("x", dev, lib().fp8bs_rmsnorm, xp, ld, _opt(res, "res", _FLOATS, (M, K), dev), res_out,
            OUT_F32 if res_f32 else OUT_BF16, _ptr(norm_w, "norm_w", _FLOATS, (K,), dev),
            norm_w.dtype == torch.float32, eps, y, q, s, _fmt(scale_fmt), M, K)


def fp8bs_rmsnorm(x: torch.Tensor, res: Optional[torch.Tensor], res_out: Optional[torch.Tensor], norm_w: torch.Tensor,
                  eps: float, y: Optional[torch.Tensor], q: Optional[torch.Tensor], s: Optional[torch.Tensor],
                  scale_fmt=SCALE_FP32) -> None:
    """RMSNorm of x + res: x bf16 [M, K] (row stride free), res [M, K] bf16 or
    float32 or None, the sum into res_out (res itself if you like), the norm
    times norm_w [K] (bf16 or float32) into y bf16 [M, K] and / or as codes q
    e4m3 [M, K] with scales s float32 [M, K/128]."""
    M, K, dev, xp, ld = _main2(x, "x", _BF16, "M, K")
    like = (getattr(res, "dtype", None),) if getattr(res, "dtype", None) in _FLOATS else _FLOATS
    _rmsnorm(dev, xp, ld, M, K, res, norm_w, eps, _opt(res_out, "res_out", like, (M, K), dev),
             _opt(y, "y", _BF16, (M, K), dev), _opt(q, "q", _F8, (M, K), dev), _opt(s, "s", _F32, (M, K // BLOCK), dev), scale_fmt)


def rmsnorm(x, norm_w, eps: float, residual=None):
    """fp8bs_rmsnorm: y bf16 [M, K]; with a residual (y, x + residual)."""
    M, K, dev, xp, ld = _main2(x, "x", _BF16, "M, K")
    y = x.new_empty(M, K, dtype=torch.bfloat16)
    h = None if residual is None else x.new_empty(M, K, dtype=getattr(residual, "dtype", None))
    _rmsnorm(dev, xp, ld, M, K, residual, norm_w, eps, _at(h), y.data_ptr(), None, None, SCALE_FP32)
    return y if residual is None else (y, h)


def rmsnorm_quant(x, norm_w, eps: float, residual=None, scale_fmt="fp32", return_y: bool = False):
    """fp8bs_rmsnorm: (q e4m3 [M, K], s float32 [M, K/128]), then y bf16 if
    return_y, then x + residual if there is a residual."""
    M, K, dev, xp, ld = _main2(x, "x", _BF16, "M, K")
    q, s = x.new_empty(M, K, dtype=torch.float8_e4m3fn), x.new_empty(M, K // BLOCK, dtype=torch.float32)
    y = x.new_empty(M, K, dtype=torch.bfloat16) if return_y else None
    h = None if residual is None else x.new_empty(M, K, dtype=getattr(residual, "dtype", None))
    _rmsnorm(dev, xp, ld, M, K, residual, norm_w, eps, _at(h), _at(y), q.data_ptr(), s.data_ptr(), scale_fmt)
    return tuple(t for t in (q, s, y, h) if t is not None)


def _rmsnorm_bwd(dev, hp, ld, M, K, dy, h, norm_w, eps, dres, dx, dw, ws, nbytes) -> None:
    """fp8bs_rmsnorm_bwd of h and outputs given by their addresses."""
    _launch("h", dev, lib().fp8bs_rmsnorm_bwd, _ptr(dy, "dy", _BF16, (M, K), dev), hp, ld, _out_code(h),
            _ptr(norm_w, "norm_w", _FLOATS, (K,), dev), norm_w.dtype == torch.float32, eps,
            _opt(dres, "dres", (h.dtype,), (M, K), dev), dx, dw, M, K, ws, nbytes)


def fp8bs_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, norm_w: torch.Tensor, eps: float,
                      dres: Optional[torch.Tensor], dx: torch.Tensor, dw: Optional[torch.Tensor],
                      workspace: Optional[torch.Tensor]) -> None:
    """The norm's gradient: dy bf16 [M, K], h [M, K] what was normalised (bf16 or
    float32, row stride free), dres [M, K] of h's type or None, added to dx [M, K]
    of h's type (dx itself if you like); dw float32 [K] or None."""
    M, K, dev, hp, ld = _main2(h, "h", _FLOATS, "M, K")
    _rmsnorm_bwd(dev, hp, ld, M, K, dy, h, norm_w, eps, dres, _ptr(dx, "dx", (h.dtype,), (M, K), dev),
                 _opt(dw, "dw", _F32, (K,), dev), *_scratch(workspace, dev))


def rmsnorm_bwd(dy, h, norm_w, eps: float, dres=None):
    """fp8bs_rmsnorm_bwd: (dx [M, K] of h's type, dw float32 [K])."""
    M, K, dev, hp, ld = _main2(h, "h", _FLOATS, "M, K")
    need = lib().fp8bs_rmsnorm_bwd_workspace_size(M, K)
    if need < 0:
        raise ValueError("sizes out of range")
    dx, dw = h.new_empty(M, K, dtype=h.dtype), h.new_empty(K, dtype=torch.float32)
    ws = h.new_empty(need, dtype=torch.uint8) if need else None
    _rmsnorm_bwd(dev, hp, ld, M, K, dy, h, norm_w, eps, dres, dx.data_ptr(), dw.data_ptr(), _at(ws), need)
    return dx, dw


def _moe_gate(dev, zp, ld, T, E, logits, topk, bias, groups, topk_groups, score, normalize, route_scale, indices,
              weights) -> None:
    """fp8bs_moe_gate of logits and outputs given by their addresses."""
    _launch("logits", dev, lib().fp8bs_moe_gate, zp, ld, _out_code(logits), _opt(bias, "bias", _F32, (E,), dev), T, E,
            topk, groups, topk_groups, _score(score), normalize, route_scale, indices, weights)


def fp8bs_moe_gate(logits: torch.Tensor, bias: Optional[torch.Tensor], groups: int, topk_groups: int, score,
                   normalize: bool, route_scale: float, indices: torch.Tensor, weights: torch.Tensor) -> None:
    """The gate: logits [T, E] (bf16 or float32, row stride free) -> indices
    int32 [T, topk] (-1 where no expert is left) and weights float32 [T, topk]."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    topk = _shape2(indices, "indices must be [T, topk]", "indices")[1]
    _moe_gate(dev, zp, ld, T, E, logits, topk, bias, groups, topk_groups, score, normalize, route_scale,
              _ptr(indices, "indices", _I32, (T, topk), dev), _ptr(weights, "weights", _F32, (T, topk), dev))


def moe_gate(logits, topk: int, bias=None, groups: int = 1, topk_groups: Optional[int] = None, score="sigmoid",
             normalize: bool = True, route_scale: float = 1.0):
    """fp8bs_moe_gate: (indices int32 [T, topk], weights float32 [T, topk]), for
    moe_route and moe_combine.  All groups are kept unless topk_groups says so."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    indices, weights = logits.new_empty(T, topk, dtype=torch.int32), logits.new_empty(T, topk, dtype=torch.float32)
    _moe_gate(dev, zp, ld, T, E, logits, topk, bias, groups, groups if topk_groups is None else topk_groups, score,
              normalize, route_scale, indices.data_ptr(), weights.data_ptr())
    return indices, weights


def _sequences(cu_seq: Optional[torch.Tensor], dev):
    """(pointer, sequences) of boundaries [S + 1]; one sequence without them."""
    if cu_seq is None:
        return None, 1
    if not isinstance(cu_seq, torch.Tensor) or cu_seq.dim() != 1 or cu_seq.shape[0] < 1:
        raise _misfit("cu_seq must be [S + 1]", cu_seq=cu_seq)
    return _ptr(cu_seq, "cu_seq", _I32, cu_seq.shape, dev), cu_seq.shape[0] - 1


def _moe_balance(dev, zp, ld, T, E, logits, indices, cu, S, score, counts, probs, loss, ws, nbytes) -> None:
    """fp8bs_moe_balance of logits, boundaries and outputs given by their addresses."""
    topk = _shape2(indices, "indices must be [T, topk]", "indices")[1]
    _launch("logits", dev, lib().fp8bs_moe_balance, zp, ld, _out_code(logits),
            _ptr(indices, "indices", _I32, (T, topk), dev), cu, T, S, E, topk, _score(score), counts, probs, loss, ws, nbytes)


def fp8bs_moe_balance(logits: torch.Tensor, indices: torch.Tensor, cu_seq: Optional[torch.Tensor], score,
                      counts: torch.Tensor, probs: torch.Tensor, loss: torch.Tensor,
                      workspace: Optional[torch.Tensor]) -> None:
    """Of each sequence (cu_seq int32 [S + 1]; None: one of all tokens): counts
    int32 [S, E] of the gate's indices [T, topk], probs float32 [S, E] the mean
    share of the token's scores, loss float32 [S]."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    cu, S = _sequences(cu_seq, dev)
    _moe_balance(dev, zp, ld, T, E, logits, indices, cu, S, score, _ptr(counts, "counts", _I32, (S, E), dev),
                 _ptr(probs, "probs", _F32, (S, E), dev), _ptr(loss, "loss", _F32, (S,), dev), *_scratch(workspace, dev))


def moe_balance(logits, indices, cu_seq=None, score="sigmoid"):
    """fp8bs_moe_balance: (loss float32 [S], counts int32 [S, E], probs float32 [S, E])."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    cu, S = _sequences(cu_seq, dev)
    need = lib().fp8bs_moe_balance_workspace_size(T, S, E)
    if need < 0:
        raise ValueError("sizes out of range")
    counts, probs = logits.new_empty(S, E, dtype=torch.int32), logits.new_empty(S, E, dtype=torch.float32)
    loss = logits.new_empty(S, dtype=torch.float32)
    ws = logits.new_empty(need, dtype=torch.uint8) if need else None
    _moe_balance(dev, zp, ld, T, E, logits, indices, cu, S, score, counts.data_ptr(), probs.data_ptr(),
                 loss.data_ptr(), _at(ws), need)
    return loss, counts, probs


def _moe_gate_bwd(dev, zp, ld, T, E, logits, indices, d_weights, score, normalize, route_scale, cu_seq, counts, d_loss,
                  d_logits, out_code) -> None:
    """fp8bs_moe_gate_bwd of logits and an output given by their addresses."""
    topk = _shape2(indices, "indices must be [T, topk]", "indices")[1]
    cu, S = _sequences(cu_seq, dev)
    _launch("logits", dev, lib().fp8bs_moe_gate_bwd, zp, ld, _out_code(logits),
            _ptr(indices, "indices", _I32, (T, topk), dev), _opt(d_weights, "d_weights", _F32, (T, topk), dev),
            _score(score), normalize, route_scale, cu, _opt(counts, "counts", _I32, (S, E), dev),
            _opt(d_loss, "d_loss", _F32, (S,), dev), T, S, E, topk, d_logits, out_code)


def fp8bs_moe_gate_bwd(logits: torch.Tensor, indices: torch.Tensor, d_weights: Optional[torch.Tensor], score,
                       normalize: bool, route_scale: float, cu_seq: Optional[torch.Tensor],
                       counts: Optional[torch.Tensor], d_loss: Optional[torch.Tensor], d_logits: torch.Tensor) -> None:
    """The gradient by the logits of the gate's weights (d_weights float32 [T,
    topk] or None) and of the balance losses (d_loss float32 [S] with their
    counts, or None): d_logits [T, E] bf16 or float32."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    _moe_gate_bwd(dev, zp, ld, T, E, logits, indices, d_weights, score, normalize, route_scale, cu_seq, counts, d_loss,
                  _ptr(d_logits, "d_logits", _FLOATS, (T, E), dev), _out_code(d_logits))


def moe_gate_bwd(logits, indices, d_weights=None, score="sigmoid", normalize: bool = True, route_scale: float = 1.0,
                 cu_seq=None, counts=None, d_loss=None, out_dtype=torch.float32) -> torch.Tensor:
    """fp8bs_moe_gate_bwd: d_logits [T, E]."""
    T, E, dev, zp, ld = _main2(logits, "logits", _FLOATS, "T, E")
    d_logits = logits.new_empty(T, E, dtype=out_dtype)
    _moe_gate_bwd(dev, zp, ld, T, E, logits, indices, d_weights, score, normalize, route_scale, cu_seq, counts, d_loss,
                  d_logits.data_ptr(), _out_code(d_logits))
    return d_logits


def _swiglu(dev, gp, ldg, M, N, up, y, q, s, scale_fmt, n_rows) -> None:
    """fp8bs_swiglu of the gate and outputs given by their addresses."""
    up_, ldu = _rows2(up, "up", _BF16, (M, N), dev)
    _launch("gate", dev, lib().fp8bs_swiglu, gp, ldg, up_, ldu, _count(n_rows, dev), y, q, s, _fmt(scale_fmt), M, N)


def fp8bs_swiglu(gate: torch.Tensor, up: torch.Tensor, y: Optional[torch.Tensor], q: Optional[torch.Tensor],
                 s: Optional[torch.Tensor], scale_fmt=SCALE_FP32, n_rows: Optional[torch.Tensor] = None) -> None:
    """silu(gate) * up, both bf16 [M, N] (row strides free, e.g. the halves of one
    product's output), into y bf16 [M, N] and / or as codes q e4m3 [M, N] with
    scales s float32 [M, N/128].  Rows from n_rows (one int32 on the device, e.g.
    offsets[-1:] of moe_route) on are left alone."""
    M, N, dev, gp, ldg = _main2(gate, "gate", _BF16, "M, N")
    _swiglu(dev, gp, ldg, M, N, up, _opt(y, "y", _BF16, (M, N), dev), _opt(q, "q", _F8, (M, N), dev),
            _opt(s, "s", _F32, (M, N // BLOCK), dev), scale_fmt, n_rows)


def swiglu(gate, up, n_rows=None) -> torch.Tensor:
    """fp8bs_swiglu: bf16 [M, N], not initialised from row n_rows on."""
    M, N, dev, gp, ldg = _main2(gate, "gate", _BF16, "M, N")
    y = gate.new_empty(M, N, dtype=torch.bfloat16)
    _swiglu(dev, gp, ldg, M, N, up, y.data_ptr(), None, None, SCALE_FP32, n_rows)
    return y


def swiglu_quant(gate, up, scale_fmt="fp32", n_rows=None, return_y: bool = False):
    """fp8bs_swiglu: (q e4m3 [M, N], s float32 [M, N/128]), then y bf16 if
    return_y; not initialised from row n_rows on."""
    M, N, dev, gp, ldg = _main2(gate, "gate", _BF16, "M, N")
    q, s = gate.new_empty(M, N, dtype=torch.float8_e4m3fn), gate.new_empty(M, N // BLOCK, dtype=torch.float32)
    y = gate.new_empty(M, N, dtype=torch.bfloat16) if return_y else None
    _swiglu(dev, gp, ldg, M, N, up, _at(y), q.data_ptr(), s.data_ptr(), scale_fmt, n_rows)
    return (q, s, y) if return_y else (q, s)


def fp8bs_swiglu_bwd(dy: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, dgate: torch.Tensor, dup: torch.Tensor,
                     n_rows: Optional[torch.Tensor] = None) -> None:
    """The gradient of fp8bs_swiglu: dy bf16 [M, N] -> dgate, dup bf16 [M, N] (row
    strides free, e.g. the halves of one tensor); rows from n_rows on are left alone."""
    M, N, dev, gp, ldg = _main2(gate, "gate", _BF16, "M, N")
    up_, ldu = _rows2(up, "up", _BF16, (M, N), dev)
    dgp, lddg = _rows2(dgate, "dgate", _BF16, (M, N), dev)
    dup_, lddu = _rows2(dup, "dup", _BF16, (M, N), dev)
    _launch("gate", dev, lib().fp8bs_swiglu_bwd, _ptr(dy, "dy", _BF16, (M, N), dev), gp, ldg, up_, ldu,
            _count(n_rows, dev), dgp, lddg, dup_, lddu, M, N)


def swiglu_bwd(dy, gate, up, n_rows=None):
    """fp8bs_swiglu_bwd: (dgate, dup) bf16 [M, N], the halves of one [M, 2N]
    tensor; not initialised from row n_rows on."""
    M, N = _shape2(gate, "gate must be [M, N]", "gate")
    d = gate.new_empty(M, 2 * N, dtype=torch.bfloat16)
    dgate, dup = d[:, :N], d[:, N:]
    fp8bs_swiglu_bwd(dy, gate, up, dgate, dup, n_rows)
    return dgate, dup


def _moe_combine_bwd(dy, out, R, N, w, T, topk, row_of, d_out, d_w) -> None:
    """fp8bs_moe_combine_bwd of outputs given by their addresses."""
    dev = out.device
    _launch("out", dev, lib().fp8bs_moe_combine_bwd, _ptr(dy, "dy", _FLOATS, (T, N), dev), _out_code(dy),
            _ptr(out, "out", _BF16, (R, N), dev), _ptr(w, "w", _F32, (T, topk), dev),
            _ptr(row_of, "row_of", _I32, (T, topk), dev), d_out, d_w, T, topk, R, N)


def fp8bs_moe_combine_bwd(dy: torch.Tensor, out: torch.Tensor, w: torch.Tensor, row_of: torch.Tensor,
                          d_out: torch.Tensor, d_w: torch.Tensor) -> None:
    """The gradient of fp8bs_moe_combine: dy [T, N] bf16 or float32 -> d_out bf16
    [R, N] (rows without a pair untouched) and d_w float32 [T, topk]."""
    R, N = _shape2(out, "out must be [R, N]", "out")
    T, topk = _shape2(w, "w must be [T, topk]", "w")
    dev = out.device
    _moe_combine_bwd(dy, out, R, N, w, T, topk, row_of, _ptr(d_out, "d_out", _BF16, (R, N), dev),
                     _ptr(d_w, "d_w", _F32, (T, topk), dev))


def moe_combine_bwd(dy, out, w, row_of):
    """fp8bs_moe_combine_bwd: (d_out bf16 [R, N], d_w float32 [T, topk]); rows
    of d_out that no pair maps to are not initialised."""
    R, N = _shape2(out, "out must be [R, N]", "out")
    T, topk = _shape2(w, "w must be [T, topk]", "w")
    d_out, d_w = out.new_empty(R, N, dtype=torch.bfloat16), out.new_empty(T, topk, dtype=torch.float32)
    _moe_combine_bwd(dy, out, R, N, w, T, topk, row_of, d_out.data_ptr(), d_w.data_ptr())
    return d_out, d_w
