"""ctypes binding of the operators around the sampler (include/strata_tail.h).

``strata_norm_rows``, ``strata_project_rows``, ``strata_draw_rows`` and ``strata_tail_errors`` keep the C names
and write into the caller's tensors.  ``norm_rows``, ``project_rows`` and ``draw_rows`` allocate their outputs
(and the projection's workspace) with PyTorch, on the stream that they run on.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from ._binding import (STRATA_DTYPE_BF16, STRATA_DTYPE_F32, StrataError, _check, _logits_args, _stream, _typed,  # noqa: F401
                       lib)

STRATA_DTYPE_F8 = 2
STRATA_TAIL_MAX_WIDTH = 131072
STRATA_TAIL_MAX_ADAPTERS = 1024
STRATA_TAIL_MAX_RANK = 256

EXPORTED = ("strata_norm_rows", "strata_project_workspace", "strata_project_rows", "strata_draw_rows",
            "strata_tail_errors")

__all__ = ["norm_rows", "project_rows", "draw_rows", "tail_errors", "STRATA_DTYPE_F8", "STRATA_TAIL_MAX_WIDTH",
           "STRATA_TAIL_MAX_ADAPTERS", "STRATA_TAIL_MAX_RANK", *EXPORTED]


def _declare() -> None:
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    sig = {
        "strata_norm_rows": ([vp, i64, vp, i64, vp, i32, i32, i32, f32, vp, i64, vp, i64, vp, i64, vp, vp], i32),
        "strata_project_workspace": ([i32, i32, i32], i64),
        "strata_project_rows": ([vp, i64, vp, vp, i64, vp, i32, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, i64, vp,
                                 i64, vp], i32),
        "strata_draw_rows": ([vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "strata_tail_errors": ([ctypes.POINTER(ctypes.c_uint32), vp], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res


_declare()


def _rows(t, name, width=None, dtype=None, rows=None):
    """(address, row stride) of a [rows, width] CUDA tensor whose rows are contiguous; None -> (None, 0)."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, width] with contiguous rows")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if (width is not None and t.shape[1] != width) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected [{rows}, {width}]")
    return t.data_ptr(), int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), int(t.shape[1]))


def _vector(t, n, dtype, name) -> Optional[int]:
    if t is not None and (t.dim() != 1 or t.shape[0] != n):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected [{n}]")
    return _typed(t, dtype, name)


def _same_device(*tensors):
    import torch
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")


# ------------------------------------------------------------------------------ C-named calls
def strata_norm_rows(x, weight, residual=None, eps: float = 1e-6, residual_out=None, y=None, q=None, scale=None,
                     stream=None) -> None:
    import torch
    if x.dtype == torch.float32:
        dt = STRATA_DTYPE_F32
    elif x.dtype == torch.bfloat16:
        dt = STRATA_DTYPE_BF16
    else:
        raise TypeError(f"unsupported row dtype {x.dtype}")
    px, ldx = _rows(x, "x")
    T, H = int(x.shape[0]), int(x.shape[1])
    _same_device(x, weight, residual, residual_out, y, q, scale)
    pr, ldr = _rows(residual, "residual", H, x.dtype, T)
    pro, ldro = _rows(residual_out, "residual_out", H, x.dtype, T)
    py, ldy = _rows(y, "y", H, x.dtype, T)
    pq, ldq = _rows(q, "q", H, torch.float8_e4m3fn, T)
    _check(lib.strata_norm_rows(px, ldx, pr, ldr, _vector(weight, H, x.dtype, "weight"), dt, T, H, float(eps), pro, ldro,
                                py, ldy, pq, ldq, _vector(scale, T, torch.float32, "scale"), _stream(stream)))


def strata_project_workspace(T: int, S: int, R: int) -> int:
    return int(lib.strata_project_workspace(int(T), int(S), int(R)))


def strata_project_rows(x, w, y, x_scale=None, w_scale=None, a=None, b=None, row_adapter=None, adapter_scale=None,
                        workspace=None, stream=None) -> None:
    import torch
    if x.dtype == torch.bfloat16:
        dt = STRATA_DTYPE_BF16
    elif x.dtype == torch.float8_e4m3fn:
        dt = STRATA_DTYPE_F8
    else:
        raise TypeError(f"unsupported row dtype {x.dtype}")
    px, ldx = _rows(x, "x")
    T, K = int(x.shape[0]), int(x.shape[1])
    pw, ldw = _rows(w, "w", K, x.dtype)
    N = int(w.shape[0])
    _same_device(x, w, y, x_scale, w_scale, a, b, row_adapter, adapter_scale, workspace)
    py, ldy = _rows(y, "y", N, torch.bfloat16, T)
    S = R = 0
    if a is not None or b is not None:
        if a is None or b is None or row_adapter is None or adapter_scale is None:
            raise ValueError("a, b, row_adapter and adapter_scale go together")
        S, R = int(a.shape[0]), int(a.shape[1])
        if tuple(a.shape) != (S, R, K) or tuple(b.shape) != (S, N, R):
            raise ValueError(f"a is {tuple(a.shape)} and b {tuple(b.shape)}, expected [S, R, {K}] and [S, {N}, R]")
    _check(lib.strata_project_rows(
        px, ldx, _vector(x_scale, T, torch.float32, "x_scale"), pw, ldw, _vector(w_scale, N, torch.float32, "w_scale"), dt,
        T, N, K, _typed(a, torch.bfloat16, "a"), _typed(b, torch.bfloat16, "b"), S, R,
        _vector(row_adapter, T, torch.int32, "row_adapter") if S else None,
        _vector(adapter_scale, S, torch.float32, "adapter_scale") if S else None, py, ldy,
        _typed(workspace, torch.uint8, "workspace"), 0 if workspace is None else int(workspace.numel()), _stream(stream)))


def strata_draw_rows(logits, u, out_ids, temperature=None, top_k=None, top_p=None, min_p=None, out_lps=None, V=None,
                     stream=None) -> None:
    import torch
    ptr, dt, B, V, ld = _logits_args(logits, V)
    if B == 1:
        ld = max(ld, V + (-V) % 8)          # the stride of one row means nothing
    _same_device(logits, u, out_ids, temperature, top_k, top_p, min_p, out_lps)
    f32 = torch.float32
    _check(lib.strata_draw_rows(
        ptr, dt, B, V, ld, _vector(u, B, f32, "u"), _vector(temperature, B, f32, "temperature"),
        _vector(top_k, B, torch.int32, "top_k"), _vector(top_p, B, f32, "top_p"), _vector(min_p, B, f32, "min_p"),
        _vector(out_ids, B, torch.int32, "out_ids"), _vector(out_lps, B, f32, "out_lps"), _stream(stream)))


def strata_tail_errors(stream=None) -> int:
    bits = ctypes.c_uint32()
    _check(lib.strata_tail_errors(ctypes.byref(bits), _stream(stream)))
    return int(bits.value)


# ------------------------------------------------------------------------------ calls that allocate
class _on:
    """Allocate on the stream that the call runs on, so that the memory is not given away before it is done."""

    def __init__(self, stream, like):
        import torch
        self.ctx = None
        if stream is not None:
            self.ctx = torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)
                                         if isinstance(stream, int) else stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def norm_rows(x, weight, residual=None, eps: float = 1e-6, y: bool = True, f8: bool = False, stream=None,
              out=None) -> dict:
    """The norm of hidden rows: ``y`` and, with ``f8``, ``q`` and ``scale``; with a residual also ``residual``,
    the sum that the next layer adds to."""
    import torch
    o = out if out is not None else {}
    with _on(stream, x):
        if residual is not None and "residual" not in o:
            o["residual"] = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if y and "y" not in o:
            o["y"] = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if f8 and "q" not in o:
            o["q"] = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        if f8 and "scale" not in o:
            o["scale"] = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    strata_norm_rows(x, weight, residual, eps, o.get("residual"), o.get("y"), o.get("q"), o.get("scale"), stream)
    return o


def project_rows(x, w, x_scale=None, w_scale=None, a=None, b=None, row_adapter=None, adapter_scale=None, stream=None,
                 out=None):
    """``x w^T`` with the rows' low-rank adapters, as a bfloat16 [T, N] tensor."""
    import torch
    T, N = int(x.shape[0]), int(w.shape[0])
    need = strata_project_workspace(T, a.shape[0], a.shape[1]) if a is not None else 0
    with _on(stream, x):
        y = torch.empty(T, N, dtype=torch.bfloat16, device=x.device) if out is None else out
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    strata_project_rows(x, w, y, x_scale, w_scale, a, b, row_adapter, adapter_scale, ws, stream)
    return y


def draw_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, V=None, lps: bool = True, stream=None,
              out=None) -> dict:
    """One id per logit row from the random numbers ``u`` (one in [0, 1) for each row): ``ids`` and ``lps``."""
    import torch
    o = out if out is not None else {}
    with _on(stream, logits):
        if "ids" not in o:
            o["ids"] = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
        if lps and "lps" not in o:
            o["lps"] = torch.empty(logits.shape[0], dtype=torch.float32, device=logits.device)
    strata_draw_rows(logits, u, o["ids"], temperature, top_k, top_p, min_p, o.get("lps"), V, stream)
    return o


def tail_errors(stream=None) -> int:
    """The error bits that these calls' kernels raised on the current device since the last look (waits)."""
    return strata_tail_errors(stream)
