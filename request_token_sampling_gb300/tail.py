"""Binding of the operators around the sampler (include/strata_tail.h).

``strata_norm_rows``, ``strata_project_rows``, ``strata_draw_rows`` and ``strata_tail_errors`` keep the C names
and write into the caller's tensors.  ``norm_rows``, ``project_rows`` and ``draw_rows`` allocate their outputs
(and the projection's workspace) with PyTorch, on the stream that they run on.

The calls go through a small compiled module (csrc/tail_binding.cpp, loaded by the first of them), which checks the
tensors, allocates and makes the C call; ``lib`` holds the C functions themselves for ctypes.
"""
from __future__ import annotations

import ctypes
import os

from ._binding import _check, _stream, lib
from .build import MODULE_PATH

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


def _load_module() -> None:
    """Load the compiled half of this binding (csrc/tail_binding.cpp) at the first call of an operator: the rest of
    the package does not need it, nor PyTorch.  Like the library that it calls, it has to be built."""
    global _module
    global _norm, _project, _draw
    from importlib.machinery import ExtensionFileLoader
    from importlib.util import module_from_spec, spec_from_loader
    import torch  # noqa: F401  (its libraries and types come first)
    if not os.path.exists(MODULE_PATH):
        raise ImportError(f"the PyTorch binding is not built ({MODULE_PATH}); "
                          "run `python -c 'import __graft_entry__ as g; g.build()'`")
    loader = ExtensionFileLoader("_strata_tail", MODULE_PATH)
    module = module_from_spec(spec_from_loader("_strata_tail", loader))
    loader.exec_module(module)
    _norm, _project, _draw = module.norm, module.project, module.draw
    _module = module


_module = None


def _compiled():
    """The compiled module, loaded."""
    if _module is None:
        _load_module()
    return _module


def _norm(*args):
    _load_module()
    return _norm(*args)


def _project(*args):
    _load_module()
    return _project(*args)


def _draw(*args):
    _load_module()
    return _draw(*args)


def _done(out):
    """What a compiled call gave: its outputs, or a C error code."""
    if out.__class__ is int:
        _check(out)
    return out


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


# ------------------------------------------------------------------------------ C-named calls
def strata_norm_rows(x, weight, residual=None, eps: float = 1e-6, residual_out=None, y=None, q=None, scale=None,
                     stream=None) -> None:
    _done(_norm(x, weight, residual, eps, False, False, False, dict(residual=residual_out, y=y, q=q, scale=scale),
                _handle(stream)))


def strata_project_workspace(T: int, S: int, R: int) -> int:
    return int(lib.strata_project_workspace(int(T), int(S), int(R)))


def strata_project_rows(x, w, y, x_scale=None, w_scale=None, a=None, b=None, row_adapter=None, adapter_scale=None,
                        workspace=None, stream=None) -> None:
    _done(_project(x, w, x_scale, w_scale, a, b, row_adapter, adapter_scale, y, workspace, False, _handle(stream)))


def strata_draw_rows(logits, u, out_ids, temperature=None, top_k=None, top_p=None, min_p=None, out_lps=None, V=None,
                     stream=None) -> None:
    _done(_draw(logits, u, temperature, top_k, top_p, min_p, V, False, False, dict(ids=out_ids, lps=out_lps),
                _handle(stream)))


def strata_tail_errors(stream=None) -> int:
    bits = ctypes.c_uint32()
    _check(lib.strata_tail_errors(ctypes.byref(bits), _stream(stream)))
    return int(bits.value)


# ------------------------------------------------------------------------------ calls that allocate
def _side(stream, like):
    """A context in which PyTorch allocates for `stream`: memory of a call belongs to the stream it runs on, or
    the allocator could give it away before the call is done."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device) if isinstance(stream, int) else stream)


def norm_rows(x, weight, residual=None, eps: float = 1e-6, y: bool = True, f8: bool = False, stream=None,
              out=None) -> dict:
    """The norm of hidden rows: ``y`` and, with ``f8``, ``q`` and ``scale``; with a residual also ``residual``,
    the sum that the next layer adds to."""
    if stream is not None:
        with _side(stream, x):
            return norm_rows(x, weight, residual, eps, y, f8, None, out)
    return _done(_norm(x, weight, residual, eps, residual is not None, bool(y), bool(f8), {} if out is None else out, None))


def project_rows(x, w, x_scale=None, w_scale=None, a=None, b=None, row_adapter=None, adapter_scale=None, stream=None,
                 out=None):
    """``x w^T`` with the rows' low-rank adapters, as a bfloat16 [T, N] tensor.  Rows that are allocated here start on
    16 bytes, whatever N is: they can go to ``draw_rows`` and to the sampler as they are."""
    if stream is not None:
        with _side(stream, x):
            return project_rows(x, w, x_scale, w_scale, a, b, row_adapter, adapter_scale, None, out)
    return _done(_project(x, w, x_scale, w_scale, a, b, row_adapter, adapter_scale, out, None, True, None))


def draw_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, V=None, lps: bool = True, stream=None,
              out=None) -> dict:
    """One id per logit row from the random numbers ``u`` (one in [0, 1) for each row): ``ids`` and ``lps``."""
    if stream is not None:
        with _side(stream, logits):
            return draw_rows(logits, u, temperature, top_k, top_p, min_p, V, lps, None, out)
    return _done(_draw(logits, u, temperature, top_k, top_p, min_p, V, True, bool(lps), {} if out is None else out, None))


def tail_errors(stream=None) -> int:
    """The error bits that these calls' kernels raised on the current device since the last look (waits)."""
    return strata_tail_errors(stream)
