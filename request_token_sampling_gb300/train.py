"""Binding of the operators that score and train the end of a model (include/strata_train.h).

The ``strata_`` calls keep the C names and write into the caller's tensors.  ``layer_norm_rows``, ``cross_entropy_rows``,
``distill_rows`` and the ``_grad`` of each allocate their outputs and workspaces with PyTorch, on the stream that they run on.
A step of the end of a model is

    n = layer_norm_rows(x, weight, bias=bias, residual=residual)
    o = cross_entropy_rows(n["y"], head, ids)                                # loss, lse
    d = cross_entropy_grad(n["y"], head, ids, o["lse"], g)                   # dx, dw
    e = layer_norm_grad(d["dx"], n["residual"], weight, n["mean"], n["rstd"])  # dx, dweight, dbias

and a prompt's log-probabilities are ``-cross_entropy_rows(...)["loss"]``.  Automatic differentiation passes these calls by: the
``_grad`` of each is its way back, and a call of the others that it would have to record (an input requires a gradient, outside of
``torch.no_grad()``) warns.

Outputs of up to 32 KB that one call allocates share a storage: what keeps one of them, or writes its storage out
(``torch.save``), has them all; ``clone()`` parts them.
"""
from __future__ import annotations

import ctypes

from . import tail
from ._binding import lib
from .tail import _done, _handle, _side

STRATA_LOSS_MAX_ROWS = 131072
STRATA_LOSS_MAX_WIDTH = 32768
STRATA_DISTILL_MAX_TOKENS = 128

EXPORTED = ("strata_layer_norm_rows", "strata_layer_norm_workspace", "strata_layer_norm_grad", "strata_loss_workspace",
            "strata_cross_entropy_rows", "strata_cross_entropy_grad", "strata_distill_rows", "strata_distill_grad")

__all__ = ["layer_norm_rows", "layer_norm_grad", "cross_entropy_rows", "cross_entropy_grad", "distill_rows", "distill_grad",
           "STRATA_LOSS_MAX_ROWS", "STRATA_LOSS_MAX_WIDTH", "STRATA_DISTILL_MAX_TOKENS", *EXPORTED]


def _declare() -> None:
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    rows = [vp, i64, vp, i64, i32, i32, i32]
    sig = {
        "strata_layer_norm_rows": ([vp, i64, vp, i64, vp, vp, i32, i32, i32, f32, vp, i64, vp, i64, vp, vp, vp], i32),
        "strata_layer_norm_workspace": ([i32, i32], i64),
        "strata_layer_norm_grad": ([vp, i64, vp, i64, vp, vp, vp, vp, i64, i32, i32, i32, vp, i64, vp, vp, vp, i64, vp], i32),
        "strata_loss_workspace": ([i32, i32, i32, i32, i32], i64),
        "strata_cross_entropy_rows": (rows + [vp, vp, vp, vp, i64, vp], i32),
        "strata_cross_entropy_grad": (rows + [vp, vp, vp, vp, i64, vp, i64, vp, i64, vp], i32),
        "strata_distill_rows": (rows + [i32, vp, vp, f32, vp, vp, vp, i64, vp], i32),
        "strata_distill_grad": (rows + [i32, vp, vp, f32, vp, vp, vp, i64, vp, i64, vp, i64, vp], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res


_declare()


def _load(name):
    """The compiled call `name`, loaded; later calls go to it directly."""
    call = getattr(tail._compiled(), name)
    globals()["_" + name] = call
    return call


def _layer_norm(*args):
    return _load("layer_norm")(*args)


def _layer_norm_grad(*args):
    return _load("layer_norm_grad")(*args)


def _loss(*args):
    return _load("loss")(*args)


def _loss_grad(*args):
    return _load("loss_grad")(*args)


# ------------------------------------------------------------------------------ C-named calls
def strata_layer_norm_rows(x, weight, bias=None, residual=None, eps: float = 1e-5, residual_out=None, y=None, mean=None, rstd=None,
                           stream=None) -> None:
    _done(_layer_norm(x, weight, bias, residual, eps, False, False, False,
                      dict(residual=residual_out, y=y, mean=mean, rstd=rstd), _handle(stream)))


def strata_layer_norm_workspace(T: int, H: int) -> int:
    return int(lib.strata_layer_norm_workspace(int(T), int(H)))


def strata_layer_norm_grad(dy, x, weight, mean, rstd, dresidual=None, dx=None, dweight=None, dbias=None, workspace=None,
                           stream=None) -> None:
    _done(_layer_norm_grad(dy, x, weight, mean, rstd, dresidual, False, False, False,
                           dict(dx=dx, dweight=dweight, dbias=dbias), workspace, False, _handle(stream)))


def strata_loss_workspace(T: int, V: int, H: int, K: int = 0, grad: bool = False) -> int:
    return int(lib.strata_loss_workspace(int(T), int(V), int(H), int(K), int(bool(grad))))


def strata_cross_entropy_rows(x, w, ids, loss, lse, workspace, stream=None) -> None:
    _done(_loss(x, w, ids, None, 1.0, False, dict(loss=loss, lse=lse), workspace, False, _handle(stream)))


def strata_cross_entropy_grad(x, w, ids, lse, g, dx=None, dw=None, workspace=None, stream=None) -> None:
    _done(_loss_grad(x, w, ids, None, 1.0, lse, g, False, False, dict(dx=dx, dw=dw), workspace, False, _handle(stream)))


def strata_distill_rows(x, w, ids, teacher, temperature, loss, lse, workspace, stream=None) -> None:
    _done(_loss(x, w, ids, _teacher(teacher), temperature, False, dict(loss=loss, lse=lse), workspace, False,
                _handle(stream)))


def strata_distill_grad(x, w, ids, teacher, temperature, lse, g, dx=None, dw=None, workspace=None, stream=None) -> None:
    _done(_loss_grad(x, w, ids, _teacher(teacher), temperature, lse, g, False, False, dict(dx=dx, dw=dw), workspace,
                     False, _handle(stream)))


def _teacher(teacher):
    if teacher is None:
        raise TypeError("teacher must be a tensor")
    return teacher


# ------------------------------------------------------------------------------ calls that allocate
def layer_norm_rows(x, weight, bias=None, residual=None, eps: float = 1e-5, y: bool = True, stats: bool = True, stream=None,
                    out=None) -> dict:
    """The layer norm of hidden rows: ``y`` and, with ``stats``, the ``mean`` and ``rstd`` of each row, which the way back
    takes; with a residual also ``residual``, the sum that the next layer adds to."""
    if stream is not None:
        with _side(stream, x):
            return layer_norm_rows(x, weight, bias, residual, eps, y, stats, None, out)
    return _done(_layer_norm(x, weight, bias, residual, eps, residual is not None, bool(y), bool(stats),
                             {} if out is None else out, None))


def layer_norm_grad(dy, x, weight, mean, rstd, dresidual=None, dx: bool = True, dweight: bool = True, bias: bool = True, stream=None,
                    out=None) -> dict:
    """From the gradient of ``y``: ``dx`` (with ``dresidual``, the gradient that goes around the norm, added), ``dweight``
    and, with ``bias``, ``dbias``.  ``x`` are the rows that were normed: with a residual its sum."""
    if stream is not None:
        with _side(stream, x):
            return layer_norm_grad(dy, x, weight, mean, rstd, dresidual, dx, dweight, bias, None, out)
    return _done(_layer_norm_grad(dy, x, weight, mean, rstd, dresidual, bool(dx), bool(dweight), bool(bias),
                                  {} if out is None else out, None, True, None))


def cross_entropy_rows(x, w, ids, stream=None, out=None) -> dict:
    """``loss`` and ``lse`` of each row's logits ``x w^T`` for the token ``ids`` (int32; negative: the row is left out); the
    logits are not kept.  ``-loss`` is the token's log-probability."""
    if stream is not None:
        with _side(stream, x):
            return cross_entropy_rows(x, w, ids, None, out)
    return _done(_loss(x, w, ids, None, 1.0, True, {} if out is None else out, None, True, None))


def cross_entropy_grad(x, w, ids, lse, g, dx: bool = True, dw: bool = True, stream=None, out=None) -> dict:
    """``dx`` and ``dw`` of the sum of ``g * loss`` (``g``: float32, one for each row)."""
    if stream is not None:
        with _side(stream, x):
            return cross_entropy_grad(x, w, ids, lse, g, dx, dw, None, out)
    return _done(_loss_grad(x, w, ids, None, 1.0, lse, g, bool(dx), bool(dw), {} if out is None else out, None, True, None))


def distill_rows(x, w, ids, teacher, temperature: float = 1.0, stream=None, out=None) -> dict:
    """``loss`` and ``lse`` of each row's logits ``x w^T`` against a teacher's top tokens: ``ids`` [rows, tokens] (int32;
    negative: not there) and their logits or log-probabilities ``teacher`` (float32), as ``Sampler.logprobs`` gives them."""
    if stream is not None:
        with _side(stream, x):
            return distill_rows(x, w, ids, teacher, temperature, None, out)
    return _done(_loss(x, w, ids, _teacher(teacher), temperature, True, {} if out is None else out, None, True, None))


def distill_grad(x, w, ids, teacher, lse, g, temperature: float = 1.0, dx: bool = True, dw: bool = True, stream=None, out=None) -> dict:
    """``dx`` and ``dw`` of the sum of ``g * loss`` (``g``: float32, one for each row)."""
    if stream is not None:
        with _side(stream, x):
            return distill_grad(x, w, ids, teacher, lse, g, temperature, dx, dw, None, out)
    return _done(_loss_grad(x, w, ids, _teacher(teacher), temperature, lse, g, bool(dx), bool(dw),
                            {} if out is None else out, None, True, None))
