"""Binding of include/ssm_head.h: the head with its loss, cross entropy over the vocabulary or distillation
from a teacher's top logits, and its gradients.  The logits are never kept.

As in ``block``: argument marshalling only (compiled, ``csrc/block_binding.cpp``), every step of the
computation runs in the library's CUDA kernels on PyTorch's current stream (or ``stream``), and a missing
library raises.  Streams, devices and preallocated results are those of ``block``.
h [..., cols] and w [vocab, cols] are CUDA tensors of one type, float32 or bfloat16, whose last dimension
is dense and whose rows lie at one stride; the other arguments are contiguous.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding, block
from .binding import SSM_BF16, _check

SSM_MAX_HEAD_ENTRIES = 128
SSM_HEAD_FINE_G = 2

EXPORTED = ("ssm_head_workspace_size", "ssm_head_ce_fwd", "ssm_head_ce_bwd", "ssm_head_distill_fwd",
            "ssm_head_distill_bwd")


class HeadDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("cols", ctypes.c_int), ("vocab", ctypes.c_int),
                ("io", ctypes.c_int), ("entries", ctypes.c_int), ("entry_io", ctypes.c_int),
                ("temperature", ctypes.c_float), ("ignore_index", ctypes.c_longlong),
                ("flags", ctypes.c_uint)]


class HeadLoss(NamedTuple):
    loss: torch.Tensor
    lse: torch.Tensor | None


_vp, _sz, _i, _ll = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_longlong
_L = None


def lib():
    """The loaded library with this header's argument types set (raises if it is missing)."""
    global _L
    if _L is None:
        L = binding.lib()
        d = ctypes.POINTER(HeadDesc)
        ends, ws = [d, _vp, _ll, _vp, _ll], [_vp, _sz, _vp]
        L.ssm_head_workspace_size.argtypes = [d, _i, _i]
        L.ssm_head_workspace_size.restype = _sz
        L.ssm_head_ce_fwd.argtypes = ends + [_vp] * 3 + ws
        L.ssm_head_distill_fwd.argtypes = ends + [_vp] * 4 + ws
        L.ssm_head_ce_bwd.argtypes = ends + [_vp] * 4 + [_ll, _vp] + ws
        L.ssm_head_distill_bwd.argtypes = ends + [_vp] * 5 + [_ll, _vp] + ws
        _L = L
    return _L


def _calls():
    if _L is None:
        lib()
    return block._B or block._calls()


def ssm_head_workspace_size(rows, cols, vocab, io=SSM_BF16, entries=0, grads=0, aligned=True,
                            fine=False) -> int:
    """Bytes of ``ws``: ``entries`` 0 for cross entropy, ``grads`` 0 for the forward, else 1 (d_h) + 2
    (d_w); ``aligned``: w's rows are 16-byte aligned; ``fine``: as the backward's."""
    return int(lib().ssm_head_workspace_size(
        HeadDesc(rows, cols, vocab, io, entries, io, 1.0, -100, SSM_HEAD_FINE_G if fine else 0), grads,
        1 if aligned else 0))


def ssm_head_ce_fwd(h, w, target, ignore_index=-100, ws=None, out=None, stream=None,
                    debug_flags=0) -> HeadLoss:
    """Per row of h [..., cols]: loss = log sum_v exp(z_v) - z_target for z = h w^T, w [vocab, cols] and
    target int64 [...]; and lse, the first term, for the backward.

    Rows whose target is ``ignore_index`` have loss and lse 0, cost no product and are not read.  Any
    other target outside the vocabulary gives NaN in its row, and SSM_ERR_INVALID_ARG as the
    workspace's status: pass ``ws`` (ssm_head_workspace_size bytes) and read it with
    ssm_scan_status(ws).  ``out`` = (loss, lse), preallocated, optional.  ``debug_flags``:
    SSM_DEBUG_NO_WAIT (tests of the error path only)."""
    r = _calls().head_ce_fwd(h, w, target, ignore_index, ws, out, stream, debug_flags)
    if type(r) is int:
        _check("ssm_head_ce_fwd", r)
    return HeadLoss(*r)


def ssm_head_ce_bwd(h, w, target, lse, d_loss, ignore_index=-100, want_dh=True, want_dw=True, ws=None,
                    out=None, stream=None, debug_flags=0, fine=False) -> dict:
    """Backward of ssm_head_ce_fwd, given its lse and the gradient d_loss [...] of each row's loss; returns
    {"d_h", "d_w"} in the type of h and w (None where not wanted).  ``out`` = a dict of preallocated
    results with the same keys, optional.

    ``fine`` (bf16, more than 256 rows): the gradient of the logits, which is rounded to bf16 between the products
    otherwise, is kept to 16 bits in two terms, so that the results have no error but their own rounding; the
    backward takes twice the time.  Up to 256 rows, and fp32 ones, are as exact in either case."""
    into = out if out is None else (out["d_h"], out["d_w"])
    r = _calls().head_ce_bwd(h, w, target, ignore_index, lse, d_loss, want_dh, want_dw, ws, into, stream,
                             debug_flags | SSM_HEAD_FINE_G if fine else debug_flags)
    if type(r) is int:
        _check("ssm_head_ce_bwd", r)
    return {"d_h": r[0], "d_w": r[1]} if out is None else out


def ssm_head_distill_fwd(h, w, t_idx, t_logit, temperature=1.0, ws=None, out=None, stream=None,
                         debug_flags=0) -> HeadLoss:
    """Per row of h [..., cols]: tau^2 KL(p || q), with tau the ``temperature`` (1e-6 .. 1e6), p the softmax of a
    teacher's logits t_logit / tau over its entries (t_idx int64, both [..., entries], 1 .. 128 of
    them; an index below 0: no entry) and q that of h w^T / tau over the whole vocabulary; and lse of
    the latter, for the backward.  Rows without an entry have loss and lse 0, cost no product and are
    not read.  An index beyond the vocabulary gives NaN in its row; ``ws``, ``out`` and
    ``debug_flags`` as in ssm_head_ce_fwd."""
    r = _calls().head_distill_fwd(h, w, t_idx, t_logit, temperature, ws, out, stream, debug_flags)
    if type(r) is int:
        _check("ssm_head_distill_fwd", r)
    return HeadLoss(*r)


def ssm_head_distill_bwd(h, w, t_idx, t_logit, lse, d_loss, temperature=1.0, want_dh=True,
                         want_dw=True, ws=None, out=None, stream=None, debug_flags=0,
                         fine=False) -> dict:
    """Backward of ssm_head_distill_fwd, given its lse and the gradient d_loss [...] of each row's loss
    (the teacher's logits have none); results and ``fine`` as in ssm_head_ce_bwd."""
    into = out if out is None else (out["d_h"], out["d_w"])
    r = _calls().head_distill_bwd(h, w, t_idx, t_logit, temperature, lse, d_loss, want_dh, want_dw, ws,
                                  into, stream, debug_flags | SSM_HEAD_FINE_G if fine else debug_flags)
    if type(r) is int:
        _check("ssm_head_distill_bwd", r)
    return {"d_h": r[0], "d_w": r[1]} if out is None else out
