"""Binding of include/ssm_block.h: the norms before and after the scan and 8-bit activation
checkpoints.

As in ``binding``: argument marshalling only, every step of the computation runs in the
library's CUDA kernels on PyTorch's current stream (or ``stream``), and a missing library raises.
The marshalling itself is compiled (``csrc/block_binding.cpp``), since a token's call costs more on
the host than on the GPU; ``lib()`` gives the C entry points themselves.
A call on another ``stream`` behaves as under ``torch.cuda.stream(stream)``: its results and workspace
come from that stream's memory.  The caller orders it after what makes its inputs, keeps them until it is
done, and orders the use of its results after it.
Every tensor, and the stream, of a call belongs to the GPU of its first tensor, which need not be the
current one.
Activations are CUDA tensors [..., cols], float32 or bfloat16, whose last dimension is dense and
whose rows lie at one stride (a slice of a wider tensor is fine); parameters are contiguous fp32.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import SSM_BF16, SSM_F32, _check

SSM_NORM_FIRST = 1        # gated_norm: norm of y, then the gate
SSM_WGRAD_ACCUMULATE = 1  # wgrad: add to d_W
SSM_MAX_NORM_COLS = 32768

EXPORTED = ("ssm_add_norm_fwd", "ssm_add_norm_bwd", "ssm_add_layer_norm_fwd",
            "ssm_add_layer_norm_bwd", "ssm_gated_norm_fwd", "ssm_gated_norm_bwd",
            "ssm_norm_bwd_workspace_size", "ssm_ckpt8_save", "ssm_ckpt8_load",
            "ssm_ckpt8_wgrad_workspace_size", "ssm_ckpt8_wgrad")


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("cols", ctypes.c_int), ("group", ctypes.c_int),
                ("io", ctypes.c_int), ("res_io", ctypes.c_int), ("flags", ctypes.c_uint),
                ("eps", ctypes.c_float)]


class Ckpt8(NamedTuple):
    """An activation held in 8 bits: q int8 [..., cols], e uint8 [..., ceil(cols / 32)]; the value
    is q * 2^(e - 133) for any e below 255 (zeros hold zeros), NaN where e is 255."""
    q: torch.Tensor
    e: torch.Tensor


class AddNorm(NamedTuple):
    out: torch.Tensor
    res_out: torch.Tensor | None
    rstd: torch.Tensor | None
    res8: Ckpt8 | None
    x8: Ckpt8 | None
    out8: Ckpt8 | None


class AddLayerNorm(NamedTuple):
    out: torch.Tensor
    res_out: torch.Tensor | None
    mean: torch.Tensor | None
    rstd: torch.Tensor | None
    res8: Ckpt8 | None
    x8: Ckpt8 | None
    out8: Ckpt8 | None


class GatedNorm(NamedTuple):
    out: torch.Tensor
    rstd: torch.Tensor | None
    y8: Ckpt8 | None
    z8: Ckpt8 | None
    out8: Ckpt8 | None


_vp, _sz, _i, _u, _ll = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint,
                         ctypes.c_longlong)
_L = None


def lib():
    """The loaded library with this header's argument types set (raises if it is missing)."""
    global _L
    if _L is None:
        L = binding.lib()
        d = ctypes.POINTER(NormDesc)
        L.ssm_add_norm_fwd.argtypes = ([d, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll, _vp, _ll] +
                                       [_vp] * 8)
        L.ssm_add_norm_bwd.argtypes = ([d, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll] +
                                       [_vp] * 5 + [_vp, _ll, _vp, _ll, _vp, _vp, _vp, _sz, _vp])
        L.ssm_add_layer_norm_fwd.argtypes = ([d, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _ll, _vp,
                                              _ll] + [_vp] * 9)
        L.ssm_add_layer_norm_bwd.argtypes = ([d, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll] +
                                             [_vp] * 6 + [_vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp,
                                                          _sz, _vp])
        L.ssm_gated_norm_fwd.argtypes = [d, _vp, _ll, _vp, _ll, _vp, _vp, _ll] + [_vp] * 8
        L.ssm_gated_norm_bwd.argtypes = ([d, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ll, _vp, _vp,
                                          _vp, _vp, _vp, _ll, _vp, _ll, _vp, _vp, _sz, _vp])
        L.ssm_norm_bwd_workspace_size.argtypes = [d, _i]
        L.ssm_norm_bwd_workspace_size.restype = _sz
        L.ssm_ckpt8_save.argtypes = [_vp, _ll, _vp, _vp, _ll, _i, _i, _vp]
        L.ssm_ckpt8_load.argtypes = [_vp, _vp, _vp, _ll, _ll, _i, _i, _vp]
        L.ssm_ckpt8_wgrad_workspace_size.argtypes = [_ll, _i, _i, _i, _i]
        L.ssm_ckpt8_wgrad_workspace_size.restype = _sz
        L.ssm_ckpt8_wgrad.argtypes = [_vp, _ll, _vp, _vp, _vp, _ll, _i, _i, _i, _u, _vp, _sz, _vp]
        _L = L
    return _L


_IO = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_B = None


def _calls():
    """The compiled module that marshals the calls (csrc/block_binding.cpp)."""
    global _B
    if _B is None:
        lib()
        try:
            from . import _block
        except ImportError as e:
            raise RuntimeError("bwd_ssm_conv_gb300/_block.so is not built for this PyTorch: run "
                               "python -m bwd_ssm_conv_gb300.build") from e
        _block.use_ckpt8(Ckpt8)
        _B = _block
    return _B


# ---- residual add + RMSNorm -----------------------------------------------------------------

def ssm_add_norm_fwd(x, w=None, residual=None, scale=None, eps=1e-5, res_dtype=None, save8=False,
                     save_x8=False, save_out8=False, want_res=True, want_rstd=True, out=None,
                     stream=None) -> AddNorm:
    """s = residual + scale * x; out = w * s / sqrt(mean(s^2) + eps), per row of x [..., cols].

    ``residual`` (and s, returned as ``res_out``) is fp32 or of x's type; without a residual
    ``res_dtype`` sets that type.  ``save8`` / ``save_x8`` / ``save_out8``: also keep s, x or out as
    8-bit checkpoints (for ssm_add_norm_bwd, its d_scale, and the next projection's
    ssm_ckpt8_wgrad).  ``out`` = (out, res_out), preallocated, optional."""
    r = (_B or _calls()).add_norm_fwd(x, w, residual, scale, eps, res_dtype, save8, save_x8,
                                      save_out8, want_res, want_rstd, out, stream)
    if type(r) is int:
        _check("ssm_add_norm_fwd", r)
    return AddNorm(*r)


def ssm_norm_bwd_workspace_size(rows, cols, sums=1, group=0, io=SSM_BF16, res_io=SSM_F32) -> int:
    return int(lib().ssm_norm_bwd_workspace_size(NormDesc(rows, cols, group, io, res_io, 0, 1.0),
                                                 sums))


def ssm_add_norm_bwd(d_out, res, rstd, w=None, d_res_out=None, scale=None, x=None, res_dtype=None,
                     want_dres=True, want_dx=True, ws=None, out=None, stream=None) -> dict:
    """Backward of ssm_add_norm_fwd; returns {"d_res", "d_x", "d_w", "d_scale"} (None where not
    wanted or not applicable).

    ``res``: the forward's res_out, or its 8-bit checkpoint res8.  ``x`` (a tensor or a Ckpt8)
    is needed for d_scale only.  ``d_res_out``: the gradient that reaches res_out past the norm.
    The stream's type is that of ``res`` or ``d_res_out``, else ``res_dtype``, else d_out's.
    ``out`` = a dict of preallocated outputs with the same keys, optional."""
    into = out if out is None else (out["d_res"], out["d_x"], out["d_w"], out["d_scale"])
    r = (_B or _calls()).add_norm_bwd(d_out, res, rstd, w, d_res_out, scale, x, res_dtype,
                                      want_dres, want_dx, ws, into, stream)
    if type(r) is int:
        _check("ssm_add_norm_bwd", r)
    return {"d_res": r[0], "d_x": r[1], "d_w": r[2], "d_scale": r[3]} if out is None else out


# ---- residual add + layer norm ----------------------------------------------------------------

def ssm_add_layer_norm_fwd(x, w=None, b=None, residual=None, scale=None, eps=1e-5, res_dtype=None,
                           save8=False, save_x8=False, save_out8=False, want_res=True,
                           want_stats=True, out=None, stream=None) -> AddLayerNorm:
    """s = residual + scale * x; out = w * (s - mean) / sqrt(mean((s - mean)^2) + eps) + b, per row of
    x [..., cols]; mean and 1 / sqrt(...) are returned with ``want_stats``.  The other arguments are
    those of ssm_add_norm_fwd."""
    r = (_B or _calls()).add_layer_norm_fwd(x, w, residual, scale, eps, res_dtype, save8, save_x8,
                                            save_out8, want_res, want_stats, out, stream, b)
    if type(r) is int:
        _check("ssm_add_layer_norm_fwd", r)
    return AddLayerNorm(*r)


def ssm_add_layer_norm_bwd(d_out, res, mean, rstd, w=None, d_res_out=None, scale=None, x=None,
                           res_dtype=None, want_dres=True, want_dx=True, want_db=True, ws=None,
                           out=None, stream=None) -> dict:
    """Backward of ssm_add_layer_norm_fwd; returns {"d_res", "d_x", "d_w", "d_b", "d_scale"} (None
    where not wanted or not applicable).  ``mean`` and ``rstd`` are the forward's, the other
    arguments those of ssm_add_norm_bwd."""
    into = out if out is None else (out["d_res"], out["d_x"], out["d_w"], out["d_scale"],
                                    out["d_b"])
    r = (_B or _calls()).add_layer_norm_bwd(d_out, res, rstd, w, d_res_out, scale, x, res_dtype,
                                            want_dres, want_dx, ws, into, stream, mean, want_db)
    if type(r) is int:
        _check("ssm_add_layer_norm_bwd", r)
    return ({"d_res": r[0], "d_x": r[1], "d_w": r[2], "d_b": r[4], "d_scale": r[3]} if out is None
            else out)


# ---- gated RMSNorm ----------------------------------------------------------------------------

def ssm_gated_norm_fwd(y, z, w=None, group=0, eps=1e-5, norm_first=False, save8=False,
                       save_out8=False, want_rstd=True, out=None, stream=None) -> GatedNorm:
    """Per group of ``group`` columns (0: all) of y, z [..., cols]:
    out = w * v / sqrt(mean(v^2) + eps) with v = y silu(z), or, with ``norm_first``,
    out = w * y / sqrt(mean(y^2) + eps) * silu(z).

    ``save8``: keep y and z as 8-bit checkpoints for ssm_gated_norm_bwd; ``save_out8``: keep out
    for the next projection's ssm_ckpt8_wgrad.  ``out``: preallocated, optional."""
    r = (_B or _calls()).gated_norm_fwd(y, z, w, group, eps, SSM_NORM_FIRST if norm_first else 0,
                                        save8, save_out8, want_rstd, out, stream)
    if type(r) is int:
        _check("ssm_gated_norm_fwd", r)
    return GatedNorm(*r)


def ssm_gated_norm_bwd(d_out, y, z, rstd, w=None, group=0, norm_first=False, ws=None, out=None,
                       stream=None) -> dict:
    """Backward of ssm_gated_norm_fwd; returns {"d_y", "d_z", "d_w"} (d_w None without w).

    ``y`` and ``z``: the forward's inputs, or their 8-bit checkpoints y8 and z8.  ``out`` = a dict
    of preallocated outputs with the same keys, optional (d_z may be a slice of the gradient of a
    wider projection)."""
    into = out if out is None else (out["d_y"], out["d_z"], out["d_w"])
    r = (_B or _calls()).gated_norm_bwd(d_out, y, z, rstd, w, group,
                                        SSM_NORM_FIRST if norm_first else 0, ws, into, stream)
    if type(r) is int:
        _check("ssm_gated_norm_bwd", r)
    return {"d_y": r[0], "d_z": r[1], "d_w": r[2]} if out is None else out


# ---- 8-bit activation checkpoints ---------------------------------------------------------------

def ssm_ckpt8_save(x, out=None, stream=None) -> Ckpt8:
    """x [..., cols] as an 8-bit checkpoint (int8 values, one power-of-two scale per 32 columns)."""
    r = (_B or _calls()).ckpt8_save(x, out, stream)
    if type(r) is int:
        _check("ssm_ckpt8_save", r)
    return r


def ssm_ckpt8_load(c, dtype=torch.bfloat16, out=None, stream=None):
    """The values of a checkpoint, as ``dtype`` (both types hold them exactly)."""
    r = (_B or _calls()).ckpt8_load(c, dtype, out, stream)
    if type(r) is int:
        _check("ssm_ckpt8_load", r)
    return r


def ssm_ckpt8_wgrad_workspace_size(tokens, m, k, io=SSM_BF16, aligned=True) -> int:
    return int(lib().ssm_ckpt8_wgrad_workspace_size(tokens, m, k, io, 1 if aligned else 0))


def ssm_ckpt8_wgrad(g, x8, accumulate=False, ws=None, out=None, stream=None, debug_flags=0):
    """The gradient d_W [m][k] (fp32) of a projection y = x W^T from g = dL/dy [..., m] and the
    8-bit checkpoint x8 of x [..., k]: d_W = sum over rows of g x^T.  ``accumulate`` adds it to
    ``out``.  Where a bounded wait inside the kernel gave up, that part of d_W is NaN and the workspace's
    status is SSM_ERR_TIMEOUT: pass ``ws`` (ssm_ckpt8_wgrad_workspace_size bytes) and read it with
    ssm_scan_status(ws).  ``debug_flags``: SSM_DEBUG_NO_WAIT (tests of the error path only)."""
    flags = (SSM_WGRAD_ACCUMULATE if accumulate else 0) | debug_flags
    r = (_B or _calls()).ckpt8_wgrad(g, x8, flags, ws, out, stream)
    if type(r) is int:
        _check("ssm_ckpt8_wgrad", r)
    return r
