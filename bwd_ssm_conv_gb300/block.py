"""ctypes binding of include/ssm_block.h: the norms before and after the scan and 8-bit
activation checkpoints.

As in ``binding``: argument marshalling only, every step of the computation runs in the
library's CUDA kernels on PyTorch's current stream (or ``stream``), and a missing library raises.
Activations are CUDA tensors [..., cols], float32 or bfloat16, whose last dimension is dense and
whose rows lie at one stride (a slice of a wider tensor is fine); parameters are contiguous fp32.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple

import torch

from . import binding
from .binding import SSM_BF16, SSM_F32, _check

SSM_NORM_FIRST = 1        # gated_norm: norm of y, then the gate
SSM_WGRAD_ACCUMULATE = 1  # wgrad: add to d_W
SSM_MAX_NORM_COLS = 32768
SSM_CKPT8_BLOCK = 32

EXPORTED = ("ssm_add_norm_fwd", "ssm_add_norm_bwd", "ssm_gated_norm_fwd", "ssm_gated_norm_bwd",
            "ssm_norm_bwd_workspace_size", "ssm_ckpt8_save", "ssm_ckpt8_load",
            "ssm_ckpt8_wgrad_workspace_size", "ssm_ckpt8_wgrad")


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("cols", ctypes.c_int), ("group", ctypes.c_int),
                ("io", ctypes.c_int), ("res_io", ctypes.c_int), ("flags", ctypes.c_uint),
                ("eps", ctypes.c_float)]


class Ckpt8(NamedTuple):
    """An activation held in 8 bits: q int8 [..., cols], e uint8 [..., ceil(cols / 32)]; the value
    is q * 2^(e - 133), NaN where e is 255."""
    q: torch.Tensor
    e: torch.Tensor


class AddNorm(NamedTuple):
    out: torch.Tensor
    res_out: torch.Tensor | None
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


# What a call of given sizes needs besides its tensors; the same for every call of those sizes on a
# device, so it is worked out once.

@lru_cache(maxsize=1024)
def _desc(rows, cols, group, io, res_io, flags, eps):
    return NormDesc(rows, cols, group, io, res_io, flags, eps)


@lru_cache(maxsize=1024)
def _norm_ws(rows, cols, group, sums, device):
    with torch.cuda.device(device):
        return int(lib().ssm_norm_bwd_workspace_size(
            NormDesc(rows, cols, group, SSM_F32, SSM_F32, 0, 1.0), sums))


@lru_cache(maxsize=1024)
def _wgrad_ws(tokens, m, k, io, aligned, device):
    with torch.cuda.device(device):
        return int(lib().ssm_ckpt8_wgrad_workspace_size(tokens, m, k, io, aligned))


def _io(t: torch.Tensor, name: str) -> int:
    io = _IO.get(t.dtype)
    if io is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return io


def _rows(t, name, shape=None, dtype=None):
    """(pointer, row stride) of an activation [..., cols]; (None, 0) for None."""
    if t is None:
        return None, 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    return t.data_ptr(), _row_stride(name, t.shape, t.stride())


@lru_cache(maxsize=1024)
def _row_stride(name, shape, strides):
    """The one stride between the rows of a tensor that is not contiguous."""
    cols = shape[-1]
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    ld, span = None, None  # one stride for all rows: outer dimensions step over whole inner ones
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld, span = stride, size * stride
        elif stride != span:
            raise ValueError(f"{name}'s rows must lie at one stride")
        else:
            span *= size
    if ld is None:
        ld = cols
    if ld < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return ld


def _f32(t, name, n):
    """Pointer of a contiguous fp32 tensor of n elements; None for None."""
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of {n} elements")
    return t.data_ptr()


def _kept(c, name, shape):
    """Pointers of a checkpoint of an activation of that shape."""
    if c is None:
        return None, None
    q, e = c
    if not (q.dtype == torch.int8 and e.dtype == torch.uint8 and q.is_cuda and e.is_cuda and
            q.is_contiguous() and e.is_contiguous()):
        raise ValueError(f"{name} must hold contiguous int8 and uint8 CUDA tensors")
    if q.shape != shape or e.shape != (*shape[:-1], -(-shape[-1] // SSM_CKPT8_BLOCK)):
        raise ValueError(f"{name} must hold an activation of shape {tuple(shape)}, got "
                         f"{tuple(q.shape)} with scales {tuple(e.shape)}")
    return q.data_ptr(), e.data_ptr()


def _new_ckpt8(shape, device):
    return Ckpt8(torch.empty(shape, dtype=torch.int8, device=device),
                 torch.empty(*shape[:-1], -(-shape[-1] // SSM_CKPT8_BLOCK), dtype=torch.uint8,
                             device=device))


def _ptrs(c):
    return (None, None) if c is None else (c.q.data_ptr(), c.e.data_ptr())


def _on(stream, t, *made):
    """The call's stream (by default the current one of t's device); tensors made here for a stream
    other than the current one are marked as used there, so that their memory is not given out
    again before that stream is done."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    if stream != torch.cuda.current_stream(t.device):
        for m in made:
            for u in m if isinstance(m, tuple) else (m,):
                if u is not None:
                    u.record_stream(stream)
    return stream.cuda_stream


def _workspace(nbytes, device, ws):
    """(workspace, its bytes, the one made here)"""
    if ws is not None:
        size = ws.numel() * ws.element_size()
        if not ws.is_cuda or not ws.is_contiguous() or size < nbytes:
            raise ValueError("workspace too small (or not a contiguous CUDA tensor)")
        return ws, size, None
    if nbytes < 256:
        nbytes = 256
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, nbytes, ws


# ---- residual add + RMSNorm -----------------------------------------------------------------

def ssm_add_norm_fwd(x, w=None, residual=None, scale=None, eps=1e-5, res_dtype=None, save8=False,
                     save_x8=False, save_out8=False, want_res=True, want_rstd=True, out=None,
                     stream=None) -> AddNorm:
    """s = residual + scale * x; out = w * s / sqrt(mean(s^2) + eps), per row of x [..., cols].

    ``residual`` (and s, returned as ``res_out``) is fp32 or of x's type; without a residual
    ``res_dtype`` sets that type.  ``save8`` / ``save_x8`` / ``save_out8``: also keep s, x or out as
    8-bit checkpoints (for ssm_add_norm_bwd, its d_scale, and the next projection's
    ssm_ckpt8_wgrad).  ``out`` = (out, res_out), preallocated, optional."""
    io = _io(x, "x")
    shape, dev = x.shape, x.device
    cols = shape[-1]
    rdt = residual.dtype if residual is not None else (res_dtype or x.dtype)
    if out is None:
        o = torch.empty_like(x)
        res = (None if not want_res else torch.empty_like(residual) if residual is not None else
               torch.empty(shape, dtype=rdt, device=dev))
        po, pr = (o.data_ptr(), 0), (None if res is None else res.data_ptr(), 0)
    else:
        o, res = out
        po, pr = _rows(o, "out", shape, x.dtype), _rows(res, "res_out", shape, rdt)
    rows = x.numel() // cols if cols else 0
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if want_rstd else None
    res8 = _new_ckpt8(shape, dev) if save8 else None
    x8 = _new_ckpt8(shape, dev) if save_x8 else None
    out8 = _new_ckpt8(shape, dev) if save_out8 else None
    rc = (_L or lib()).ssm_add_norm_fwd(
        _desc(rows, cols, 0, io, _IO.get(rdt, -1), 0, eps), *_rows(x, "x"),
        *_rows(residual, "residual", shape), _f32(scale, "scale", cols), _f32(w, "w", cols), *po,
        *pr, None if rstd is None else rstd.data_ptr(), *_ptrs(res8), *_ptrs(x8), *_ptrs(out8),
        _on(stream, x, *(() if out is not None else (o, res)), rstd, res8, x8, out8))
    if rc:
        _check("ssm_add_norm_fwd", rc)
    return AddNorm(o, res, rstd, res8, x8, out8)


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
    io = _io(d_out, "d_out")
    shape, dev = d_out.shape, d_out.device
    cols = shape[-1]
    res8, x8 = isinstance(res, tuple), isinstance(x, tuple)
    rdt = (d_res_out.dtype if d_res_out is not None else
           res.dtype if not res8 else res_dtype or d_out.dtype)
    if out is None:
        d_res = (None if not want_dres else
                 torch.empty_like(d_res_out) if d_res_out is not None else
                 torch.empty(shape, dtype=rdt, device=dev))
        d_x = torch.empty_like(d_out) if want_dx else None
        d_w = torch.empty_like(w) if w is not None else None
        d_scale = torch.empty_like(scale) if scale is not None and x is not None else None
        g = dict(d_res=d_res, d_x=d_x, d_w=d_w, d_scale=d_scale)
        made = (d_res, d_x, d_w, d_scale)
    else:
        g, made = out, ()
        d_res, d_x, d_w, d_scale = g["d_res"], g["d_x"], g["d_w"], g["d_scale"]
    rows = d_out.numel() // cols if cols else 0
    sums = (d_w is not None) + (d_scale is not None)
    ws, size, mine = _workspace(_norm_ws(rows, cols, 0, sums, dev) if sums else 0, dev, ws)
    rc = (_L or lib()).ssm_add_norm_bwd(
        _desc(rows, cols, 0, io, _IO.get(rdt, -1), 0, 1.0), *_rows(d_out, "d_out"),
        *_rows(d_res_out, "d_res_out", shape, rdt),
        *_rows(None if res8 else res, "res", shape, rdt),
        *_kept(res if res8 else None, "res", shape),
        *_rows(None if x8 else x, "x", shape, d_out.dtype), *_kept(x if x8 else None, "x", shape),
        _f32(rstd, "rstd", rows), _f32(scale, "scale", cols), _f32(w, "w", cols),
        *_rows(d_res, "d_res", shape, rdt), *_rows(d_x, "d_x", shape, d_out.dtype),
        _f32(d_w, "d_w", cols), _f32(d_scale, "d_scale", cols), ws.data_ptr(), size,
        _on(stream, d_out, *made, mine))
    if rc:
        _check("ssm_add_norm_bwd", rc)
    return g


# ---- gated RMSNorm ----------------------------------------------------------------------------

def ssm_gated_norm_fwd(y, z, w=None, group=0, eps=1e-5, norm_first=False, save8=False,
                       save_out8=False, want_rstd=True, out=None, stream=None) -> GatedNorm:
    """Per group of ``group`` columns (0: all) of y, z [..., cols]:
    out = w * v / sqrt(mean(v^2) + eps) with v = y silu(z), or, with ``norm_first``,
    out = w * y / sqrt(mean(y^2) + eps) * silu(z).

    ``save8``: keep y and z as 8-bit checkpoints for ssm_gated_norm_bwd; ``save_out8``: keep out
    for the next projection's ssm_ckpt8_wgrad.  ``out``: preallocated, optional."""
    io = _io(y, "y")
    shape, dev = y.shape, y.device
    cols = shape[-1]
    if out is None:
        o = torch.empty_like(y)
        po = (o.data_ptr(), 0)
    else:
        o, po = out, _rows(out, "out", shape, y.dtype)
    groups = max(cols // group, 1) if group else 1
    rstd = torch.empty(*shape[:-1], groups, dtype=torch.float32, device=dev) if want_rstd else None
    y8 = _new_ckpt8(shape, dev) if save8 else None
    z8 = _new_ckpt8(shape, dev) if save8 else None
    out8 = _new_ckpt8(shape, dev) if save_out8 else None
    rc = (_L or lib()).ssm_gated_norm_fwd(
        _desc(y.numel() // cols if cols else 0, cols, group, io, io,
              SSM_NORM_FIRST if norm_first else 0, eps),
        *_rows(y, "y"), *_rows(z, "z", shape, y.dtype), _f32(w, "w", cols), *po,
        None if rstd is None else rstd.data_ptr(), *_ptrs(y8), *_ptrs(z8), *_ptrs(out8),
        _on(stream, y, None if out is not None else o, rstd, y8, z8, out8))
    if rc:
        _check("ssm_gated_norm_fwd", rc)
    return GatedNorm(o, rstd, y8, z8, out8)


def ssm_gated_norm_bwd(d_out, y, z, rstd, w=None, group=0, norm_first=False, ws=None, out=None,
                       stream=None) -> dict:
    """Backward of ssm_gated_norm_fwd; returns {"d_y", "d_z", "d_w"} (d_w None without w).

    ``y`` and ``z``: the forward's inputs, or their 8-bit checkpoints y8 and z8.  ``out`` = a dict
    of preallocated outputs with the same keys, optional (d_z may be a slice of the gradient of a
    wider projection)."""
    io = _io(d_out, "d_out")
    shape, dev = d_out.shape, d_out.device
    cols = shape[-1]
    if out is None:
        d_y, d_z = torch.empty_like(d_out), torch.empty_like(d_out)
        d_w = torch.empty_like(w) if w is not None else None
        g = dict(d_y=d_y, d_z=d_z, d_w=d_w)
        made = (d_y, d_z, d_w)
    else:
        g, made = out, ()
        d_y, d_z, d_w = g["d_y"], g["d_z"], g["d_w"]
    rows, groups = d_out.numel() // cols if cols else 0, cols // group if group else 1
    ws, size, mine = _workspace(_norm_ws(rows, cols, group, 1, dev) if d_w is not None else 0, dev,
                                ws)
    y8, z8 = isinstance(y, tuple), isinstance(z, tuple)
    rc = (_L or lib()).ssm_gated_norm_bwd(
        _desc(rows, cols, group, io, io, SSM_NORM_FIRST if norm_first else 0, 1.0),
        *_rows(d_out, "d_out"), *_rows(None if y8 else y, "y", shape, d_out.dtype),
        *_kept(y if y8 else None, "y", shape), *_rows(None if z8 else z, "z", shape, d_out.dtype),
        *_kept(z if z8 else None, "z", shape), _f32(rstd, "rstd", rows * groups),
        _f32(w, "w", cols), *_rows(d_y, "d_y", shape, d_out.dtype),
        *_rows(d_z, "d_z", shape, d_out.dtype), _f32(d_w, "d_w", cols), ws.data_ptr(), size,
        _on(stream, d_out, *made, mine))
    if rc:
        _check("ssm_gated_norm_bwd", rc)
    return g


# ---- 8-bit activation checkpoints ---------------------------------------------------------------

def ssm_ckpt8_save(x, out=None, stream=None) -> Ckpt8:
    """x [..., cols] as an 8-bit checkpoint (int8 values, one power-of-two scale per 32 columns)."""
    io = _io(x, "x")
    shape = x.shape
    cols = shape[-1]
    c = _new_ckpt8(shape, x.device) if out is None else out
    rc = (_L or lib()).ssm_ckpt8_save(
        *_rows(x, "x"), *(_ptrs(c) if out is None else _kept(c, "out", shape)),
        x.numel() // cols if cols else 0, cols, io, _on(stream, x, c if out is None else None))
    if rc:
        _check("ssm_ckpt8_save", rc)
    return c


def ssm_ckpt8_load(c, dtype=torch.bfloat16, out=None, stream=None):
    """The values of a checkpoint, as ``dtype`` (both types hold them exactly)."""
    q = c[0]
    shape = q.shape
    cols = shape[-1]
    if out is None:
        o = torch.empty(shape, dtype=dtype, device=q.device)
        po = (o.data_ptr(), 0)
    else:
        o, po = out, _rows(out, "out", shape)
    rc = (_L or lib()).ssm_ckpt8_load(*_kept(c, "c", shape), *po, q.numel() // cols if cols else 0,
                                      cols, _io(o, "out"),
                                      _on(stream, q, o if out is None else None))
    if rc:
        _check("ssm_ckpt8_load", rc)
    return o


def ssm_ckpt8_wgrad_workspace_size(tokens, m, k, io=SSM_BF16, aligned=True) -> int:
    return int(lib().ssm_ckpt8_wgrad_workspace_size(tokens, m, k, io, 1 if aligned else 0))


def ssm_ckpt8_wgrad(g, x8, accumulate=False, ws=None, out=None, stream=None):
    """The gradient d_W [m][k] (fp32) of a projection y = x W^T from g = dL/dy [..., m] and the
    8-bit checkpoint x8 of x [..., k]: d_W = sum over rows of g x^T.  ``accumulate`` adds it to
    ``out``."""
    io = _io(g, "g")
    m, k = g.shape[-1], x8[0].shape[-1]
    tokens = g.numel() // m if m else 0
    if accumulate and out is None:
        raise ValueError("accumulate needs the tensor to add to (out)")
    o = torch.empty(m, k, dtype=torch.float32, device=g.device) if out is None else out
    if out is not None and out.shape != (m, k):
        raise ValueError(f"out must have shape {(m, k)}, got {tuple(out.shape)}")
    pg, ld = _rows(g, "g")
    pq, pe = _kept(x8, "x8", (*g.shape[:-1], k))
    aligned = not ((pg | pq) & 15 or (ld or m) & 7)
    ws, size, mine = _workspace(_wgrad_ws(tokens, m, k, io, aligned, g.device), g.device, ws)
    rc = (_L or lib()).ssm_ckpt8_wgrad(
        pg, ld, pq, pe, _f32(o, "out", m * k), tokens, m, k, io,
        SSM_WGRAD_ACCUMULATE if accumulate else 0, ws.data_ptr(), size,
        _on(stream, g, o if out is None else None, mine))
    if rc:
        _check("ssm_ckpt8_wgrad", rc)
    return o
