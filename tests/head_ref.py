"""Plain 64-bit forms of the layer norm and of the head with its losses, on CPU tensors, straight from
the formulas of include/ssm_block.h and include/ssm_head.h, and the error bounds of the tests.

A value's bound counts roundings: half a step of its type (finfo.eps / 2, relative) where it is stored,
and 2^-24 relative for each fp32 operation, carried through the formula with the sum of the magnitudes
of its terms.  A sum of n terms in the kernels' order (a few per thread, then a tree) is off by at
most SUM 2^-24 of the sum of its terms' magnitudes."""
import torch

f64 = torch.float64
U = 2.0 ** -24
SUM = 50  # additions that one term goes through: at most 32 in a thread, 5 in a warp, 32 over warps / 4


def within(name, got, want, bound):
    """Every element of ``got`` is within ``bound`` (64 bits) of ``want``, beside its type's rounding."""
    g, want = got.detach().cpu().to(f64), want.to(f64)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    assert bool(torch.isfinite(g).all()), f"{name}: non-finite values"
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else U
    limit = bound + half * (want.abs() + bound) + 1e-37
    off = (g - want).abs()
    worst = (off / limit).max() if off.numel() else torch.tensor(0.0)
    assert float(worst) <= 1.0, f"{name}: {float(worst):.2f} times its bound, " \
        f"off by {float(off.max()):.3e}"


def _sums(rows):
    """Additions that a term of a sum over rows goes through: a block's rows (one of at least 152
    blocks, of up to 32 rows at a time), then the blocks' sums, 128 slices of them and a tree."""
    return rows // 152 + 32 + 16 + 16


def layer_norm(x, residual, scale, w, b, eps):
    """(out, s, mean, rstd) and the bounds of out, mean and rstd, s in fp32 being exact."""
    x = x.to(f64)
    branch = x if scale is None else scale.to(f64) * x
    s = branch if residual is None else branch + residual.to(f64)
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    n = (s - mean) * rstd
    W = torch.ones_like(s[0]) if w is None else w.to(f64)
    out = n * W if b is None else n * W + b.to(f64)
    # s itself rounds twice; the mean's error; then the squares', which the errors of s - mean enter
    ds = U * (2 * branch.abs() + 2 * s.abs())
    dmean = SUM * U * s.abs().mean(1, keepdim=True) + ds.mean(1, keepdim=True)
    doff = ds + dmean + U * (s - mean).abs()
    dvar = (2 * (s - mean).abs() * doff).mean(1, keepdim=True) + (doff ** 2).mean(1, keepdim=True) \
        + SUM * U * var
    drstd = rstd * (0.5 * dvar / (var + eps) + 4 * U) + rstd * (dvar / (var + eps)) ** 2
    dn = doff * rstd + (s - mean).abs() * drstd + U * n.abs()
    dout = W.abs() * dn + 2 * U * (n * W).abs() + U * out.abs()
    return (out, s, mean[:, 0], rstd[:, 0]), (dout, ds, dmean[:, 0], drstd[:, 0])


def layer_norm_bwd(d_out, s, mean, rstd, d_s, scale, w, x):
    """(d_res, d_x, d_w, d_b, d_scale) and their bounds; s, mean and rstd as the backward gets them."""
    rows = d_out.shape[0]
    d, s = d_out.to(f64), s.to(f64)
    mean, rstd = mean.to(f64)[:, None], rstd.to(f64)[:, None]
    n = (s - mean) * rstd
    dn = 2 * U * n.abs()
    W = torch.ones_like(s[0]) if w is None else w.to(f64)
    a = d * W
    ma, mn = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    up = torch.zeros_like(a) if d_s is None else d_s.to(f64)
    r = up + rstd * (a - ma - n * mn)
    dma = (SUM + 2) * U * a.abs().mean(1, keepdim=True)
    dmn = (SUM + 5) * U * (a * n).abs().mean(1, keepdim=True)
    dr = rstd * (3 * U * a.abs() + 2 * U * ma.abs() + dma + n.abs() * dmn + mn.abs() * (dn + 4 * U * n.abs())) \
        + 2 * U * (up.abs() + r.abs())
    sc = torch.ones_like(W) if scale is None else scale.to(f64)
    d_x, dd_x = r * sc, dr * sc.abs() + U * (r * sc).abs()
    A = _sums(rows) * U
    d_w, dd_w = (d * n).sum(0), A * (d * n).abs().sum(0) + (d.abs() * (dn + U * n.abs())).sum(0)
    d_b, dd_b = d.sum(0), A * d.abs().sum(0)
    out, bound = [r, d_x, d_w, d_b], [dr, dd_x, dd_w, dd_b]
    if x is not None:
        x = x.to(f64)
        out.append((r * x).sum(0))
        bound.append(A * (r * x).abs().sum(0) + (dr * x.abs()).sum(0))
    return out, bound
