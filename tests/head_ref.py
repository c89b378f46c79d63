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


# ---- the head -----------------------------------------------------------------------------------------

def _product(io, a, b, n):
    """The error of a sum of n products a b with magnitudes a_abs b_abs: bf16 terms have exact products and
    the tensor cores truncate each of the n / 16 additions, and the 16 products in it, at 2^-23 of the
    largest magnitude so far (two units: the terms' alignment and the sum's); fp32 terms add six such
    products per 16, taken out every 128 and added in fp32, and leave out 2^-22 of each product."""
    size = a.abs() @ b.abs()
    steps = n / 16 + 4
    if io == torch.float32:
        return size * (2.0 ** -22 * (1 + 48 + 4) + U * (n / 128 + 1))
    return size * 2.0 ** -22 * steps


def _p_of(t_idx, t_logit, tau, vocab):
    """(p [rows][vocab], rows with a loss, sum p log p)"""
    there = (t_idx >= 0) & (t_logit > -float("inf"))
    t = torch.where(there, t_logit.to(f64) / tau, torch.tensor(-float("inf"), dtype=f64))
    some = there.any(1)
    p = torch.zeros_like(t)
    p[some] = torch.softmax(t[some], 1)
    logs = torch.where(p > 0, p * torch.log(p.clamp(min=1e-300)), torch.zeros_like(p)).sum(1)
    P = torch.zeros(t.shape[0], vocab, dtype=f64)
    P.scatter_add_(1, t_idx.clamp(min=0), torch.where(there, p, torch.zeros_like(p)))
    return P, some, logs


def head(h, w, P, some, logs, tau=1.0):
    """(loss, lse) and their bounds; the rows that are not in ``some`` are 0 whatever h holds."""
    io, V = h.dtype, w.shape[0]
    hh = torch.where(some[:, None], h.to(f64), torch.zeros(1, dtype=f64))
    ww = w.to(f64)
    z = hh @ ww.t() / tau
    lse = torch.logsumexp(z, 1)
    loss = tau * tau * (logs + lse * P.sum(1) - (P * z).sum(1))
    dz = _product(io, hh, ww.t(), h.shape[1]) / tau + 2 * U * z.abs()
    # 2^x is good to 2^-22 and its argument to one rounding; the sum's additions; its logarithm
    dlse = dz.amax(1) + 2.0 ** -21 + (SUM + V // 4096) * U + 4 * U * (lse.abs() + z.abs().amax(1))
    mean = P * (z.amax(1, keepdim=True) - z).abs()
    dloss = tau * tau * (dlse + (P * dz).sum(1) + 80 * U * (mean.sum(1) + logs.abs() + lse.abs()))
    zero = torch.zeros_like(lse)
    return ((torch.where(some, loss, zero), torch.where(some, lse, zero)),
            (torch.where(some, dloss, zero), torch.where(some, dlse, zero)))


def head_bwd(h, w, P, some, lse, d_loss, tau=1.0):
    """(d_h, d_w) and their bounds; lse as the backward gets it."""
    io = h.dtype
    hh = torch.where(some[:, None], h.to(f64), torch.zeros(1, dtype=f64))
    ww = w.to(f64)
    z = hh @ ww.t() / tau
    lse = lse.to(f64)[:, None]
    q = torch.exp(z - lse)
    up = torch.where(some, d_loss.to(f64), torch.zeros(1, dtype=f64))[:, None] * tau
    G = (q - P) * up
    # of q: its argument (an error e of it is a factor exp(e) <= 1 + 2 e here), 2^x
    de = _product(io, hh, ww.t(), h.shape[1]) / tau + 4 * U * (z.abs() + lse.abs())
    dG = (q * (2 * de + 2.0 ** -21) + 2.0 ** -21 * P + 8 * U * (q + P)) * up.abs()
    # between the products: bf16, or three terms of it; d_loss over the largest and back
    dG = dG + G.abs() * ((2.0 ** -8 if io == torch.bfloat16 else 2.0 ** -22) + 6 * U)
    # 2^x below the smallest normal number 2^-126 is 0, and a G (over the largest |d_loss| tau) as small
    # is a subnormal number, whose digits end at a fixed place: off by 2^-126 at most in either case
    dG = dG + 2.0 ** -126 * (up.abs() + up.abs().max())
    T, V = G.shape
    d_h, d_w = G @ ww, G.t() @ hh
    dd_h = dG @ ww.abs() + _product(io, G.abs() + dG, ww, V) + 16 * U * (G.abs() @ ww.abs())
    dd_w = dG.t() @ hh.abs() + _product(io, (G.abs() + dG).t(), hh, T) + 16 * U * (G.abs().t() @ hh.abs())
    return (d_h, d_w), (dd_h, dd_w)


def ce_rows(target, vocab, ignore=-100):
    """(P, some, logs) of class targets."""
    some = target != ignore
    P = torch.zeros(target.numel(), vocab, dtype=f64)
    P[some, target[some]] = 1.0
    return P, some, torch.zeros(target.numel(), dtype=f64)
