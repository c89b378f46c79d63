"""Plain 64-bit forms of the norms around the scan, of 8-bit checkpoints and of the weight
gradient, on CPU tensors, straight from the formulas of include/ssm_block.h."""
import torch

f64 = torch.float64


def quantise(v):
    """(q int8, e uint8) of the values of ``v`` [rows][cols], one block of 32 columns at a time."""
    v = v.to(f64)
    rows, cols = v.shape
    q = torch.zeros(rows, cols, dtype=torch.int8)
    e = torch.zeros(rows, -(-cols // 32), dtype=torch.uint8)
    for j in range(e.shape[1]):
        part = v[:, 32 * j:32 * j + 32]
        for r in range(rows):
            b = part[r]
            if not bool(torch.isfinite(b).all()):
                e[r, j] = 255
                continue
            top = float(b.abs().max())
            E = -120 if top == 0.0 else max(-120, int(torch.frexp(torch.tensor(top, dtype=f64))[1]) - 1)
            e[r, j] = E + 127
            q[r, 32 * j:32 * j + 32] = torch.round(b * 2.0 ** (6 - E)).clamp(-127, 127).to(torch.int8)
    return q, e


def kept(q, e):
    """The values a checkpoint stands for."""
    cols = q.shape[1]
    step = torch.pow(torch.tensor(2.0, dtype=f64), e.to(f64) - 133.0)
    step[e == 255] = float("nan")
    return q.to(f64) * step.repeat_interleave(32, dim=1)[:, :cols]


def through8(v):
    return kept(*quantise(v))


def add_norm(x, residual, scale, w, eps):
    """(out, s, rstd)"""
    s = x.to(f64) if scale is None else scale.to(f64) * x.to(f64)
    if residual is not None:
        s = s + residual.to(f64)
    rstd = 1.0 / torch.sqrt((s * s).mean(1) + eps)
    out = s * rstd[:, None]
    return (out if w is None else out * w.to(f64)), s, rstd


def add_norm_bwd(d_out, s, rstd, d_s, scale, w, x):
    """(d_res, d_x, d_w, d_scale); s and rstd as the backward gets them"""
    d, s, rstd = d_out.to(f64), s.to(f64), rstd.to(f64)[:, None]
    n = s * rstd
    wd = d if w is None else d * w.to(f64)
    r = rstd * (wd - n * (wd * n).mean(1, keepdim=True))
    if d_s is not None:
        r = r + d_s.to(f64)
    d_x = r if scale is None else r * scale.to(f64)
    d_scale = None if x is None else (r * x.to(f64)).sum(0)
    return r, d_x, (d * n).sum(0), d_scale


def _silu(z):
    return z * torch.sigmoid(z)


def _spread(v, G):
    return v.repeat_interleave(G, dim=1)


def gated_norm(y, z, w, group, eps, norm_first):
    """(out, rstd [rows][groups])"""
    y, z = y.to(f64), z.to(f64)
    C = y.shape[1]
    G = group or C
    v = y if norm_first else y * _silu(z)
    rstd = 1.0 / torch.sqrt((v * v).reshape(-1, C // G, G).mean(2) + eps)
    out = v * _spread(rstd, G)
    if w is not None:
        out = out * w.to(f64)
    return (out * _silu(z) if norm_first else out), rstd


def gated_norm_bwd(d_out, y, z, rstd, w, group, norm_first):
    """(d_y, d_z, d_w)"""
    d, y, z = d_out.to(f64), y.to(f64), z.to(f64)
    C = y.shape[1]
    G = group or C
    rstd = _spread(rstd.to(f64).reshape(y.shape[0], -1), G)
    wd = d if w is None else d * w.to(f64)
    gate = _silu(z)
    sg = torch.sigmoid(z)
    slope = sg * (1.0 + z * (1.0 - sg))

    def mean(v):
        return _spread(v.reshape(-1, C // G, G).mean(2), G)

    if norm_first:
        n = y * rstd
        dn = wd * gate
        return rstd * (dn - n * mean(dn * n)), wd * n * slope, (d * gate * n).sum(0)
    n = y * gate * rstd
    dv = rstd * (wd - n * mean(wd * n))
    return dv * gate, dv * y * slope, (d * n).sum(0)
