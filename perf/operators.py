"""Cases that measure the operators around the scan in a Mamba block: the norms before and after
it (with the residual stream, its scale and the gate) and 8-bit activation checkpoints with the
weight gradient that reads them.

Formulas (rows are tokens, columns channels; every sum in at least 32 bits):

  add_norm    s = residual + scale * x;  out = w * s * rstd,  rstd = (mean(s^2) + eps)^-1/2
              backward, given d_out and d_s (the gradient that reaches s past the norm):
              n = s * rstd,  r = d_s + rstd * (w d_out - n mean(w d_out n)),
              d_residual = r,  d_x = scale * r,  d_scale = sum_rows r x,  d_w = sum_rows d_out n
  gated_norm  per group of columns, gate first:  v = y silu(z),  out = w * v * rstd(v)
              norm first:  out = w * y * rstd(y) * silu(z)
              backward to y, z and w
  ckpt8       blocks of 32 columns of a row: E = floor(log2(max |v|)), at least -120,
              q = round(v 2^(6-E)) to even, within -127 .. 127; the value kept is q 2^(E-6).
              Stored as int8 q and a byte E + 127 per block (255: a value was not finite, and
              the whole block reads as NaN)
  wgrad       d_W[m][k] = sum_t g[t][m] X[t][k], X read from its 8-bit checkpoint

A training pass with ``save8`` keeps s (or y and z) in 8 bits between forward and backward; the
backward's s is then what the checkpoint holds, with the forward's rstd.
"""
import math

import torch

own = False

EPS = 1e-5
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of one request: the residual add and norm in front of a layer
        dict(name="add_norm_token_bf16", op="add_norm", io="bf16", res="f32", rows=1, cols=768,
             scaled=False, train=False, save8=False),
        # a small fp32 layer (8 x 1024 tokens), trained with the stream kept whole
        dict(name="add_norm_train_f32", op="add_norm", io="f32", res="f32", rows=8192, cols=512,
             scaled=False, train=True, save8=False),
        # the training-shaped layer (16 x 2048 tokens): scaled residual, stream saved in 8 bits
        dict(name="add_norm_train8_bf16", op="add_norm", io="bf16", res="f32", rows=32768,
             cols=768, scaled=True, train=True, save8=True),
        # a ragged batch of an odd width, the stream itself in bf16
        dict(name="add_norm_odd_bf16", op="add_norm", io="bf16", res="bf16", rows=2047, cols=1003,
             scaled=True, train=True, save8=True),
        # one token of each of 16 requests after the scan
        dict(name="gated_norm_tokens_bf16", op="gated_norm", io="bf16", rows=16, cols=1536,
             group=0, norm_first=False, strided=True, train=False, save8=False),
        # the same fp32 layer after its scan: norm of each group of 64 channels before the gate
        dict(name="gated_norm_train_f32", op="gated_norm", io="f32", rows=8192, cols=512,
             group=64, norm_first=True, strided=False, train=True, save8=False),
        # the training-shaped layer after its scan, z a slice of the projection, 8-bit y and z
        dict(name="gated_norm_train8_bf16", op="gated_norm", io="bf16", rows=32768, cols=1536,
             group=0, norm_first=False, strided=True, train=True, save8=True),
        # an activation of the long sequence (16384 tokens) kept and read back
        dict(name="ckpt8_long_bf16", op="ckpt8", io="bf16", rows=16384, cols=2048),
        # a ragged fp32 activation, the last block of a row cut short
        dict(name="ckpt8_odd_f32", op="ckpt8", io="f32", rows=3001, cols=517),
        # a small projection of a ragged fp32 batch (dt, B and C from 512 channels)
        dict(name="wgrad_narrow_f32", op="wgrad", io="f32", tokens=8189, m=64, k=512),
        # the projection out of the training-shaped layer
        dict(name="wgrad_out_bf16", op="wgrad", io="bf16", tokens=32768, m=768, k=1536),
        # the projection into the long-sequence layer
        dict(name="wgrad_in_bf16", op="wgrad", io="bf16", tokens=16384, m=4096, k=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 8, as models have them, else whatever comes."""
    n = _log_int(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["add_norm", "gated_norm", "ckpt8", "wgrad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "wgrad":
        m, k = _width(rng, 16, 4096), _width(rng, 16, 2048)
        most = min(32768, 2 ** 36 // (m * k)) if io == "bf16" else min(16384, 2 ** 34 // (m * k))
        return dict(op=op, io=io, tokens=_log_int(rng, min(64, most), most), m=m, k=k)
    train = rng.random() < 0.7
    if op == "gated_norm" and rng.random() < 0.5:
        group = rng.choice([32, 64, 96, 128, 256])
        cols = group * rng.randint(1, 2048 // group)
    else:
        group, cols = 0, _width(rng, 16, 4096)
    rows = _log_int(rng, 1, min(32768, 2 ** 25 // cols))
    if op == "ckpt8":
        return dict(op=op, io=io, rows=rows, cols=cols)
    save8 = train and io == "bf16" and rng.random() < 0.6
    if op == "add_norm":
        return dict(op=op, io=io, res=rng.choice(["f32", "bf16"]) if io == "bf16" else "f32",
                    rows=rows, cols=cols, scaled=rng.random() < 0.5, train=train, save8=save8)
    return dict(op=op, io=io, rows=rows, cols=cols, group=group, norm_first=rng.random() < 0.5,
                strided=rng.random() < 0.5, train=train, save8=save8)


# ---- inputs ---------------------------------------------------------------------------------

class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda") * std

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def activation(self, rows, cols, std=1.0):
        """Normal values with a few loud channels, as residual streams have them."""
        loud = torch.exp(1.5 * self.normal(cols).clamp(min=1.0) - 1.5)
        return self.normal(rows, cols, std=std) * loud


def prepare(case, seed):
    c, d = case, _Draw(seed)
    io = IO[c["io"]]
    if c["op"] == "wgrad":
        q, e = _quantise(d.activation(c["tokens"], c["k"]))
        return dict(case=c, g=d.normal(c["tokens"], c["m"]).to(io), q=q, e=e)
    R, C = c["rows"], c["cols"]
    s = dict(case=c)
    if c["op"] == "ckpt8":
        s["x"] = d.activation(R, C).to(io)
        return s
    s["w"] = 1.0 + d.normal(C, std=0.1)
    if c["op"] == "add_norm":
        s["x"] = d.normal(R, C, std=0.5).to(io)
        s["residual"] = d.activation(R, C).to(IO[c["res"]])
        s["scale"] = d.uniform(0.1, 1.0, C) if c["scaled"] else None
        if c["train"]:
            s["d_out"] = d.normal(R, C).to(io)
            s["d_s"] = d.normal(R, C).to(IO[c["res"]])
        else:  # the buffers that a decode loop writes to
            s["into"] = (torch.empty_like(s["x"]), torch.empty_like(s["residual"]))
        return s
    s["y"] = d.activation(R, C, std=0.5).to(io)
    z = d.normal(R, 2 * C if c["strided"] else C).to(io)
    s["z"] = z[:, C:] if c["strided"] else z  # the gate's half of an input projection
    if c["train"]:
        s["d_out"] = d.normal(R, C).to(io)
    else:
        s["into"] = torch.empty_like(s["y"])
    return s


# ---- the plain forms ------------------------------------------------------------------------

def _blocks(v):
    rows, cols = v.shape
    pad = -cols % 32
    if pad:
        v = torch.cat([v, v.new_zeros(rows, pad)], dim=1)
    return v.view(rows, -1, 32)


def _quantise(v):
    """(q int8 [rows][cols], e uint8 [rows][ceil(cols/32)]) of fp32 values."""
    rows, cols = v.shape
    b = _blocks(v)
    top = b.abs().amax(dim=2)
    fine = torch.isfinite(top)
    E = (torch.frexp(top)[1] - 1).clamp(min=-120)
    E = torch.where(top == 0, torch.full_like(E, -120), E)
    up = ((6 - E + 127) << 23).view(torch.float32)  # 2^(6-E)
    q = torch.round(b * up[:, :, None]).clamp(-127, 127)
    q = torch.where(fine[:, :, None], q, torch.zeros_like(q)).to(torch.int8)
    e = torch.where(fine, E + 127, torch.full_like(E, 255)).to(torch.uint8)
    return q.view(rows, -1)[:, :cols].contiguous(), e


def _values(q, e):
    """What a checkpoint stands for, in fp32."""
    rows, cols = q.shape
    E = e.to(torch.int32)
    step = torch.where(E == 255, torch.full_like(E, 0x7fc00000), (E - 6) << 23)
    return (_blocks(q.float()) * step.view(torch.float32)[:, :, None]).view(rows, -1)[:, :cols]


def _add_norm(s):
    c, f = s["case"], torch.float32
    io, res = IO[c["io"]], IO[c["res"]]
    x, w, scale = s["x"].to(f), s["w"], s["scale"]
    stream = s["residual"].to(f) + (x if scale is None else scale * x)
    rstd = 1.0 / torch.sqrt(stream.square().mean(dim=1, keepdim=True) + EPS)
    got = dict(out=(w * (stream * rstd)).to(io), stream=stream.to(res))
    if not c["train"]:
        return got
    kept = got["stream"].to(f)
    if c["save8"]:
        kept = _values(*_quantise(kept))
    n = kept * rstd
    wd = w * s["d_out"].to(f)
    r = s["d_s"].to(f) + rstd * (wd - n * (wd * n).mean(dim=1, keepdim=True))
    got.update(d_residual=r.to(res), d_x=(r if scale is None else scale * r).to(io),
               d_w=(s["d_out"].to(f) * n).sum(dim=0))
    if scale is not None:
        got["d_scale"] = (r * x).sum(dim=0)
    return got


def _gated_norm(s):
    c, f = s["case"], torch.float32
    io = IO[c["io"]]
    R, C = c["rows"], c["cols"]
    G = c["group"] or C
    y, z, w = s["y"].to(f).view(R, -1, G), s["z"].to(f).reshape(R, -1, G), s["w"].view(-1, G)
    gate = z / (1.0 + torch.exp(-z))
    v = y if c["norm_first"] else y * gate
    rstd = 1.0 / torch.sqrt(v.square().mean(dim=2, keepdim=True) + EPS)
    n = v * rstd
    got = dict(out=(w * n * gate if c["norm_first"] else w * n).view(R, C).to(io))
    if not c["train"]:
        return got
    if c["save8"]:
        y = _values(*_quantise(s["y"].to(f))).reshape(R, -1, G)
        z = _values(*_quantise(s["z"].to(f))).reshape(R, -1, G)
        gate = z / (1.0 + torch.exp(-z))
        n = (y if c["norm_first"] else y * gate) * rstd
    sig = 1.0 / (1.0 + torch.exp(-z))
    slope = sig * (1.0 + z * (1.0 - sig))  # d silu(z) / d z
    d = s["d_out"].to(f).view(R, -1, G)
    dn = d * w * gate if c["norm_first"] else d * w
    dv = rstd * (dn - n * (dn * n).mean(dim=2, keepdim=True))
    if c["norm_first"]:
        d_y, d_z, d_w = dv, d * w * n * slope, d * n * gate
    else:
        d_y, d_z, d_w = dv * gate, dv * y * slope, d * n
    got.update(d_y=d_y.view(R, C).to(io), d_z=d_z.view(R, C).to(io), d_w=d_w.sum(dim=0).view(C))
    return got


def _plain(s):
    c = s["case"]
    if c["op"] == "add_norm":
        return _add_norm(s)
    if c["op"] == "gated_norm":
        return _gated_norm(s)
    if c["op"] == "ckpt8":
        return dict(values=_values(*_quantise(s["x"].float())).to(s["x"].dtype))
    return dict(d_W=s["g"].float().t() @ _values(s["q"], s["e"]))


# ---- the framework's calls ------------------------------------------------------------------

def _own(s):
    import bwd_ssm_conv_gb300 as ssm
    c = s["case"]
    if c["op"] == "wgrad":
        return dict(d_W=ssm.ssm_ckpt8_wgrad(s["g"], ssm.Ckpt8(s["q"], s["e"])))
    if c["op"] == "ckpt8":
        return dict(values=ssm.ssm_ckpt8_load(ssm.ssm_ckpt8_save(s["x"]), s["x"].dtype))
    if c["op"] == "add_norm":
        if not c["train"]:
            a = ssm.ssm_add_norm_fwd(s["x"], s["w"], s["residual"], s["scale"], eps=EPS,
                                     want_rstd=False, out=s["into"])
            return dict(out=a.out, stream=a.res_out)
        a = ssm.ssm_add_norm_fwd(s["x"], s["w"], s["residual"], s["scale"], eps=EPS,
                                 save8=c["save8"])
        g = ssm.ssm_add_norm_bwd(s["d_out"], a.res8 if c["save8"] else a.res_out, a.rstd, s["w"],
                                 d_res_out=s["d_s"], scale=s["scale"],
                                 x=s["x"] if c["scaled"] else None)
        got = dict(out=a.out, stream=a.res_out, d_residual=g["d_res"], d_x=g["d_x"],
                   d_w=g["d_w"])
        if c["scaled"]:
            got["d_scale"] = g["d_scale"]
        return got
    how = dict(group=c["group"], norm_first=c["norm_first"])
    if not c["train"]:
        a = ssm.ssm_gated_norm_fwd(s["y"], s["z"], s["w"], eps=EPS, want_rstd=False,
                                   out=s["into"], **how)
        return dict(out=a.out)
    a = ssm.ssm_gated_norm_fwd(s["y"], s["z"], s["w"], eps=EPS, save8=c["save8"], **how)
    g = ssm.ssm_gated_norm_bwd(s["d_out"], a.y8 if c["save8"] else s["y"],
                               a.z8 if c["save8"] else s["z"], a.rstd, s["w"], **how)
    return dict(out=a.out, d_y=g["d_y"], d_z=g["d_z"], d_w=g["d_w"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    c = case
    b = 2 if c["io"] == "bf16" else 4
    if c["op"] == "wgrad":
        t, m, k = c["tokens"], c["m"], c["k"]
        return {"bytes": t * m * b + t * k + t * -(-k // 32) + 4 * m * k, "flops": 2.0 * t * m * k}
    n = c["rows"] * c["cols"]
    if c["op"] == "ckpt8":  # the checkpoint itself is written and read between the two
        kept = n + c["rows"] * -(-c["cols"] // 32)
        return {"bytes": 2 * n * b + 2 * kept, "flops": 4.0 * n}
    if c["op"] == "add_norm":
        r = 2 if c["res"] == "bf16" else 4
        fwd = n * (2 * b + 2 * r)
        bwd = n * (2 * b + 2 * r) if c["train"] else 0
        return {"bytes": fwd + bwd, "flops": n * (6.0 + (14.0 if c["train"] else 0.0))}
    return {"bytes": n * 3 * b + (n * 3 * b if c["train"] else 0),
            "flops": n * (10.0 + (30.0 if c["train"] else 0.0))}


# ---- the same in 64 bits ----------------------------------------------------------------------

def _exact_kept(v):
    """The values an 8-bit checkpoint of the 64-bit values ``v`` holds, column by column."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    for k in range(0, cols, 32):
        part = v[:, k:k + 32]
        top = part.abs().max(dim=1, keepdim=True).values
        power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        power = torch.where(torch.exp2(power) > top, power - 1, power)   # log2 may round
        power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)
        power = torch.where(top > 0, power, torch.full_like(power, -120.0)).clamp(min=-120.0)
        step = torch.exp2(power - 6)
        out[:, k:k + 32] = torch.round(part / step).clamp(-127, 127) * step
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = torch.float64
    if c["op"] == "wgrad":
        t, k = c["tokens"], c["k"]
        block = torch.arange(k, device="cuda") // 32
        X = s["q"].to(f) * torch.exp2(s["e"].to(f) - 133.0)[:, block]
        d_W = torch.zeros(c["m"], k, dtype=f, device="cuda")
        for t0 in range(0, t, 4096):
            d_W += torch.einsum("tm,tk->mk", s["g"][t0:t0 + 4096].to(f), X[t0:t0 + 4096])
        return dict(d_W=d_W)
    if c["op"] == "ckpt8":
        return dict(values=_exact_kept(s["x"].to(f)))
    w = s["w"].to(f)
    if c["op"] == "add_norm":
        x = s["x"].to(f)
        scale = torch.ones_like(w) if s["scale"] is None else s["scale"].to(f)
        stream = s["residual"].to(f) + scale * x
        rstd = torch.pow(torch.sum(stream * stream, 1) / c["cols"] + EPS, -0.5)[:, None]
        got = dict(out=stream * rstd * w, stream=stream)
        if c["train"]:
            kept = stream.to(IO[c["res"]]).to(f)  # what the stream's own type holds of it
            kept = _exact_kept(kept) if c["save8"] else kept
            dn = s["d_out"].to(f) * w
            n = kept * rstd
            r = s["d_s"].to(f) + rstd * dn - rstd * n * (torch.sum(dn * n, 1) / c["cols"])[:, None]
            got.update(d_residual=r, d_x=r * scale, d_w=torch.einsum("rc,rc->c", s["d_out"].to(f), n),
                       d_scale=torch.einsum("rc,rc->c", r, x) if c["scaled"] else None)
        return got
    y, z = s["y"].to(f), s["z"].to(f)
    C, G = c["cols"], c["group"] or c["cols"]

    def mean(v):  # of each group, at every column of it
        return torch.repeat_interleave(torch.sum(v.reshape(-1, C // G, G), 2) / G, G, dim=1)

    def halves(y, z):
        return y, z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)

    y, gate, _ = halves(y, z)
    v = y if c["norm_first"] else y * gate
    rstd = torch.pow(mean(v * v) + EPS, -0.5)
    got = dict(out=v * rstd * w * (gate if c["norm_first"] else 1.0))
    if c["train"]:
        if c["save8"]:
            y, z = _exact_kept(y), _exact_kept(s["z"].to(f))
        y, gate, slope = halves(y, z)
        d = s["d_out"].to(f)
        if c["norm_first"]:
            n = y * rstd
            up = d * w * gate
            got.update(d_y=rstd * (up - n * mean(up * n)), d_z=d * w * n * slope,
                       d_w=torch.sum(d * n * gate, 0))
        else:
            n = y * gate * rstd
            up = rstd * (d * w - n * mean(d * w * n))
            got.update(d_y=up * gate, d_z=up * y * slope, d_w=torch.sum(d * n, 0))
    return got
