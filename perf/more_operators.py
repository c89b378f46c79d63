"""Cases that measure the operators at a model's end: the layer norm in front of the head (with the
residual stream and its scale), and the head with its loss, cross entropy over the vocabulary or
distillation from a teacher's top logits, each with its gradients.

Formulas (rows are tokens; every sum in at least 32 bits):

  layer_norm  s = residual + scale * x;  mu = mean(s),  rstd = (mean((s - mu)^2) + eps)^-1/2,
              out = w * (s - mu) * rstd + b
              backward, given d_out and d_s (the gradient that reaches s past the norm):
              n = (s - mu) rstd,  a = w d_out,  r = d_s + rstd * (a - mean(a) - n mean(a n)),
              d_residual = r,  d_x = scale * r,  d_scale = sum_rows r x,
              d_w = sum_rows d_out n,  d_b = sum_rows d_out
  ce          z = h W^T over the vocabulary,  lse = log sum_v exp(z_v),  loss = lse - z_target
              a row whose target is IGNORE has loss, lse and gradients of 0
              backward, given d_loss of each row:
              G = (softmax(z) - onehot(target)) d_loss,  d_h = G W,  d_w = G^T h
  distill     a teacher's top k logits t at the vocabulary's indices i (an index below 0: no entry):
              p = softmax(t / tau) over a row's entries,  q = softmax(z / tau),  lse of z / tau,
              loss = tau^2 sum_j p_j (log p_j - log q_{i_j}),  0 where a row has no entry
              backward: G = tau (q - p) d_loss,  d_h = G W,  d_w = G^T h
"""
import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of one request: the norm in front of the head
        dict(name="layer_norm_token_bf16", op="layer_norm", io="bf16", res="f32", rows=1, cols=768,
             scaled=False, train=False),
        # a ragged fp32 batch of an odd width
        dict(name="layer_norm_odd_f32", op="layer_norm", io="f32", res="f32", rows=2047, cols=1003,
             scaled=True, train=True),
        # the long sequence (16384 tokens), the stream itself in bf16
        dict(name="layer_norm_long_bf16", op="layer_norm", io="bf16", res="bf16", rows=16384,
             cols=1024, scaled=False, train=True),
        # the training-shaped layer (16 x 2048 tokens) with an fp32 stream and a scaled branch
        dict(name="layer_norm_train_bf16", op="layer_norm", io="bf16", res="f32", rows=32768,
             cols=768, scaled=True, train=True),
        # the log-probability of one token as it comes (scoring, a compressor's model)
        dict(name="ce_token_bf16", op="ce", io="bf16", rows=1, cols=768, vocab=32768, train=False,
             ignored=0.0),
        # a byte-level fp32 model (8 x 1024 tokens, 512 channels)
        dict(name="ce_bytes_f32", op="ce", io="f32", rows=8192, cols=512, vocab=256, train=True,
             ignored=0.0),
        # odd sizes throughout, a third of the tokens being prompts that carry no loss
        dict(name="ce_odd_f32", op="ce", io="f32", rows=1021, cols=515, vocab=10007, train=True,
             ignored=0.33),
        # 8 x 1024 tokens of a small model with a large vocabulary, some padding
        dict(name="ce_train_bf16", op="ce", io="bf16", rows=8192, cols=768, vocab=50000, train=True,
             ignored=0.1),
        # one long sequence
        dict(name="ce_long_bf16", op="ce", io="bf16", rows=16384, cols=1024, vocab=32768,
             train=True, ignored=0.0),
        # a small fp32 student of odd sizes
        dict(name="distill_small_f32", op="distill", io="f32", rows=333, cols=256, vocab=5003, k=17,
             tau=1.0, train=True, ignored=0.1),
        # a batch of 4 x 1024 tokens, many teacher logits at a high temperature
        dict(name="distill_train_bf16", op="distill", io="bf16", rows=4096, cols=768, vocab=32768,
             k=64, tau=2.0, train=True, ignored=0.05),
        # the largest student and vocabulary
        dict(name="distill_large_bf16", op="distill", io="bf16", rows=8192, cols=1024, vocab=65536,
             k=32, tau=1.0, train=True, ignored=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 8, as models have them, else whatever comes."""
    n = _log_int(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["layer_norm", "ce", "ce", "distill", "distill"])
    io = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.8
    if op == "layer_norm":
        cols = _width(rng, 16, 4096)
        return dict(op=op, io=io, res=rng.choice(["f32", "bf16"]) if io == "bf16" else "f32",
                    rows=_log_int(rng, 1, min(32768, 2 ** 25 // cols)), cols=cols,
                    scaled=rng.random() < 0.5, train=train)
    cols, vocab = _width(rng, 64, 2048), _width(rng, 200, 65536)
    most = 2 ** 38 if io == "bf16" else 2 ** 35
    rows = _log_int(rng, 1, min(16384, most // (cols * vocab)))
    c = dict(op=op, io=io, rows=rows, cols=cols, vocab=vocab, train=train,
             ignored=rng.choice([0.0, 0.1, 0.5]))
    if op == "distill":
        c.update(k=rng.randint(1, min(100, vocab // 2)), tau=rng.choice([1.0, 1.5, 4.0]))
    return c


# ---- inputs ---------------------------------------------------------------------------------

class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda") * std

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def below(self, n, *shape):
        return torch.randint(n, shape, generator=self.g, device="cuda")

    def activation(self, rows, cols, std=1.0):
        """Normal values with a few loud channels, as residual streams have them."""
        loud = torch.exp(1.5 * self.normal(cols).clamp(min=1.0) - 1.5)
        return self.normal(rows, cols, std=std) * loud


def prepare(case, seed):
    c, d = case, _Draw(seed)
    io = IO[c["io"]]
    R, C = c["rows"], c["cols"]
    s = dict(case=c)
    if c["op"] == "layer_norm":
        s["w"], s["b"] = 1.0 + d.normal(C, std=0.1), d.normal(C, std=0.1)
        s["x"] = d.normal(R, C, std=0.5).to(io)
        # a stream whose rows have a mean of their own, which the norm takes off
        s["residual"] = (d.activation(R, C) + d.normal(R, 1)).to(IO[c["res"]])
        s["scale"] = d.uniform(0.1, 1.0, C) if c["scaled"] else None
        if c["train"]:
            s["d_out"] = d.normal(R, C).to(io)
            s["d_s"] = d.normal(R, C).to(IO[c["res"]])
        else:  # the buffers that a decode loop writes to
            s["into"] = (torch.empty_like(s["x"]), torch.empty_like(s["residual"]))
        return s
    V = c["vocab"]
    w = d.normal(V, C, std=C ** -0.5)
    if c["op"] == "ce":
        # a few words are frequent, most are rare; the ignored rows lie anywhere
        y = (V * d.uniform(0.0, 1.0, R) ** 3).long().clamp(max=V - 1)
        likely = y
        s["target"] = torch.where(d.uniform(0.0, 1.0, R) < c["ignored"], torch.full_like(y, IGNORE), y)
        valid = s["target"] != IGNORE
    else:
        k = c["k"]
        steps = d.below(V // k, R, k) + 1  # increasing, so that a row's indices differ
        order = torch.argsort(d.uniform(0.0, 1.0, R, k), dim=1)
        idx = torch.gather(torch.cumsum(steps, dim=1) - 1, 1, order)
        likely = idx[:, 0].clone()
        s["t_logit"] = torch.sort(d.normal(R, k, std=3.0), dim=1, descending=True).values
        # some rows have fewer entries, some none (padding)
        kept = d.below(k, R) + 1 + k * (d.uniform(0.0, 1.0, R) < 0.8).long()
        valid = d.uniform(0.0, 1.0, R) >= c["ignored"]
        kept = torch.where(valid, kept, torch.zeros_like(kept))
        s["t_idx"] = torch.where(torch.arange(k, device="cuda")[None] < kept[:, None], idx,
                                 torch.full_like(idx, -1))
    # hidden states that know something of the answer: from nothing to all but certain
    s["h"] = (d.normal(R, C) + d.uniform(0.0, 16.0, R, 1) * w[likely]).to(io)
    s["w"] = w.to(io)
    if c["train"]:  # of the mean over the rows that count
        s["d_loss"] = torch.full((R,), 1.0, device="cuda") / valid.sum().clamp(min=1)
    return s


# ---- the plain forms ------------------------------------------------------------------------

def _layer_norm(s):
    c, f = s["case"], torch.float32
    io, res = IO[c["io"]], IO[c["res"]]
    x, w, scale = s["x"].to(f), s["w"], s["scale"]
    stream = s["residual"].to(f) + (x if scale is None else scale * x)
    mean = stream.mean(dim=1, keepdim=True)
    rstd = 1.0 / torch.sqrt((stream - mean).square().mean(dim=1, keepdim=True) + EPS)
    got = dict(out=(w * ((stream - mean) * rstd) + s["b"]).to(io), stream=stream.to(res))
    if not c["train"]:
        return got
    n = (got["stream"].to(f) - mean) * rstd
    d_out = s["d_out"].to(f)
    a = w * d_out
    r = s["d_s"].to(f) + rstd * (a - a.mean(dim=1, keepdim=True) -
                                 n * (a * n).mean(dim=1, keepdim=True))
    got.update(d_residual=r.to(res), d_x=(r if scale is None else scale * r).to(io),
               d_w=(d_out * n).sum(dim=0), d_b=d_out.sum(dim=0))
    if scale is not None:
        got["d_scale"] = (r * x).sum(dim=0)
    return got


def _head(s):
    c, f = s["case"], torch.float32
    h, w = s["h"].to(f), s["w"].to(f)
    rows = torch.arange(c["rows"], device="cuda")
    z = h @ w.t()
    if c["op"] == "ce":
        tau = 1.0
        idx = s["target"][:, None]
        valid = (idx != IGNORE).squeeze(1)
        p = valid.to(f)[:, None]
        known = torch.zeros_like(p)  # p log p
    else:
        tau = c["tau"]
        z = z / tau
        idx = s["t_idx"]
        there = idx >= 0
        valid = there.any(dim=1)
        t = torch.where(there, s["t_logit"] / tau, torch.full_like(s["t_logit"], -math.inf))
        t = t - torch.where(valid, t.amax(dim=1), torch.zeros_like(t[:, 0]))[:, None]
        p = torch.exp(t)
        total = torch.where(valid, p.sum(dim=1), torch.ones_like(t[:, 0]))[:, None]
        p = p / total
        known = torch.where(there, p * (t - torch.log(total)), torch.zeros_like(p))
    idx = idx.clamp(min=0)
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    loss = (p * (lse[:, None] - torch.gather(z, 1, idx)) + known).sum(dim=1) * tau ** 2
    zero = torch.zeros_like(lse)
    got = dict(loss=torch.where(valid, loss, zero), lse=torch.where(valid, lse, zero))
    if c["train"]:
        G = (e / total).index_put((rows[:, None], idx), -p, accumulate=True)
        G = G * (tau * torch.where(valid, s["d_loss"], zero))[:, None]
        got.update(d_h=(G @ w).to(s["h"].dtype), d_w=(G.t() @ h).to(s["w"].dtype))
    return got


# ---- the framework's calls ------------------------------------------------------------------

def _own(s):
    import bwd_ssm_conv_gb300 as ssm
    c = s["case"]
    if c["op"] == "layer_norm":
        if not c["train"]:
            a = ssm.ssm_add_layer_norm_fwd(s["x"], s["w"], s["b"], s["residual"], s["scale"],
                                           eps=EPS, want_stats=False, out=s["into"])
            return dict(out=a.out, stream=a.res_out)
        a = ssm.ssm_add_layer_norm_fwd(s["x"], s["w"], s["b"], s["residual"], s["scale"], eps=EPS)
        g = ssm.ssm_add_layer_norm_bwd(s["d_out"], a.res_out, a.mean, a.rstd, s["w"],
                                       d_res_out=s["d_s"], scale=s["scale"],
                                       x=s["x"] if c["scaled"] else None)
        got = dict(out=a.out, stream=a.res_out, d_residual=g["d_res"], d_x=g["d_x"],
                   d_w=g["d_w"], d_b=g["d_b"])
        if c["scaled"]:
            got["d_scale"] = g["d_scale"]
        return got
    if c["op"] == "ce":
        a = ssm.ssm_head_ce_fwd(s["h"], s["w"], s["target"], ignore_index=IGNORE)
        if c["train"]:
            g = ssm.ssm_head_ce_bwd(s["h"], s["w"], s["target"], a.lse, s["d_loss"],
                                    ignore_index=IGNORE)
    else:
        a = ssm.ssm_head_distill_fwd(s["h"], s["w"], s["t_idx"], s["t_logit"], temperature=c["tau"])
        if c["train"]:
            g = ssm.ssm_head_distill_bwd(s["h"], s["w"], s["t_idx"], s["t_logit"], a.lse,
                                         s["d_loss"], temperature=c["tau"])
    got = dict(loss=a.loss, lse=a.lse)
    if c["train"]:
        got.update(d_h=g["d_h"], d_w=g["d_w"])
    return got


def run(state):
    if own:
        return _own(state)
    return _layer_norm(state) if state["case"]["op"] == "layer_norm" else _head(state)


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    c = case
    b = 2 if c["io"] == "bf16" else 4
    if c["op"] == "layer_norm":
        n = c["rows"] * c["cols"]
        r = 2 if c["res"] == "bf16" else 4
        fwd = n * (2 * b + 2 * r)
        bwd = n * (2 * b + 2 * r) if c["train"] else 0
        return {"bytes": fwd + bwd, "flops": n * (9.0 + (18.0 if c["train"] else 0.0))}
    T, V, C = c["rows"], c["vocab"], c["cols"]
    ends = T * C * b + V * C * b  # h and W, or their gradients
    lists = T * 8 if c["op"] == "ce" else T * c["k"] * 12
    product = 2.0 * T * V * C  # the logits; then the two products with G
    return {"bytes": ends * (2 if c["train"] else 1) + lists + 8 * T,
            "flops": product * (3 if c["train"] else 1)}


# ---- the same in 64 bits ----------------------------------------------------------------------

def _exact_head(c, s):
    f = torch.float64
    T, V = c["rows"], c["vocab"]
    W = s["w"].to(f)
    loss = torch.zeros(T, dtype=f, device="cuda")
    lse = torch.zeros_like(loss)
    d_h = torch.zeros(T, c["cols"], dtype=f, device="cuda")
    d_w = torch.zeros_like(W)
    step = max(1, 2 ** 27 // V)
    for a in range(0, T, step):
        part = slice(a, min(T, a + step))
        h = s["h"][part].to(f)
        P = torch.zeros(h.shape[0], V, dtype=f, device="cuda")  # the target, over the vocabulary
        if c["op"] == "ce":
            tau = 1.0
            y = s["target"][part]
            some = y != IGNORE
            P[some.nonzero().squeeze(1), y[some]] = 1.0
        else:
            tau = c["tau"]
            i, t = s["t_idx"][part], s["t_logit"][part].to(f) / tau
            some = (i >= 0).any(dim=1)
            weight = torch.where(i >= 0, torch.exp(t - t.max(dim=1, keepdim=True).values), 0.0 * t)
            weight = weight / torch.sum(weight, 1, keepdim=True).clamp(min=1e-300)
            P.scatter_add_(1, torch.where(i >= 0, i, 0 * i), weight)
        z = torch.einsum("tc,vc->tv", h, W) / tau
        l = torch.logsumexp(z, dim=1)
        kl = torch.xlogy(P, P) - P * (z - l[:, None])
        loss[part] = torch.where(some, tau * tau * torch.sum(kl, 1), 0.0 * l)
        lse[part] = torch.where(some, l, 0.0 * l)
        if c["train"]:
            G = (torch.softmax(z, dim=1) - P) * tau
            G = G * (s["d_loss"][part].to(f) * some)[:, None]
            d_h[part] = torch.einsum("tv,vc->tc", G, W)
            d_w += torch.einsum("tv,tc->vc", G, h)
    got = dict(loss=loss, lse=lse)
    if c["train"]:
        got.update(d_h=d_h, d_w=d_w)
    return got


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] != "layer_norm":
        return _exact_head(c, s)
    f = torch.float64
    x, w, n_cols = s["x"].to(f), s["w"].to(f), c["cols"]
    scale = torch.ones_like(w) if s["scale"] is None else s["scale"].to(f)
    stream = s["residual"].to(f) + scale * x
    mean = torch.sum(stream, 1)[:, None] / n_cols
    off = stream - mean
    rstd = torch.pow(torch.sum(off * off, 1) / n_cols + EPS, -0.5)[:, None]
    got = dict(out=off * rstd * w + s["b"].to(f), stream=stream)
    if c["train"]:
        kept = stream.to(IO[c["res"]]).to(f)  # what the stream's own type holds of it
        n = (kept - mean) * rstd
        d_out = s["d_out"].to(f)
        up = d_out * w
        back = up - (torch.sum(up, 1)[:, None] + n * torch.sum(up * n, 1)[:, None]) / n_cols
        r = s["d_s"].to(f) + rstd * back
        got.update(d_residual=r, d_x=r * scale, d_w=torch.einsum("rc,rc->c", d_out, n),
                   d_b=torch.sum(d_out, 0),
                   d_scale=torch.einsum("rc,rc->c", r, x) if c["scaled"] else None)
    return got
