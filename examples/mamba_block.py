"""A Mamba block (its scalar-A form) from the library's calls, trained and decoded.

    s   = residual + h                       ssm_add_norm_fwd: the stream, and u = norm(s)
    z, x, B, C, dt = u W_in^T                a library matrix product
    x   = silu(conv1d(x))                    ssm_conv_fwd
    y   = scan(x, dt, A, B, C, D)            ssm_scan_fwd
    v   = norm(y silu(z))                    ssm_gated_norm_fwd
    out = v W_out^T                          a library matrix product

Between forward and backward a block keeps its activations in 8 bits (``save8``): the stream (for the
first norm's backward), u and v (for the projections' weight gradients), y and z (for the gated
norm's backward).  The norms write these checkpoints in the pass that computes them; the backward
calls read them without unpacking them to memory first.

``Head`` ends a language model of such blocks: the last layer norm with the residual add
(ssm_add_layer_norm_fwd), the head and the loss, cross entropy against the next token (ssm_head_ce_fwd) or
distillation from a teacher's top logits (ssm_head_distill_fwd), whose logits are never kept.

``python examples/mamba_block.py`` trains a small model of such blocks for some steps with and
without the checkpoints and prints the losses, the memory kept and the time per step, then the same as a
language model over a vocabulary.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_ssm_conv_gb300 as ssm  # noqa: E402


@dataclass(frozen=True)
class Shape:
    d_model: int
    n_head: int
    head_dim: int
    d_state: int
    d_conv: int = 4
    group: int = 0          # columns per gated norm (0: all)
    chunk: int = 64

    @property
    def d_inner(self):
        return self.n_head * self.head_dim

    @property
    def widths(self):       # of the parts of the input projection: z, x, B, C, dt
        return (self.d_inner, self.d_inner, self.d_state, self.d_state, self.n_head)


class Block:
    """One block's weights; activations in ``io``, parameters in fp32."""

    def __init__(self, shape: Shape, seed: int, io=torch.bfloat16, device="cuda"):
        s, g = shape, torch.Generator().manual_seed(seed)

        def rand(*size, std):
            return (std * torch.randn(*size, generator=g)).to(device)

        self.shape, self.io = s, io
        self.p = dict(
            w1=torch.ones(s.d_model, device=device), w2=torch.ones(s.d_inner, device=device),
            W_in=rand(sum(s.widths), s.d_model, std=s.d_model ** -0.5),
            W_out=rand(s.d_model, s.d_inner, std=s.d_inner ** -0.5),
            c=rand(s.d_inner, s.d_conv, std=0.3),
            A=-torch.exp(torch.rand(s.n_head, generator=g)).to(device),
            D=torch.ones(s.d_inner, device=device),
            dt_bias=torch.full((s.n_head,), -2.0, device=device))

    def _project(self, u):
        """The parts of the input projection; z stays a slice of it."""
        p = u @ self.p["W_in"].to(self.io).t()
        z, x, B, C, dt = p.split(self.shape.widths, dim=-1)
        return z, x, B.contiguous(), C.contiguous(), dt.contiguous()

    def forward(self, h, residual, save8=True):
        """h [n_s][L][d_model], residual the stream (or None); (out, stream, what backward needs)."""
        s, p = self.shape, self.p
        n, L, _ = h.shape
        a = ssm.ssm_add_norm_fwd(h, p["w1"], residual, res_dtype=torch.float32, save8=save8,
                                 save_out8=save8)
        z, x, B, C, dt = self._project(a.out)
        sx = torch.nn.functional.pad(x.transpose(1, 2), (s.d_conv - 1, 0)).contiguous()
        x = ssm.ssm_conv_fwd(sx, p["c"]).view(n, L, s.n_head, s.head_dim)
        scan = dict(dt=dt, A=p["A"], B=B.view(n, L, 1, -1), C=C.view(n, L, 1, -1), D=p["D"],
                    dt_bias=p["dt_bias"], chunk=s.chunk, softplus=True)
        y, _, ckpt = ssm.ssm_scan_fwd(x, **scan)
        y = y.view(n, L, s.d_inner)
        v = ssm.ssm_gated_norm_fwd(y, z, p["w2"], group=s.group, save8=save8, save_out8=save8)
        out = v.out @ p["W_out"].to(self.io).t()
        # x is computed again from sx in the backward
        kept = dict(rstd=a.rstd, s=a.res8 if save8 else a.res_out, u=a.out8 if save8 else a.out,
                    y=v.y8 if save8 else y, z=v.z8 if save8 else z, rstd_v=v.rstd,
                    v=v.out8 if save8 else v.out, sx=sx, scan=scan, ckpt=ckpt)
        return out, a.res_out, kept

    @staticmethod
    def _weight_grad(g, x):
        """sum over rows of g x^T in fp32, from x's checkpoint or from x itself (a library product of
        the activations' type with fp32 sums)."""
        if isinstance(x, ssm.Ckpt8):
            return ssm.ssm_ckpt8_wgrad(g, x)
        g, x = g.flatten(0, -2), x.flatten(0, -2)
        return g.t() @ x if g.dtype == torch.float32 else torch.mm(g.t(), x, out_dtype=torch.float32)

    def backward(self, d_out, d_stream, kept):
        """(d_h, d_residual, gradients by name); d_stream: the gradient that reaches the stream past
        this block, or None."""
        s, p, k = self.shape, self.p, kept
        n, L, _ = d_out.shape
        g = {}
        g["W_out"] = self._weight_grad(d_out, k["v"])
        d_v = d_out @ p["W_out"].to(self.io)
        d_p = torch.empty(n, L, sum(s.widths), dtype=self.io, device=d_out.device)
        d_zxbcdt = d_p.split(s.widths, dim=-1)
        d_y = torch.empty(n, L, s.d_inner, dtype=self.io, device=d_out.device)
        b = ssm.ssm_gated_norm_bwd(d_v, k["y"], k["z"], k["rstd_v"], p["w2"], group=s.group,
                                   out=dict(d_y=d_y, d_z=d_zxbcdt[0],
                                            d_w=torch.empty_like(p["w2"])))
        g["w2"] = b["d_w"]
        x = ssm.ssm_conv_fwd(k["sx"], p["c"]).view(n, L, s.n_head, s.head_dim)
        b = ssm.ssm_scan_bwd(x, dy=d_y.view(x.shape), ckpt=k["ckpt"], want_ds0=False, **k["scan"])
        g["A"], g["D"], g["dt_bias"] = b["d_A"], b["d_D"], b["d_dt_bias"]
        d_sx, g["c"], _ = ssm.ssm_conv_bwd(k["sx"], p["c"], b["d_x"].view(n, L, s.d_inner))
        for part, d in zip(d_zxbcdt[1:], (d_sx[:, :, s.d_conv - 1:].transpose(1, 2),
                                          b["d_B"].view(n, L, -1), b["d_C"].view(n, L, -1),
                                          b["d_dt"])):
            part.copy_(d)
        g["W_in"] = self._weight_grad(d_p, k["u"])
        d_u = d_p @ p["W_in"].to(self.io)
        b = ssm.ssm_add_norm_bwd(d_u, k["s"], k["rstd"], p["w1"], d_res_out=d_stream,
                                 res_dtype=torch.float32)
        g["w1"] = b["d_w"]
        return b["d_x"], b["d_res"], g

    def new_cache(self, n_seqs):
        """The conv and scan states that decode() rolls."""
        s, dev = self.shape, self.p["A"].device
        return (torch.zeros(n_seqs, s.d_inner, s.d_conv - 1, dtype=self.io, device=dev),
                torch.zeros(n_seqs, s.n_head, s.head_dim, s.d_state, device=dev))

    def decode(self, h, residual, cache):
        """One token per sequence: h [n_s][d_model]; (out, stream)."""
        s, p = self.shape, self.p
        n = h.shape[0]
        a = ssm.ssm_add_norm_fwd(h, p["w1"], residual, res_dtype=torch.float32, want_rstd=False)
        z, x, B, C, dt = self._project(a.out)
        y = ssm.ssm_decode_step(x.contiguous().view(n, s.n_head, s.head_dim), cache[0], p["c"], dt,
                                p["A"], B.view(n, 1, -1), C.view(n, 1, -1), cache[1], D=p["D"],
                                dt_bias=p["dt_bias"], softplus=True)
        v = ssm.ssm_gated_norm_fwd(y.view(n, s.d_inner), z, p["w2"], group=s.group,
                                   want_rstd=False)
        return v.out @ p["W_out"].to(self.io).t(), a.res_out


class Head:
    """The end of a language model: the last norm and the head's weights, one row per word (the embedding
    may be the same); parameters in fp32."""

    def __init__(self, d_model, vocab, seed: int, io=torch.bfloat16, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.io = io
        self.p = dict(w=torch.ones(d_model, device=device), b=torch.zeros(d_model, device=device),
                      W=(d_model ** -0.5 * torch.randn(vocab, d_model, generator=g)).to(device))

    def embed(self, tokens):
        return self.p["W"][tokens].to(self.io)

    def weights(self):
        """A copy of W in the activations' type."""
        return self.p["W"].to(self.io)

    def forward(self, h, residual, target, teacher=None, temperature=1.0, W=None):
        """The loss of each row of h [...][d_model] and what backward needs.  target [...]: the next
        tokens, -100 where there is none; or teacher: (t_idx, t_logit) of each row.  W: weights(), where more
        than one call takes it."""
        a = ssm.ssm_add_layer_norm_fwd(h, self.p["w"], self.p["b"], residual, res_dtype=torch.float32)
        W = self.weights() if W is None else W
        if teacher is None:
            r = ssm.ssm_head_ce_fwd(a.out, W, target)
        else:
            r = ssm.ssm_head_distill_fwd(a.out, W, *teacher, temperature=temperature)
        return r.loss, dict(norm=a, W=W, lse=r.lse, target=target, teacher=teacher,
                            temperature=temperature)

    def backward(self, d_loss, kept):
        """(d_h, d_residual, gradients by name) of sum(d_loss * loss)."""
        a, k = kept["norm"], kept
        if k["teacher"] is None:
            b = ssm.ssm_head_ce_bwd(a.out, k["W"], k["target"], k["lse"], d_loss)
        else:
            b = ssm.ssm_head_distill_bwd(a.out, k["W"], *k["teacher"], k["lse"], d_loss,
                                         temperature=k["temperature"])
        n = ssm.ssm_add_layer_norm_bwd(b["d_h"], a.res_out, a.mean, a.rstd, self.p["w"],
                                       res_dtype=torch.float32)
        return n["d_x"], n["d_res"], dict(w=n["d_w"], b=n["d_b"], W=b["d_w"].float())


def kept_bytes(kept):
    """Bytes of the activations that a block keeps for its backward."""
    total = 0
    for v in kept.values():
        for t in (v.values() if isinstance(v, dict) else v if isinstance(v, tuple) else (v,)):
            total += t.numel() * t.element_size() if torch.is_tensor(t) else 0
    return total


def train_step(blocks, h, target, save8, lr=0.0):
    """One step of regression of the last stream onto ``target``; (loss per token, bytes kept)."""
    kept, stream, x, n_bytes = [], None, h, 0
    for b in blocks:
        x, stream, k = b.forward(x, stream, save8)
        kept.append(k)
        n_bytes += kept_bytes(k)
    tokens = h.shape[0] * h.shape[1]
    d_stream = stream + x.float() - target
    loss = 0.5 * (d_stream ** 2).sum() / tokens
    d_stream /= tokens
    d_x = d_stream.to(blocks[0].io)
    for b, k in zip(reversed(blocks), reversed(kept)):
        d_x, d_stream, g = b.backward(d_x, d_stream, k)
        for name, v in g.items():
            b.p[name] -= lr * v
        b.p["A"].clamp_(max=-0.01)
    return float(loss), n_bytes


def lm_step(blocks, head, tokens, save8=True, lr=0.0, teacher=None, temperature=1.0):
    """One step of a language model on tokens [n_s][L], each to be told from those before it; the mean
    loss.  The embedding is the head's weights."""
    target = torch.full_like(tokens, -100)  # the last token of a sequence has no next one
    target[:, :-1] = tokens[:, 1:]
    kept, stream, x = [], None, head.embed(tokens)
    for b in blocks:
        x, stream, k = b.forward(x, stream, save8)
        kept.append(k)
    loss, last = head.forward(x, stream, target, teacher, temperature)
    rows = tokens.numel() if teacher is not None else max(1, tokens.shape[0] * (tokens.shape[1] - 1))
    d_x, d_stream, g_head = head.backward(torch.full_like(loss, 1.0 / rows), last)
    for b, k in zip(reversed(blocks), reversed(kept)):
        d_x, d_stream, g = b.backward(d_x, d_stream, k)
        for name, v in g.items():
            b.p[name] -= lr * v
        b.p["A"].clamp_(max=-0.01)
    # the first block's h is the embedding
    g_head["W"].index_add_(0, tokens.flatten(), d_x.float().flatten(0, 1))
    for name, v in g_head.items():
        head.p[name] -= lr * v
    return float(loss.sum() / rows)


def score(blocks, head, tokens):
    """The log-probability of each token of tokens [n_s][L] after the first, a token at a time."""
    n, L = tokens.shape
    caches, W = [b.new_cache(n) for b in blocks], head.weights()
    out = torch.empty(n, L - 1, device=tokens.device)
    for t in range(L - 1):
        x, stream = head.embed(tokens[:, t]), None
        for b, c in zip(blocks, caches):
            x, stream = b.decode(x, stream, c)
        loss, _ = head.forward(x, stream, tokens[:, t + 1].contiguous(), W=W)
        out[:, t] = -loss
    return out


def main():
    shape = Shape(d_model=768, n_head=24, head_dim=64, d_state=128)
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(8, 1024, shape.d_model, generator=g, device="cuda").bfloat16()
    target = torch.randn(8, 1024, shape.d_model, generator=g, device="cuda")
    for save8 in (False, True):
        blocks = [Block(shape, seed=i) for i in range(4)]
        losses = [train_step(blocks, h, target, save8, lr=1e-3)[0] for _ in range(10)]
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        for _ in range(5):
            _, n = train_step(blocks, h, target, save8)
        end.record()
        torch.cuda.synchronize()
        print(f"save8={save8}: loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
              f"{n / 2 ** 20:.0f} MiB kept, {start.elapsed_time(end) / 5:.2f} ms per step")

    blocks, head = [Block(shape, seed=i) for i in range(4)], Head(shape.d_model, 32768, seed=9)
    tokens = torch.randint(32768, (8, 1024), generator=g, device="cuda")
    losses = [lm_step(blocks, head, tokens, lr=1e-2) for _ in range(10)]
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(5):
        lm_step(blocks, head, tokens)
    end.record()
    torch.cuda.synchronize()
    print(f"language model over 32768 words: loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
          f"{start.elapsed_time(end) / 5:.2f} ms per step, log-probability a token at a time "
          f"{score(blocks, head, tokens[:1, :16]).mean():.4f}")


if __name__ == "__main__":
    main()
