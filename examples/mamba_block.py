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

``python examples/mamba_block.py`` trains a small model of such blocks for some steps with and
without the checkpoints and prints the losses, the memory kept and the time per step.
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


if __name__ == "__main__":
    main()
