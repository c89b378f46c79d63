"""What the head keeps of its digits, where the bounds of head_ref are wide: long sums, fp32 operands, losses
near 0, temperatures, a few rows; against 64 bits on the GPU."""
import pytest
import torch

from bwd_ssm_conv_gb300 import head

pytestmark = pytest.mark.gpu
f64 = torch.float64


def _gradients(z, target, up, h, w):
    """(d_h, d_w) in 64 bits, and what their terms come to without their signs' cancelling between the
    softmax and the targets."""
    q = torch.softmax(z, 1)
    P = torch.zeros_like(q)
    P[torch.arange(z.shape[0], device=z.device), target] = 1.0
    G, size = (q - P) * up.to(f64)[:, None], (q + P) * up.to(f64).abs()[:, None]
    h, w = h.to(f64), w.to(f64)
    return (G @ w, G.t() @ h), (size @ w.abs(), size.t() @ h.abs())


def test_logits_of_many_columns_are_alike_in_both_directions():
    """65536 products of one sign: logits of 1160.  The tensor cores lose up to 2^-24 of a sum with each 16
    products, 64 times between two emptyings (1024 columns): 2^-18 of a logit at most, 4.4e-3, nearly all of
    which is that of lse too, as both are the same sums.  Left in one sum the 4096 additions of the backward
    alone lost 0.3.  Besides G and the result are rounded to bf16, 2^-8 of their terms in all."""
    T, D, V = 70, 65536, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.rand(T, D, generator=g, device="cuda").add(1).bfloat16()
    w = torch.rand(V, D, generator=g, device="cuda").add(1).mul(2.0 ** -7).bfloat16()
    y = torch.randint(V, (T,), generator=g, device="cuda")
    up = torch.ones(T, device="cuda")
    a = head.ssm_head_ce_fwd(h, w, y)
    got = head.ssm_head_ce_bwd(h, w, y, a.lse, up)
    z = h.to(f64) @ w.to(f64).t()
    assert float((a.lse - torch.logsumexp(z, 1)).abs().max()) < 4.4e-3 + 2.0 ** -14
    want, size = _gradients(z, y, up, h, w)
    for n, v, s in zip(("d_h", "d_w"), want, size):
        assert float(((got[n].to(f64) - v).abs() / s).max()) < 2.0 ** -8 + 2.0 ** -8 + 4.4e-3
