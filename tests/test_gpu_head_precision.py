"""What the head keeps of its digits, where the bounds of head_ref are wide: long sums, fp32 operands, losses
near 0, temperatures, a few rows; against 64 bits on the GPU."""
import math

import pytest
import torch

from bwd_ssm_conv_gb300 import head
from test_gpu_head import _ce, _inputs

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
    """65536 products of one sign: logits of 1160.  The tensor cores lose up to 2^-23 of what they have
    summed with each 16 products, 64 times between two emptyings (1024 columns): 2^-18 of a logit, 4.4e-3, nearly all of
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


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("tau", [1e-6, 1e-3, 1.0, 1e6])
def test_a_teacher_is_as_exact_at_any_temperature(T, tau):
    """Logits a few temperatures apart, around 7: their distances, exact to 2^-24, over tau are below 40, so that
    p is good to 40 x 2^-23 and expf's two units, 5e-6.  The student is even (W is 0), so that nothing else is off."""
    D, V, k = 16, 64, 5
    g = torch.Generator().manual_seed(4)
    h, w = torch.randn(T, D, generator=g).cuda(), torch.zeros(V, D).cuda()
    t_logit = (7.0 + tau * 4 * torch.randn(T, k, generator=g)).cuda()
    t_idx = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(T)]).cuda()
    a = head.ssm_head_distill_fwd(h, w, t_idx, t_logit, temperature=tau)
    got = head.ssm_head_distill_bwd(h, w, t_idx, t_logit, a.lse, torch.ones(T).cuda(), temperature=tau)
    tau = float(torch.tensor(tau, dtype=torch.float32))  # as the call has it
    t = t_logit.to(f64) / tau
    assert float((t.amax(1) - t.amin(1)).max()) < 40
    p = torch.softmax(t, 1)
    want = (p * (torch.log_softmax(t, 1) + math.log(V))).sum(1)
    assert float(((a.loss.to(f64) / tau ** 2 - want).abs() / want).max()) < 1e-5
    G = torch.full((T, V), 1.0 / V, dtype=f64, device="cuda").scatter_add_(1, t_idx, -p) * tau
    want = G.t() @ h.to(f64)
    assert float((got["d_w"].to(f64) - want).norm() / want.norm()) < 1e-5


@pytest.mark.parametrize("T", [3, 70])
def test_a_teachers_logits_of_any_size(T):
    """Their quotients by the temperature are past fp32, their distances take p to 1 and 0."""
    t_logit = torch.tensor([1e35, 3e34, -2e37]).repeat(T, 1).cuda()
    t_idx = torch.arange(3).repeat(T, 1).cuda()
    h, w = torch.ones(T, 8).cuda(), torch.zeros(16, 8).cuda()
    a = head.ssm_head_distill_fwd(h, w, t_idx, t_logit, temperature=1e-4)
    assert float((a.loss.to(f64) / 1e-8 - math.log(16)).abs().max()) < 1e-5


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 9, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_no_row_that_counts_beside_weights_that_are_not_finite(T, io, bad):
    i = _inputs(T, 72, 300, io, seed=7)
    i["target"][:] = -100
    i["w"][5] = bad
    a, g = _ce(i)
    for t in (a.loss, a.lse, g["d_h"], g["d_w"]):
        assert bool((t == 0).all())


def _above_a_tie(n, cols, share, factor, seed):
    """bf16 [n][cols] of values in [1, 2), whose sum over n times ``factor`` (an integer) lies above the middle
    between two bf16 numbers by ``share`` of itself, or a little more."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(128, 256, (n, cols), generator=g, device="cuda")  # units of 2^-7
    m = n // 8  # the rows that make up what the sum lacks
    rest = x[m:].sum(0)
    total = (rest + 192 * m) * factor
    step = 2 ** (torch.floor(torch.log2(total.to(f64))).long() - 7)  # between two bf16 numbers
    middle = total // step * step + step // 2
    aim = torch.ceil(middle.to(f64) * (1 + share) / factor).long()
    lack = aim - rest
    x[:m] = lack // m
    x[:m] += torch.arange(m, device="cuda")[:, None] < lack % m
    assert bool((x.sum(0) == aim).all()) and 128 <= int(x.min()) and int(x.max()) < 256
    return (x.to(f64) / 128).bfloat16()


def _even(T, D, V, h, w):
    """Gradients for logits of 0 and targets of 0: G is 141 x 2^-k, which is what bf16 makes of 1 / V."""
    q = torch.tensor(1.0 / V).bfloat16().double()
    assert float(q) * V == pytest.approx(1.0, abs=1e-3) and (float(q) * 2.0 ** 40) % 141 == 0
    y, up = torch.zeros(T, dtype=torch.long, device="cuda"), torch.ones(T, device="cuda")
    a = head.ssm_head_ce_fwd(h, w, y)
    return float(q), head.ssm_head_ce_bwd(h, w, y, a.lse, up)


# Sums of equal signs lose up to 2^-23 of what they are with each 16 terms: left in one sum the 29747 words
# lose 2^-23 x 1859 / 2 = 1.1e-4 of it and the 65536 rows 2.4e-4; emptied every 4096 terms at most 256 additions
# are lost by, 1.5e-5, and what is emptied is added with rounding to nearest (16 x 2^-24).  A sum that is 3e-5
# above the middle between two bf16 numbers is then rounded up as it should be.
def test_sums_over_many_words_are_rounded_as_they_should_be():
    T, D, V = 8192, 2048, 29747
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[1:] = _above_a_tie(V - 1, D, 3e-5, 141, seed=1)
    q, g = _even(T, D, V, torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"), w)
    want = (w.to(f64).sum(0) * q).bfloat16()
    assert int((g["d_h"] != want).sum()) == 0


def test_sums_over_many_rows_are_rounded_as_they_should_be():
    T, D, V = 65536, 4096, 3718
    h = _above_a_tie(T, D, 3e-5, 141, seed=2)
    q, g = _even(T, D, V, h, torch.zeros(V, D, dtype=torch.bfloat16, device="cuda"))
    want = (h.to(f64).sum(0) * q).bfloat16()
    assert int((g["d_w"][1:] != want).sum()) == 0
