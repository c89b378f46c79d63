"""What the head keeps of its digits, where the bounds of head_ref are wide: long sums, fp32 operands, losses
near 0, temperatures, a few rows; against 64 bits on the GPU."""
import math

import pytest
import torch

import head_ref as ref
from bwd_ssm_conv_gb300 import binding, head
from head_ref import within
from test_gpu_head import DT, _ce, _ce_rows, _check, _distill, _entries, _inputs, _nan

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
    summed with each 16 products, 64 times at most between two emptyings (1024 columns): 2^-18 of a logit, 4.4e-3,
    part of which is that of lse too.  Left in one sum the 4096 additions of the backward
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


def _within_fine(got, i, rows, lse, tau=1.0):
    """Within the bounds of fp32 operands, whose G has 2^-22, and 2^-16 of each value of G besides; the results'
    own rounding apart."""
    h, w = i["h"].float(), i["w"].float()
    want, bound = ref.head_bwd(h, w, rows[0], rows[1], lse.cpu(), i["d_loss"], tau)
    z = torch.where(rows[1][:, None], h.to(f64), torch.zeros(1, dtype=f64)) @ w.to(f64).t() / tau
    up = torch.where(rows[1], i["d_loss"].to(f64) * tau, torch.zeros(1, dtype=f64))[:, None]
    G = ((torch.exp(z - lse.cpu().to(f64)[:, None]) - rows[0]) * up).abs()
    h = torch.where(rows[1][:, None], h, torch.zeros(1))
    for n, v, e, size in zip(("d_h", "d_w"), want, bound, (G @ w.to(f64).abs(), G.t() @ h.to(f64).abs())):
        if got[n] is not None:
            within(n, got[n], v, e + 2.0 ** -16 * size)


FINE = [  # (T, D, V): one stage to several, splits of either sum, odd sizes
    (5, 8, 40), (64, 64, 256), (70, 72, 700), (300, 515, 777), (129, 40, 5003), (900, 264, 300), (256, 72, 700),
    (257, 72, 700)]


@pytest.mark.parametrize("T,D,V", FINE)
def test_fine_gradients(T, D, V):
    i = _inputs(T, D, V, "bf16", seed=T + V)
    rows = _ce_rows(i)
    h, w, y, up = (i[n].cuda() for n in ("h", "w", "target", "d_loss"))
    a = head.ssm_head_ce_fwd(h, w, y)
    got = head.ssm_head_ce_bwd(h, w, y, a.lse, up, fine=True,
                               out=dict(d_h=_nan((T, D), h.dtype), d_w=_nan((V, D), h.dtype)))
    _within_fine(got, i, rows, a.lse)
    plain = head.ssm_head_ce_bwd(h, w, y, a.lse, up)
    if T <= 256:  # the same in any case
        assert torch.equal(plain["d_h"], got["d_h"]) and torch.equal(plain["d_w"], got["d_w"])
    else:
        with pytest.raises(AssertionError, match="times its bound"):  # what it is there for
            _within_fine(plain, i, rows, a.lse)
    # one gradient at a time, in a workspace of its size whatever that holds
    for grads, n in ((1, "d_h"), (2, "d_w")):
        ws = torch.full((head.ssm_head_workspace_size(T, D, V, grads=grads, aligned=D % 8 == 0, fine=True),),
                        255, dtype=torch.uint8, device="cuda")
        one = head.ssm_head_ce_bwd(h, w, y, a.lse, up, want_dh=grads == 1, want_dw=grads == 2, ws=ws,
                                   fine=True)
        _within_fine(one, i, rows, a.lse)
        assert binding.ssm_scan_status(ws) == binding.SSM_OK


@pytest.mark.parametrize("T,D,V,k,tau", [(33, 24, 20, 20, 1.0), (130, 72, 513, 64, 4.0), (300, 515, 777, 100, 0.7)])
def test_fine_gradients_of_distillation(T, D, V, k, tau):
    i = _inputs(T, D, V, "bf16", seed=T + k)
    i["t_idx"], i["t_logit"] = _entries(T, V, k, seed=k)
    rows = ref._p_of(i["t_idx"], i["t_logit"], tau, V)
    h, w, t_idx, t_logit, up = (i[n].cuda() for n in ("h", "w", "t_idx", "t_logit", "d_loss"))
    a = head.ssm_head_distill_fwd(h, w, t_idx, t_logit, temperature=tau)
    got = head.ssm_head_distill_bwd(h, w, t_idx, t_logit, a.lse, up, temperature=tau, fine=True)
    _within_fine(got, i, rows, a.lse, tau)


def test_fine_gradients_in_several_pieces_and_where_they_make_no_difference():
    T, D, V = 16384, 40, 9000  # 590 MB of G in two terms
    i = _inputs(T, D, V, "bf16", seed=5, ignored=0.1)
    h, w, y, up = (i[n].cuda() for n in ("h", "w", "target", "d_loss"))
    a = head.ssm_head_ce_fwd(h, w, y)
    got = head.ssm_head_ce_bwd(h, w, y, a.lse, up, fine=True)
    some = y != -100
    want, size = _gradients(h.to(f64) @ w.to(f64).t(), y.clamp(min=0), up * some, h, w)
    # 2^-16 of G, 60 units of 2^-24 of its softmax, 260 additions by 2^-23 in a stretch of the sums
    for n, v, s in zip(("d_h", "d_w"), want, size):
        within(n, got[n], v.cpu(), ((2.0 ** -16 + 60 * 2.0 ** -24 + 130 * 2.0 ** -23) * s).cpu())
    for T, io in ((4, "bf16"), (70, "f32"), (3, "f32")):
        i = _inputs(T, 72, 300, io, seed=T, ignored=0.0)
        h, w, y, up = (i[n].cuda() for n in ("h", "w", "target", "d_loss"))
        a = head.ssm_head_ce_fwd(h, w, y)
        p, q = (head.ssm_head_ce_bwd(h, w, y, a.lse, up, fine=fine) for fine in (False, True))
        assert torch.equal(p["d_h"], q["d_h"]) and torch.equal(p["d_w"], q["d_w"])


def test_a_fine_call_that_gives_up_reports_timeout():
    T, D, V = 300, 72, 700
    i = _inputs(T, D, V, "bf16", seed=6)
    h, w, y, up = (i[n].cuda() for n in ("h", "w", "target", "d_loss"))
    a = head.ssm_head_ce_fwd(h, w, y)
    ws = torch.empty(head.ssm_head_workspace_size(T, D, V, grads=3, fine=True), dtype=torch.uint8,
                     device="cuda")
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, up, ws=ws, fine=True, debug_flags=binding.SSM_DEBUG_NO_WAIT)
    assert binding.ssm_scan_status(ws) == binding.SSM_ERR_TIMEOUT
    assert bool(torch.isnan(g["d_h"]).all()) and bool(torch.isnan(g["d_w"]).all())
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, up, ws=ws, fine=True)
    assert binding.ssm_scan_status(ws) == binding.SSM_OK
    _within_fine(g, i, _ce_rows(i), a.lse)


@pytest.mark.parametrize("T,D,V", [(333, 256, 5003), (1021, 515, 10007), (40, 768, 3001)])
def test_fp32_products_keep_all_three_terms(T, D, V):
    """In the 2-norm, where errors of either sign do not add up as in a bound of each value: of G by its terms,
    the softmax and the targets, 2^-24 (16 + 16) where lse and z / tau are rounded below 32 (uniformly:
    1.1e-6 over sqrt 3), 2^-22 of the exponential and 3 x 2^-24 of the products left out; 1e-6 in all.  Without
    either product with the third terms it is 3e-6 to 2e-5.  lse: half a unit, and as much of what is left out
    of a logit."""
    i = _inputs(T, D, V, "f32", seed=T)
    a, g = _ce(i)
    h, w, y, up = (i[n].cuda() for n in ("h", "w", "target", "d_loss"))
    some = y != -100
    z = h.to(f64) @ w.to(f64).t()
    want = torch.logsumexp(z, 1)
    assert float(want.abs().max()) < 32
    assert float((a.lse - want)[some].norm() / want[some].norm()) < 2 * 2.0 ** -24
    up = torch.where(some, up, 0.0 * up)
    q = torch.softmax(z, 1)
    P = torch.zeros_like(q)
    P[torch.arange(T).cuda(), y.clamp(min=0)] = 1.0
    up = up.to(f64)[:, None]
    for n, left, right in (("d_h", lambda G: G, w), ("d_w", lambda G: G.t(), h)):
        right = right.to(f64)
        want = left((q - P) * up) @ right
        size = torch.sqrt((left(q * up) @ right).norm() ** 2 + (left(P * up) @ right).norm() ** 2)
        assert float((g[n] - want).norm() / size) < 1e-6, n


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40])
def test_a_loss_near_zero_keeps_its_digits(T, io):
    """Two words, logits 32 and 32 - d that are exact: the loss is log(1 + exp(-d)), formed from one sum next to 1
    (2^-24), an exponential (2^-22 of it and 2^-24 of its argument, 12) and a logarithm.  lse - z in fp32 is a
    multiple of 2^-18, which the losses here are a third of that or more away from."""
    losses = []
    for eighths in range(72, 98):
        h = torch.zeros(T, 8, dtype=DT[io])
        h[:, 0] = 4
        w = torch.zeros(2, 8, dtype=DT[io])
        w[0, 0], w[1, 0] = 8, 8 - eighths / 32
        assert 4 * float(w[1, 0]) == 32 - eighths / 8
        want = math.log1p(math.exp(-eighths / 8))
        if not 1 / 3 < want * 2 ** 18 % 1 < 2 / 3:
            continue
        losses.append(want)
        a = head.ssm_head_ce_fwd(h.cuda(), w.cuda(), torch.zeros(T, dtype=torch.long).cuda())
        assert float((a.loss.to(f64) - want).abs().max()) < 2.0 ** -24 + 2.0 ** -19 * want
    assert len(losses) >= 6 and min(losses) < 2e-5 and max(losses) > 1e-4


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("D,V", [(72, 700), (515, 1001), (1030, 40), (2304, 65)])
def test_a_few_bf16_rows_keep_G_in_fp32(T, D, V):
    """The bounds of fp32 operands, for what is stored in bf16."""
    i = _inputs(T, D, V, "bf16", seed=T * D, ignored=0.0)
    a, g = _ce(i)
    rows = _ce_rows(i)
    want, bound = ref.head_bwd(i["h"].float(), i["w"].float(), rows[0], rows[1], a.lse.cpu(), i["d_loss"])
    for n, v, e in zip(("d_h", "d_w"), want, bound):
        within(n, g[n], v, e)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("tau", [1e-6, 1e-4, 1e4, 1e6])
def test_temperatures_up_to_their_limits(T, tau, io):
    """Logits, the teacher's too, of a few temperatures."""
    i = _inputs(T, 72, 300, io, seed=11)
    i["h"] = (i["h"].float() * tau).to(DT[io])
    i["t_idx"], t = _entries(T, 300, 9, seed=5)
    i["t_logit"] = t * tau
    exact = float(torch.tensor(tau, dtype=torch.float32))
    _check(*_distill(i, tau), i, ref._p_of(i["t_idx"], i["t_logit"], exact, 300), exact)


@pytest.mark.parametrize("T,V,additions", [(70, 600, 16), (8192, 16000, 32)])
@pytest.mark.parametrize("D", [768, 1024, 2040])
def test_bf16_logits_are_as_good_as_fp32_sums(T, V, additions, D):
    """Products of one sign.  An addition to a sum in tensor memory loses a quarter of 2^-23 of it on average, and
    the sum grows evenly, so that n of them between two emptyings lose n / 2 x 2^-25 (16 with few tiles, 32 with
    many); half a unit of lse, and one of the sums outside.  Of 64 additions 5.7e-7 to 6.3e-7 were lost."""
    g = torch.Generator(device="cuda").manual_seed(D)
    h = torch.rand(T, D, generator=g, device="cuda").add(1).bfloat16()
    w = torch.rand(V, D, generator=g, device="cuda").add(1).mul(2.0 ** -6).bfloat16()
    y = torch.randint(V, (T,), generator=g, device="cuda")
    a = head.ssm_head_ce_fwd(h, w, y)
    want = torch.cat([torch.logsumexp(p.to(f64) @ w.to(f64).t(), 1) for p in h.split(1024)])
    off = float((a.lse.to(f64) - want).norm() / want.norm())
    assert off < additions / 2 * 2.0 ** -25 + 3 * 2.0 ** -25, off


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 300), (2, 20011), (8, 3001), (40, 3001), (300, 20011)])
@pytest.mark.parametrize("distil", [False, True])
def test_a_loss_far_below_one(T, V, distil, io):
    """A word that is all but certain, every other logit 18 to 32 below it, all exact: the loss, 4e-7 to 3e-5, is
    the others' sum without the 1 beside it.  An exponential is good to 2^-22, its argument, up to 32 log2(e), to
    two roundings; a term is scaled by at most 20 more of the former as sums are joined; and 64 additions."""
    g = torch.Generator().manual_seed(T + V)
    tau = 2.0 if distil else 1.0
    h = torch.zeros(T, 16)
    h[:, 0], h[:, 1] = 4 * tau, 1
    y = torch.randint(V, (T,), generator=g)
    w = torch.zeros(V, 16)
    w[:, 0] = -torch.randint(72, 128, (V,), generator=g) / 16  # 4.5 .. 7.9
    top = int(y[0])  # one word for all rows
    w[top, 0] = 0
    y[:] = top
    z = (h.to(f64) @ w.to(f64).t() / tau).cuda()
    assert torch.equal(h.bfloat16().float(), h) and torch.equal(w.bfloat16().float(), w)
    others = z.clone()
    others[:, top] = -float("inf")
    want = torch.log1p(torch.exp(others - z[:, top, None]).sum(1))
    h, w = h.to(DT[io]).cuda(), w.to(DT[io]).cuda()
    if distil:
        idx, t = y[:, None].cuda(), torch.zeros(T, 1, device="cuda")
        got, want = head.ssm_head_distill_fwd(h, w, idx, t, temperature=tau).loss, tau * tau * want
    else:
        got = head.ssm_head_ce_fwd(h, w, y.cuda()).loss
    limit = 21 * 2.0 ** -22 + 2 * 32 * 2.0 ** -24 + 64 * 2.0 ** -24
    off = float(((got.to(f64) - want) / want).abs().max())
    assert float(want.max()) < 1e-3 and off < limit, (off, limit)
