"""The head with its losses against their 64-bit forms (head_ref, where the bounds are derived), on the
GPU."""
import time

import pytest
import torch

import head_ref as ref
from bwd_ssm_conv_gb300 import SsmError, binding, block, head
from head_ref import within

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
f64 = torch.float64


def _nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _inputs(T, D, V, io, seed, ignored=0.3):
    """Hidden states that know something of their target; upstream gradients of every size and sign."""
    g = torch.Generator().manual_seed(seed)
    w = _rand(g, V, D, std=D ** -0.5)
    y = torch.randint(V, (T,), generator=g)
    h = _rand(g, T, D) + 12 * torch.rand(T, 1, generator=g) * w[y]
    y[torch.rand(T, generator=g) < ignored] = -100
    up = _rand(g, T) * torch.exp(2 * _rand(g, T))
    return dict(h=h.to(DT[io]), w=w.to(DT[io]), target=y, d_loss=up)


def _entries(T, V, k, seed):
    """(t_idx, t_logit): entries that are missing, rows without any, a word twice, logits of -infinity."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(V, generator=g)[:k] if V >= k else torch.randint(V, (k,), generator=g)
                       for _ in range(T)])
    logit = _rand(g, T, k, std=2.0)
    idx[torch.rand(T, k, generator=g) < 0.2] = -1
    idx[torch.rand(T, generator=g) < 0.15] = -7
    if k > 2:
        twice = torch.rand(T, generator=g) < 0.3
        idx[twice, 1] = idx[twice, 0]
        logit[torch.rand(T, generator=g) < 0.2, 2] = -float("inf")
    return idx, logit


def _ce(i, want=("loss", "d_h", "d_w"), h=None, w=None, **how):
    """The calls on the GPU, results in buffers of NaN."""
    h = i["h"].cuda() if h is None else h
    w = i["w"].cuda() if w is None else w
    y = i["target"].cuda()
    T = y.shape[0]
    a = head.ssm_head_ce_fwd(h, w, y, out=(_nan((T,), torch.float32), _nan((T,), torch.float32)), **how)
    into = dict(d_h=_nan(h.shape, h.dtype) if "d_h" in want else None,
                d_w=_nan(w.shape, w.dtype) if "d_w" in want else None)
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, i["d_loss"].cuda(), out=into, **how)
    return a, g


def _distill(i, tau, h=None, w=None, **how):
    h = i["h"].cuda() if h is None else h
    w = i["w"].cuda() if w is None else w
    e = i["t_idx"].cuda(), i["t_logit"].cuda()
    T = h.shape[0]
    a = head.ssm_head_distill_fwd(h, w, *e, temperature=tau,
                                  out=(_nan((T,), torch.float32), _nan((T,), torch.float32)), **how)
    g = head.ssm_head_distill_bwd(h, w, *e, a.lse, i["d_loss"].cuda(), temperature=tau,
                                  out=dict(d_h=_nan(h.shape, h.dtype), d_w=_nan(w.shape, w.dtype)), **how)
    return a, g


def _check(a, g, i, rows, tau=1.0):
    (loss, lse), (dloss, dlse) = ref.head(i["h"], i["w"], *rows, tau=tau)
    within("loss", a.loss, loss, dloss)
    within("lse", a.lse, lse, dlse)
    (d_h, d_w), (dd_h, dd_w) = ref.head_bwd(i["h"], i["w"], rows[0], rows[1], a.lse.cpu(), i["d_loss"], tau)
    if g["d_h"] is not None:
        within("d_h", g["d_h"], d_h, dd_h)
    if g["d_w"] is not None:
        within("d_w", g["d_w"], d_w, dd_w)


def _ce_rows(i):
    return ref.ce_rows(i["target"], i["w"].shape[0])


SIZES = [  # (T, D, V): one of each; either side of a stage, of a CTA's half and of a pair's tile
    (1, 1, 1), (1, 8, 2), (3, 5, 7), (1, 768, 1000), (64, 64, 256), (65, 72, 257), (127, 63, 129),
    (128, 65, 511), (130, 264, 513), (257, 129, 300), (300, 515, 777), (2, 256, 3000),
    (700, 40, 1025), (513, 512, 256), (1000, 96, 600), (200, 1030, 130),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_ce(T, D, V, io):
    i = _inputs(T, D, V, io, seed=T + D + V, ignored=0.0 if T == 1 else 0.3)
    _check(*_ce(i), i, _ce_rows(i))


KD = [  # (T, D, V, k, tau)
    (1, 8, 3, 1, 1.0), (5, 40, 9, 3, 2.0), (64, 64, 300, 17, 1.0), (130, 72, 513, 64, 4.0),
    (300, 515, 777, 100, 1.5), (257, 96, 1030, 128, 0.7), (1, 768, 1000, 128, 1.0),
    (33, 24, 2, 2, 1.0), (40, 16, 20, 128, 1.0),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("entry_io", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,V,k,tau", KD)
def test_distill(T, D, V, k, tau, io, entry_io):
    i = _inputs(T, D, V, io, seed=T + V + k)
    i["t_idx"], t = _entries(T, V, k, seed=k)
    i["t_logit"] = t.to(DT[entry_io])
    _check(*_distill(i, tau), i, ref._p_of(i["t_idx"], i["t_logit"], tau, V), tau)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D,V", [(8, 3), (72, 700), (515, 1001), (1030, 40), (2048, 300)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
def test_a_few_rows(T, D, V, io):
    """Up to 2 and 4 rows, 8 in fp32, forward and backward are kernels of their own; rows that do not count among them."""
    i = _inputs(T, D, V, io, seed=T * D + V, ignored=0.0)
    if T > 2:
        i["target"][T // 2] = -100
        i["h"][T // 2] = float("nan")
    _check(*_ce(i), i, _ce_rows(i))
    k = min(V, 20)
    i["t_idx"], i["t_logit"] = _entries(T, V, k, seed=T)
    i["h"] = torch.nan_to_num(i["h"])
    _check(*_distill(i, 1.5), i, ref._p_of(i["t_idx"], i["t_logit"], 1.5, V), 1.5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lead,tail", [(0, 8), (8, 0), (3, 2), (1, 8)])  # aligned slices, and not
def test_strided_and_misaligned_rows(lead, tail, io):
    for T in (70, 3):  # 3: a few rows
        _strided(T, 136, 270, io, lead, tail)


def _strided(T, D, V, io, lead, tail):
    i = _inputs(T, D, V, io, seed=4)

    def strided(t):
        wide = _nan((t.shape[0], lead + D + tail), t.dtype)
        wide[:, lead:lead + D] = t.cuda()
        return wide[:, lead:lead + D]

    h, w, y = strided(i["h"]), strided(i["w"]), i["target"].cuda()
    a = head.ssm_head_ce_fwd(h, w, y)
    d_h = strided(torch.zeros(T, D, dtype=DT[io]))
    flat = _nan((V * D + 1,), DT[io])  # d_w anywhere, but without gaps
    d_w = flat[lead & 1:][:V * D].view(V, D)
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, i["d_loss"].cuda(), out=dict(d_h=d_h, d_w=d_w))
    _check(a, g, i, _ce_rows(i))
    wide = d_h._base
    assert bool(torch.isnan(wide[:, :lead]).all()) and bool(torch.isnan(wide[:, lead + D:]).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("want", ["d_h", "d_w"])
def test_each_gradient_by_itself(want, io):
    i = _inputs(150, 72, 400, io, seed=6)
    both = _ce(i)[1]
    only = _ce(i, want=(want,))[1]
    other = "d_w" if want == "d_h" else "d_h"
    assert only[other] is None and torch.equal(only[want], both[want])
    a = head.ssm_head_ce_fwd(i["h"].cuda(), i["w"].cuda(), i["target"].cuda())
    g = head.ssm_head_ce_bwd(i["h"].cuda(), i["w"].cuda(), i["target"].cuda(), a.lse,
                             i["d_loss"].cuda(), want_dh=want == "d_h", want_dw=want == "d_w")
    assert g[other] is None and torch.equal(g[want], both[want])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 64, 300])
def test_rows_without_a_loss_are_zeros_whatever_they_hold(T, io):
    i = _inputs(T, 72, 300, io, seed=7)
    i["target"][:] = -100
    i["h"][:] = float("nan")
    for a, g in (_ce(i), _distill(dict(i, t_idx=torch.full((T, 5), -1), t_logit=torch.zeros(T, 5)), 2.0)):
        for t in (a.loss, a.lse, g["d_h"], g["d_w"]):
            assert bool((t == 0).all())
    if T > 1:  # beside rows that have one
        i = _inputs(T, 72, 300, io, seed=8, ignored=0.4)
        clean = _ce(i)
        i["h"][i["target"] == -100] = float("inf")
        i["d_loss"][i["target"] == -100] = float("nan")
        a, g = _ce(i)
        for p, q in zip((*clean[0], *clean[1].values()), (*a, *g.values())):
            assert torch.equal(p, q)


def test_words_outside_the_vocabulary_spoil_their_row_only():
    T, D, V = 90, 64, 300
    i = _inputs(T, D, V, "bf16", seed=9, ignored=0.2)
    good = dict(i, target=i["target"].clone())
    bad = torch.tensor([3, 40, 88])
    i["target"][bad] = torch.tensor([V, -1, 1 << 40])
    good["target"][bad] = -100  # what the others should be like
    h, w, y, up = i["h"].cuda(), i["w"].cuda(), i["target"].cuda(), i["d_loss"].cuda()
    ws = torch.full((max(head.ssm_head_workspace_size(T, D, V, grads=n) for n in (0, 3)),), 255,
                    dtype=torch.uint8, device="cuda")
    a = head.ssm_head_ce_fwd(h, w, y, ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_ERR_INVALID_ARG
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, up, ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_ERR_INVALID_ARG
    for t in (a.loss, a.lse, g["d_h"]):
        assert bool(torch.isnan(t[bad.cuda()]).all())
        t[bad.cuda()] = 0
    _check(a, g, good, _ce_rows(good))
    # a teacher's word beyond the vocabulary
    t_idx, t_logit = _entries(T, V, 4, seed=1)
    t_idx[:, 3] = 5
    good = t_idx.clone()
    t_idx[bad, 1], good[bad] = V, -1
    i.update(t_idx=t_idx, t_logit=t_logit)
    a, g = _distill(i, 1.0)
    for t in (a.loss, a.lse, g["d_h"]):
        assert bool(torch.isnan(t[bad.cuda()]).all())
        t[bad.cuda()] = 0
    _check(a, g, i, ref._p_of(good, t_logit, 1.0, V))
    # the next call clears the status
    head.ssm_head_ce_fwd(h, w, torch.zeros_like(y), ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_OK


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_large_logits_and_gradients_of_zero(io):
    """Logits of thousands: one word takes everything, and losses are differences of large numbers;
    upstream gradients of 0 for all rows, then for some."""
    i = _inputs(100, 64, 500, io, seed=10)
    i["h"] = (i["h"].float() * 300).to(DT[io])
    _check(*_ce(i), i, _ce_rows(i))
    i = _inputs(100, 64, 500, io, seed=11)
    i["d_loss"].zero_()
    a, g = _ce(i)
    assert bool((g["d_h"] == 0).all()) and bool((g["d_w"] == 0).all())
    i["d_loss"][20:40] = torch.linspace(-1e-30, 1e-6, 20)
    _check(a, _ce(i)[1], i, _ce_rows(i))


def test_bad_values_stay_in_their_rows():
    i = _inputs(80, 64, 300, "f32", seed=12, ignored=0.0)
    i["h"][7, 3], i["h"][70, 5] = float("nan"), float("inf")
    i["d_loss"][33] = float("inf")
    fine = torch.ones(80, dtype=torch.bool)
    fine[[7, 70, 33]] = False
    a, g = _ce(i)
    assert bool(torch.isfinite(a.loss.cpu()[fine]).all()) and bool(torch.isfinite(g["d_h"].cpu()[fine]).all())
    assert bool(torch.isnan(a.loss[7])) and not bool(torch.isfinite(g["d_h"].cpu()[[7, 33]]).any())
    i["t_idx"], i["t_logit"] = _entries(80, 300, 5, seed=3)
    i["t_idx"][:, 3:] = torch.tensor([5, 6])
    i["t_logit"][11, 4] = float("nan")
    i["h"] = torch.nan_to_num(i["h"])
    a, g = _distill(i, 1.0)
    assert torch.isnan(a.loss).nonzero().flatten().tolist() == [11]


def test_a_dirty_workspace_and_the_same_bits_every_time():
    """Whatever the workspace holds; on another stream; twice at once on two streams; replayed."""
    T, D, V = 300, 136, 700
    i = _inputs(T, D, V, "bf16", seed=13)
    i["t_idx"], i["t_logit"] = _entries(T, V, 9, seed=2)
    c = {k: v.cuda() for k, v in i.items()}
    n = max(head.ssm_head_workspace_size(T, D, V, entries=9, grads=n) for n in (0, 3))

    def once(stream=None, ws=None):
        a = head.ssm_head_ce_fwd(c["h"], c["w"], c["target"], stream=stream, ws=ws)
        g = head.ssm_head_ce_bwd(c["h"], c["w"], c["target"], a.lse, c["d_loss"], stream=stream, ws=ws)
        b = head.ssm_head_distill_fwd(c["h"], c["w"], c["t_idx"], c["t_logit"], 2.0, stream=stream, ws=ws)
        k = head.ssm_head_distill_bwd(c["h"], c["w"], c["t_idx"], c["t_logit"], b.lse, c["d_loss"], 2.0,
                                      stream=stream, ws=ws)
        return [*a, *g.values(), *b, *k.values()]

    first = once()
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for p, q in zip(first, once(ws=ws)):
            assert torch.equal(p, q)
    torch.cuda.synchronize()
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    both = [once(stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    for again in both:
        for p, q in zip(first, again):
            assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    graph.replay()
    for p, q in zip(first, held):
        assert torch.equal(p, q)
    # other rows count, other targets: the number of rows is the device's to know
    c["target"].copy_(torch.where(torch.arange(T).cuda() % 3 == 0, c["target"].clamp(min=0), -100))
    c["h"].copy_(c["h"].flip(0))
    graph.replay()
    for p, q in zip(once(), held):
        assert torch.equal(p, q)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("ignored", [0.0, 0.35, 0.9])
@pytest.mark.parametrize("T,D,V", [(333, 256, 5003), (600, 40, 9900), (1021, 64, 9985), (250, 130, 14500)])
def test_as_many_tiles_as_a_few_rounds(T, D, V, ignored, io):
    """The width of a tile then goes by the rows that count; tiles may go past the end of a piece."""
    i = _inputs(T, D, V, io, seed=T + V, ignored=ignored)
    _check(*_ce(i), i, _ce_rows(i))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 4, 8])
def test_a_few_rows_read_nothing_that_a_call_before_left(T, io):
    """Whatever the workspace holds, call after call on other targets; with two calls at once; replayed."""
    D, V = 16, 5003
    i = _inputs(T, D, V, io, seed=31, ignored=0.0)
    i["t_idx"], i["t_logit"] = _entries(T, V, 4, seed=8)
    c = {k: v.cuda() for k, v in i.items()}
    kind = binding.SSM_BF16 if io == "bf16" else binding.SSM_F32
    n = max(head.ssm_head_workspace_size(T, D, V, io=kind, entries=4, grads=n) for n in (0, 1, 2, 3))

    def once(target, ws=None, stream=None):
        how = dict(ws=ws, stream=stream)
        a = head.ssm_head_ce_fwd(c["h"], c["w"], target, **how)
        g = head.ssm_head_ce_bwd(c["h"], c["w"], target, a.lse, c["d_loss"], **how)
        b = head.ssm_head_distill_fwd(c["h"], c["w"], c["t_idx"], c["t_logit"], 2.0, **how)
        k = head.ssm_head_distill_bwd(c["h"], c["w"], c["t_idx"], c["t_logit"], b.lse, c["d_loss"], 2.0,
                                      **how)
        return [*a, *g.values(), *b, *k.values()]

    g = torch.Generator().manual_seed(5)
    targets = [torch.randint(V, (T,), generator=g).cuda() for _ in range(12)]
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    first = []
    for y in targets:
        want = torch.softmax(c["h"].double() @ c["w"].double().T, -1)
        want[torch.arange(T), y] -= 1
        want = (want * c["d_loss"].double()[:, None]).T @ c["h"].double()
        got = once(y, ws)
        # Every word of d_W: a row of it is at most sqrt(T) of all rows' d_loss h, which G and the result,
        # each rounded to bf16 at most, leave within 2 x 2^-8 sqrt(8) = 2^-5.5.
        off = (got[3].double() - want).norm(dim=1) / (c["d_loss"][:, None] * c["h"]).double().norm()
        assert off.max().item() < 2 ** -5.4
        first.append(got)
    for fill in (0, 255, 127):
        for y, want in zip(targets, first):
            ws.fill_(fill)
            for p, q in zip(want, once(y, ws)):
                assert torch.equal(p, q)
    torch.cuda.synchronize()
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    both = [once(y, stream=s) for y in targets for s in sides]
    torch.cuda.synchronize()
    for j, again in enumerate(both):
        for p, q in zip(first[j // 2], again):
            assert torch.equal(p, q)
    y = targets[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once(y)
    for other, want in zip(targets, first):
        y.copy_(other)
        graph.replay()
        for p, q in zip(want, held):
            assert torch.equal(p, q)


@pytest.mark.parametrize("io,T,V", [("bf16", 16384, 20000), ("f32", 8192, 12000)])
def test_a_vocabulary_in_several_pieces(io, T, V):
    """More of G than is kept at a time; in 64 bits on the GPU."""
    D = 40
    i = _inputs(T, D, V, io, seed=14, ignored=0.1)
    a, g = _ce(i)
    h, w, y, up = i["h"].cuda().to(f64), i["w"].cuda().to(f64), i["target"].cuda(), i["d_loss"].cuda()
    some = y != -100
    d_h, d_w = torch.zeros_like(h), torch.zeros_like(w)
    size_h, size_w = torch.zeros_like(h), torch.zeros_like(w)
    for t in range(0, T, 1024):
        s = slice(t, t + 1024)
        z = h[s] @ w.t()
        lse = torch.logsumexp(z, 1)
        loss = torch.where(some[s], lse - z.gather(1, y[s].clamp(min=0)[:, None])[:, 0], 0 * lse)
        # logits below 20, 40 products each: 1e-4 is 2^-23 (40 / 16 + 4) sum |h w| several times over
        assert float((a.loss[s].to(f64) - loss).abs().max()) < 1e-4
        G = torch.softmax(z, 1)
        G[torch.arange(G.shape[0]).cuda(), y[s].clamp(min=0)] -= 1.0
        G *= (up[s] * some[s])[:, None]
        d_h[s], size_h[s] = G @ w, G.abs() @ w.abs()
        d_w += G.t() @ h[s]
        size_w += G.abs().t() @ h[s].abs()
    # G to bf16 (2^-8) or fp32 with logits good to 1e-4 and sums over 20000 words (2^-12 of them at worst)
    share = 2.0 ** -8 + 1e-3 if io == "bf16" else 1e-3
    for name, got, want, size in (("d_h", g["d_h"], d_h, size_h), ("d_w", g["d_w"], d_w, size_w)):
        within(name, got, want.cpu(), (share * size).cpu())


def test_a_vocabulary_past_32_bit_offsets():
    V, D, T = 2_200_000, 1024, 3  # 2.25e9 elements of w
    g = torch.Generator(device="cuda").manual_seed(15)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(0, D ** -0.5, generator=g)
    h = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    y = torch.tensor([V - 1, 7, V - 300]).cuda()
    a = head.ssm_head_ce_fwd(h, w, y)
    z = torch.cat([h.to(f64) @ w[v:v + 200_000].to(f64).t() for v in range(0, V, 200_000)], 1)
    lse = torch.logsumexp(z, 1)
    assert float((a.lse - lse).abs().max()) < 1e-4 and \
        float((a.loss - (lse - z.gather(1, y[:, None])[:, 0])).abs().max()) < 1e-4
    got = head.ssm_head_ce_bwd(h, w, y, a.lse, torch.ones(T, device="cuda"))
    G = torch.softmax(z, 1)
    G[torch.arange(T).cuda(), y] -= 1.0
    last = slice(V - 5, V)
    want, size = G[:, last].t() @ h.to(f64), G[:, last].abs().t() @ h.to(f64).abs()
    within("d_w", got["d_w"][last], want.cpu(), 2.0 ** -7 * size.cpu())
    d_h, size = torch.zeros(T, D, dtype=f64, device="cuda"), torch.zeros(T, D, dtype=f64, device="cuda")
    for v in range(0, V, 200_000):
        part = w[v:v + 200_000].to(f64)
        d_h += G[:, v:v + 200_000] @ part
        size += G[:, v:v + 200_000].abs() @ part.abs()
    within("d_h", got["d_h"], d_h.cpu(), 2.0 ** -7 * size.cpu())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_long_sums_of_one_sign(io):
    """Truncation shows where every term has the same sign: 4096 columns of equal products, the sums over
    2000 rows of the weights' gradient."""
    T, D, V = 2000, 4096, 64
    h = torch.full((T, D), 0.75, dtype=DT[io])
    w = torch.full((V, D), 1.0 / 512, dtype=DT[io])
    w[:, 0] += torch.arange(V).to(DT[io]) / 64
    i = dict(h=h, w=w, target=torch.zeros(T, dtype=torch.long), d_loss=torch.full((T,), 1.0 / T))
    _check(*_ce(i), i, _ce_rows(i))


TIMEOUT = [(40, 64, 300), (700, 200, 5000)]


@pytest.mark.parametrize("T,D,V", TIMEOUT)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_call_that_gives_up_reports_timeout_and_leaves_the_context_usable(T, D, V, io):
    i = _inputs(T, D, V, io, seed=16, ignored=0.2)
    h, w, y, up = i["h"].cuda(), i["w"].cuda(), i["target"].cuda(), i["d_loss"].cuda()
    ws = torch.empty(max(head.ssm_head_workspace_size(T, D, V, block._IO[DT[io]], grads=n) for n in (0, 3)),
                     dtype=torch.uint8, device="cuda")
    t0 = time.time()
    a = head.ssm_head_ce_fwd(h, w, y, ws=ws, debug_flags=binding.SSM_DEBUG_NO_WAIT)
    assert binding.ssm_scan_status(ws) == binding.SSM_ERR_TIMEOUT
    assert bool(torch.isnan(a.loss).all()) and bool(torch.isnan(a.lse).all())
    a = head.ssm_head_ce_fwd(h, w, y, ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_OK
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, up, ws=ws, debug_flags=binding.SSM_DEBUG_NO_WAIT)
    assert binding.ssm_scan_status(ws) == binding.SSM_ERR_TIMEOUT
    assert bool(torch.isnan(g["d_h"]).all()) and bool(torch.isnan(g["d_w"]).all())
    assert time.time() - t0 < 20.0
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, up, ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_OK
    _check(a, g, i, _ce_rows(i))


def test_shapes_and_workspaces():
    h, w = torch.randn(2, 3, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    y = torch.randint(50, (2, 3), device="cuda")
    a = head.ssm_head_ce_fwd(h, w, y)
    g = head.ssm_head_ce_bwd(h, w, y, a.lse, torch.ones_like(a.loss))
    assert a.loss.shape == (2, 3) and g["d_h"].shape == h.shape and g["d_w"].shape == w.shape
    one = head.ssm_head_ce_fwd(h[0, 0], w, y[0, 0])  # a single row without a batch
    assert one.loss.shape == () and torch.equal(one.loss, head.ssm_head_ce_fwd(h[0, :1], w, y[0, :1]).loss[0])
    for bad, match in ((lambda: head.ssm_head_ce_fwd(h, w[:, :63], y), "w must have shape"),
                       (lambda: head.ssm_head_ce_fwd(h, w.bfloat16(), y), "w must be"),
                       (lambda: head.ssm_head_ce_fwd(h, w, y[:1]), "target must be"),
                       (lambda: head.ssm_head_ce_fwd(h, w, y.int()), "target must be int64"),
                       (lambda: head.ssm_head_ce_fwd(h, w, y.t()), "target must be"),
                       (lambda: head.ssm_head_ce_bwd(h, w, y, a.lse[:1], a.loss), "lse must be"),
                       (lambda: head.ssm_head_ce_bwd(h, w, y, a.lse, a.loss.double()), "d_loss must be"),
                       (lambda: head.ssm_head_distill_fwd(h, w, y, a.loss), "t_idx must be"),
                       (lambda: head.ssm_head_distill_fwd(h, w, y[..., None], a.loss), "t_logit must be"),
                       (lambda: head.ssm_head_ce_bwd(h, w, y, a.lse, a.loss, out=dict(
                           d_h=h, d_w=torch.empty(64, 50, device="cuda").t())), "d_w"),
                       (lambda: head.ssm_head_ce_fwd(h, w, y, ws=torch.empty(256, dtype=torch.uint8,
                                                                            device="cuda")), "workspace")):
        with pytest.raises((ValueError, TypeError), match=match):
            bad()
    for bad in (lambda: head.ssm_head_ce_fwd(h[:0], w, y[:0]), lambda: head.ssm_head_ce_fwd(h, w[:0], y),
                lambda: head.ssm_head_distill_fwd(h, w, y[..., None], a.loss[..., None], temperature=0.0),
                lambda: head.ssm_head_ce_bwd(h, w, y, a.lse, a.loss, want_dh=False, want_dw=False)):
        with pytest.raises(SsmError):
            bad()
