"""The layer norm, the head and their losses run together as the example's language model uses them: the
head's gradients against 64-bit autograd, scores token by token against the sequence, a step that is
captured and replayed."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import mamba_block  # noqa: E402

pytestmark = pytest.mark.gpu
f64 = torch.float64
SHAPE = mamba_block.Shape(d_model=40, n_head=3, head_dim=16, d_state=8, group=16, chunk=16)


def _relative(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def _head_inputs(io, n=3, L=29, vocab=300, k=7):
    g = torch.Generator().manual_seed(5)
    h = torch.randn(n, L, SHAPE.d_model, generator=g).to(io)
    r = torch.randn(n, L, SHAPE.d_model, generator=g)
    target = torch.randint(vocab, (n, L), generator=g)
    target[:, -1] = -100
    t_idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(n * L)]).view(n, L, k)
    t_idx[0, 3] = -1
    t_logit = 2 * torch.randn(n, L, k, generator=g)
    d_loss = torch.randn(n, L, generator=g)
    return h, r, target, (t_idx, t_logit), d_loss


@pytest.mark.parametrize("io,tol", [(torch.float32, 1e-5), (torch.bfloat16, 2e-2)])
@pytest.mark.parametrize("distil", [False, True])
def test_head_gradients_against_64_bit_autograd(io, tol, distil):
    """Tolerances in the 2-norm: fp32, 50 operations of 2^-24 each that all go one way; bf16, the norm's
    output, G and each result rounded once (3 x 2^-8), and the logits of a rounded norm."""
    h, r, target, teacher, d_loss = _head_inputs(io)
    head = mamba_block.Head(SHAPE.d_model, 300, seed=2, io=io)
    head.p["w"] += 0.1 * torch.arange(SHAPE.d_model, device="cuda") / SHAPE.d_model
    head.p["b"] += 0.2
    p = {k: v.cpu().to(f64).requires_grad_() for k, v in head.p.items()}
    with torch.no_grad():
        p["W"].copy_(p["W"].to(io))  # the head multiplies what its type holds
    h64, r64 = h.to(f64).requires_grad_(), r.to(f64).requires_grad_()
    s = h64 + r64
    u = torch.nn.functional.layer_norm(s, (SHAPE.d_model,), p["w"], p["b"], 1e-5)
    z = u @ p["W"].t()
    if distil:
        t_idx, t_logit = teacher
        some = t_idx[..., 0] >= 0
        pt = torch.softmax(t_logit.to(f64) / 2.0, -1)
        log_q = torch.log_softmax(z / 2.0, -1).gather(-1, t_idx.clamp(min=0))
        want = torch.where(some, 4.0 * (pt * (pt.log() - log_q)).sum(-1), torch.zeros((), dtype=f64))
        how = dict(teacher=(t_idx.cuda(), t_logit.cuda()), temperature=2.0)
    else:
        want = torch.nn.functional.cross_entropy(z.flatten(0, 1), target.flatten(), reduction="none")
        want, how = want.view(target.shape), {}
    (want * d_loss).sum().backward()
    loss, kept = head.forward(h.cuda(), r.cuda(), target.cuda(), **how)
    d_h, d_r, grads = head.backward(d_loss.cuda(), kept)
    assert _relative(loss, want.detach()) < tol
    for got, leaf in ((d_h, h64), (d_r, r64)) + tuple((grads[n], p[n]) for n in ("w", "b", "W")):
        assert _relative(got, leaf.grad) < tol


def test_scores_token_by_token_are_those_of_the_sequence():
    """fp32: the forms of the scan, conv and head for single tokens against those for sequences."""
    blocks = [mamba_block.Block(SHAPE, seed=i, io=torch.float32) for i in range(2)]
    head = mamba_block.Head(SHAPE.d_model, 300, seed=4, io=torch.float32)
    for n in (1, 3):
        tokens = torch.randint(300, (n, 21), generator=torch.Generator().manual_seed(n)).cuda()
        x, stream = head.embed(tokens), None
        for b in blocks:
            x, stream, _ = b.forward(x, stream, save8=False)
        target = torch.full_like(tokens, -100)
        target[:, :-1] = tokens[:, 1:]
        loss, _ = head.forward(x, stream, target)
        assert bool((loss[:, -1] == 0).all())
        got = mamba_block.score(blocks, head, tokens)
        assert _relative(-got, loss[:, :-1].cpu().double()) < 1e-4


@pytest.mark.parametrize("distil", [False, True])
def test_a_language_model_step_runs_and_moves_every_parameter(distil):
    blocks = [mamba_block.Block(SHAPE, seed=i) for i in range(2)]
    head = mamba_block.Head(SHAPE.d_model, 300, seed=4)
    tokens = torch.randint(300, (3, 29), generator=torch.Generator().manual_seed(1)).cuda()
    how = {}
    if distil:
        t_idx, t_logit = _head_inputs(torch.bfloat16)[3]
        how = dict(teacher=(t_idx.cuda(), t_logit.cuda()), temperature=2.0)
    before = {n: v.clone() for n, v in head.p.items()}
    loss = mamba_block.lm_step(blocks, head, tokens, lr=0.1, **how)
    assert loss == loss and abs(loss) < 100
    for n, v in head.p.items():
        assert bool(torch.isfinite(v).all()) and not torch.equal(v, before[n]), n


def test_forward_and_backward_captured_together_replay_the_same_bits():
    h, r, target, teacher, d_loss = (t.cuda() if torch.is_tensor(t) else tuple(x.cuda() for x in t)
                                     for t in _head_inputs(torch.bfloat16))
    head = mamba_block.Head(SHAPE.d_model, 300, seed=2)

    def once():
        out = []
        for how in ({}, dict(teacher=teacher, temperature=2.0)):
            loss, kept = head.forward(h, r, target, **how)
            d_h, d_r, g = head.backward(d_loss, kept)
            out += [loss, d_h, d_r, *g.values()]
        return out

    want = [t.clone() for t in once()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for t in held:
        t.zero_()
    graph.replay()
    for p, q in zip(want, held):
        assert torch.equal(p, q)
