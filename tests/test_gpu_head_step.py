"""The example's language model as a whole: one step of it against 64-bit autograd of the same model, and what
embedding and scoring copy."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_gpu_block_example import SHAPE, _reference, mamba_block

pytestmark = pytest.mark.gpu
f64 = torch.float64
VOCAB = 300


def _tokens(n, L, seed=1):
    return torch.randint(VOCAB, (n, L), generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("distil", [False, True])
def test_a_step_moves_every_parameter_by_its_gradient(distil):
    """The blocks', the norm's and the head's, with the embedding's part.  fp32, the difference of a parameter
    before and after over its gradient's size: 1e-4 for each of the two blocks and the head (sums of a few
    hundred terms through six stages), and 2^-24 of a parameter of 1 where its gradient is 1e-3."""
    blocks = [mamba_block.Block(SHAPE, seed=i, io=torch.float32) for i in range(2)]
    head = mamba_block.Head(SHAPE.d_model, VOCAB, seed=4, io=torch.float32)
    head.p["b"] += 0.1
    tokens = _tokens(3, 29)
    g = torch.Generator().manual_seed(2)
    t_idx = torch.stack([torch.randperm(VOCAB, generator=g)[:7] for _ in range(3 * 29)]).view(3, 29, 7)
    t_idx[0, 3] = -1
    t_logit, tau = 2 * torch.randn(3, 29, 7, generator=g), 2.0
    leaves = [{k: v.cpu().to(f64).requires_grad_() for k, v in m.p.items()} for m in (*blocks, head)]
    x = leaves[-1]["W"][tokens]
    stream = torch.zeros_like(x)
    for p in leaves[:-1]:
        x, stream = _reference(SHAPE, p, x, stream)
    p = leaves[-1]
    z = torch.nn.functional.layer_norm(stream + x, (SHAPE.d_model,), p["w"], p["b"], 1e-5) @ p["W"].t()
    if distil:
        pt = torch.softmax(t_logit.to(f64) / tau, -1)
        log_q = torch.log_softmax(z / tau, -1).gather(-1, t_idx.clamp(min=0))
        want = ((pt * (pt.log() - log_q)).sum(-1) * (t_idx[..., 0] >= 0)).mean() * tau ** 2
        how = dict(teacher=(t_idx.cuda(), t_logit.cuda()), temperature=tau)
    else:
        want = torch.nn.functional.cross_entropy(z[:, :-1].flatten(0, 1), tokens[:, 1:].flatten())
        how = {}
    want.backward()
    want = float(want.detach())
    before = [{k: v.clone() for k, v in m.p.items()} for m in (*blocks, head)]
    loss = mamba_block.lm_step(blocks, head, tokens.cuda(), save8=False, lr=1.0, **how)
    assert abs(loss - want) < 1e-5 * abs(want)
    for i, (m, was, leaf) in enumerate(zip((*blocks, head), before, leaves)):
        for n, v in m.p.items():
            moved = (was[n].to(f64) - v.to(f64)).cpu()
            assert float((moved - leaf[n].grad).norm() / leaf[n].grad.norm()) < 5e-4, (i, n)


class _Copies(TorchDispatchMode):
    """How many operations read or write a whole tensor of ``numel`` elements to make another of another type."""

    def __init__(self, numel):
        super().__init__()
        self.numel, self.n = numel, 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten._to_copy.default and args[0].numel() == self.numel:
            self.n += 1
        return out


def test_embedding_and_scoring_do_not_copy_the_weights_for_every_token():
    blocks = [mamba_block.Block(SHAPE, seed=0)]
    head = mamba_block.Head(SHAPE.d_model, VOCAB, seed=4)
    tokens = _tokens(2, 9).cuda()
    assert torch.equal(head.embed(tokens), head.p["W"].to(head.io)[tokens])
    with _Copies(head.p["W"].numel()) as copies:
        head.embed(tokens)
    assert copies.n == 0
    with _Copies(head.p["W"].numel()) as copies:
        mamba_block.score(blocks, head, tokens)
    assert copies.n == 1


@pytest.mark.parametrize("save8", [False, True])
def test_sequences_of_one_token(save8):
    """They have no next token: no scores, no loss, and nothing moves."""
    blocks = [mamba_block.Block(SHAPE, seed=0)]
    head = mamba_block.Head(SHAPE.d_model, VOCAB, seed=4)
    tokens = _tokens(3, 1).cuda()
    scores = mamba_block.score(blocks, head, tokens)
    assert scores.shape == (3, 0) and scores.dtype == torch.float32 and scores.is_cuda
    before = [{k: v.clone() for k, v in m.p.items()} for m in (*blocks, head)]
    assert mamba_block.lm_step(blocks, head, tokens, save8=save8, lr=1.0) == 0.0
    for m, was in zip((*blocks, head), before):
        for n, v in m.p.items():
            assert torch.equal(v, was[n]), n
