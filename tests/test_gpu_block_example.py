"""The example block: its gradients against 64-bit autograd of the same block, its 8-bit
checkpoints against keeping activations whole, and token-by-token decoding against the sequence."""
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


def _reference(shape, p, h, residual):
    """The block in 64 bits, a loop over tokens."""
    s = residual + h
    u = p["w1"] * s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5)
    z, x, B, C, dt = (u @ p["W_in"].t()).split(shape.widths, dim=-1)
    n, L, _ = x.shape
    K = shape.d_conv
    xp = torch.cat([x.new_zeros(n, K - 1, x.shape[-1]), x], dim=1)
    x = sum(xp[:, k:k + L] * p["c"][:, k] for k in range(K))
    x = x * torch.sigmoid(x)
    dt = torch.nn.functional.softplus(dt + p["dt_bias"])
    x4 = x.view(n, L, shape.n_head, shape.head_dim)
    state = x.new_zeros(n, shape.n_head, shape.head_dim, shape.d_state)
    ys = []
    for t in range(L):
        a = torch.exp(dt[:, t] * p["A"])[:, :, None, None]
        state = a * state + (dt[:, t, :, None] * x4[:, t])[..., None] * B[:, t, None, None, :]
        ys.append((state * C[:, t, None, None, :]).sum(-1))
    y = torch.stack(ys, 1).reshape(n, L, -1) + p["D"] * x
    v = y * z * torch.sigmoid(z)
    vg = v.view(n, L, -1, shape.group)
    vg = vg * torch.rsqrt((vg * vg).mean(-1, keepdim=True) + 1e-5)
    return (p["w2"] * vg.reshape(n, L, -1)) @ p["W_out"].t(), s


def _inputs():
    g = torch.Generator().manual_seed(3)
    return [torch.randn(2, 37, SHAPE.d_model, generator=g) for _ in range(4)]


def _relative(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def test_block_gradients_against_64_bit_autograd():
    block = mamba_block.Block(SHAPE, seed=1, io=torch.float32)
    h, r, d_out, d_stream = _inputs()
    p64 = {k: v.cpu().double().requires_grad_() for k, v in block.p.items()}
    h64, r64 = h.double().requires_grad_(), r.double().requires_grad_()
    out64, s64 = _reference(SHAPE, p64, h64, r64)
    ((out64 * d_out.double()).sum() + (s64 * d_stream.double()).sum()).backward()
    # 1e-4: fp32 sums of a few hundred terms through six stages
    out, stream, kept = block.forward(h.cuda(), r.cuda(), save8=False)
    assert _relative(out, out64.detach()) < 1e-4 and _relative(stream, s64.detach()) < 1e-6
    d_h, d_r, g = block.backward(d_out.cuda(), d_stream.cuda(), kept)
    assert _relative(d_h, h64.grad) < 1e-4 and _relative(d_r, r64.grad) < 1e-4
    for name, v in g.items():
        assert _relative(v, p64[name].grad) < 1e-4, name


def test_block_backward_from_checkpoints_is_that_of_the_values_they_hold():
    """The same backward from the checkpoints and from tensors with their values: the same formulas
    on the same numbers, so they agree to the rounding of fp32 sums, 1e-5."""
    block = mamba_block.Block(SHAPE, seed=1, io=torch.float32)
    h, r, d_out, d_stream = _inputs()
    out, stream, kept = block.forward(h.cuda(), r.cuda(), save8=True)
    same, stream_w, whole = block.forward(h.cuda(), r.cuda(), save8=False)
    assert torch.equal(out, same) and torch.equal(stream, stream_w)
    loaded = dict(kept)
    for name in ("s", "u", "y", "z", "v"):
        loaded[name] = mamba_block.ssm.ssm_ckpt8_load(kept[name], torch.float32)
        # kept within half a step of the value, or a step at the block's top (1/64 of its largest)
        v = torch.nn.functional.pad(whole[name], (0, -whole[name].shape[-1] % 32))
        top = v.unflatten(-1, (-1, 32)).abs().amax(-1).repeat_interleave(32, -1)[..., :whole[name].shape[-1]]
        assert bool(((loaded[name] - whole[name]).abs() <= top / 64).all()), name
    a = block.backward(d_out.cuda(), d_stream.cuda(), kept)
    b = block.backward(d_out.cuda(), d_stream.cuda(), loaded)
    for p, q in zip(a[:2], b[:2]):
        assert _relative(p, q.cpu().double()) < 1e-5
    for name in a[2]:
        assert _relative(a[2][name], b[2][name].cpu().double()) < 1e-5, name


def test_checkpoints_keep_less_and_losses_stay():
    shape = mamba_block.Shape(d_model=256, n_head=8, head_dim=64, d_state=16)
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(2, 256, 256, generator=g, device="cuda").bfloat16()
    target = torch.randn(2, 256, 256, generator=g, device="cuda")
    runs = {}
    for save8 in (False, True):
        blocks = [mamba_block.Block(shape, seed=i) for i in range(2)]
        runs[save8] = [mamba_block.train_step(blocks, h, target, save8, lr=1e-3) for _ in range(8)]
    assert runs[True][0][1] < 0.75 * runs[False][0][1]
    for (a, _), (b, _) in zip(runs[False], runs[True]):
        assert abs(a - b) < 0.02 * a
    assert runs[True][-1][0] < 0.98 * runs[True][0][0]


def test_decoding_token_by_token_equals_the_sequence():
    block = mamba_block.Block(SHAPE, seed=2, io=torch.float32)
    h, r, _, _ = _inputs()
    out, stream, _ = block.forward(h.cuda(), r.cuda(), save8=False)
    cache = block.new_cache(2)
    for t in range(h.shape[1]):
        o, s = block.decode(h[:, t].contiguous().cuda(), r[:, t].contiguous().cuda(), cache)
        assert torch.equal(s, stream[:, t])
        assert torch.allclose(o, out[:, t], rtol=1e-4, atol=1e-4)
