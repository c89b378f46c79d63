"""Calls on a stream other than the current one: where their results and workspaces come from, with
work pending on either stream.

A tensor freed with work pending on its stream may be handed out again at once on that stream, which
orders the next user after that work; a call on another stream is not ordered after it, so nothing that
it writes may lie there."""
import gc
from types import SimpleNamespace

import pytest
import torch

from bwd_ssm_conv_gb300 import binding, block

pytestmark = pytest.mark.gpu
ROWS, COLS = 1024, 2048  # results of 1 MiB and more: blocks of their own size in the allocator
BUSY = 20_000_000        # cycles that the current stream is kept busy: about 10 ms


def _rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _tensors(r):
    """The CUDA tensors in a call's result."""
    if torch.is_tensor(r):
        return [r]
    if isinstance(r, dict):
        r = tuple(r.values())
    return [t for v in r for t in _tensors(v)] if isinstance(r, tuple) else []


def _block_calls():
    x, y, z = (_rand(i, ROWS, COLS) for i in range(3))
    w = _rand(3, COLS)
    a = block.ssm_add_norm_fwd(x, w, y, w, save8=True, save_x8=True)
    b = block.ssm_gated_norm_fwd(y, z, w, save8=True, save_out8=True)
    return {
        "add_norm_fwd": lambda **k: block.ssm_add_norm_fwd(x, w, y, w, save8=True, save_x8=True,
                                                           save_out8=True, **k),
        "add_norm_bwd": lambda **k: block.ssm_add_norm_bwd(x, a.res8, a.rstd, w, d_res_out=y, scale=w,
                                                           x=a.x8, **k),
        "gated_norm_fwd": lambda **k: block.ssm_gated_norm_fwd(y, z, w, save8=True, save_out8=True, **k),
        "gated_norm_bwd": lambda **k: block.ssm_gated_norm_bwd(x, b.y8, b.z8, b.rstd, w, **k),
        "ckpt8_save": lambda **k: block.ssm_ckpt8_save(x, **k),
        "ckpt8_load": lambda **k: block.ssm_ckpt8_load(b.y8, torch.float32, **k),
        "ckpt8_wgrad": lambda **k: block.ssm_ckpt8_wgrad(x, b.out8, **k),
    }


def _scan_calls():
    n, L, d, N, K = 2, 512, 512, 16, 4
    sx = _rand(10, n, d, K - 1 + L)
    c, bias = _rand(11, d, K), _rand(12, d)
    x, z, dy = (_rand(13 + i, n, L, d, 1) for i in range(3))
    dt = 0.1 * _rand(16, n, L, d).abs()
    A, D = -_rand(17, d, N).abs() - 0.1, _rand(18, d)
    B, C = (_rand(19 + i, n, L, 1, N) for i in range(2))
    how = dict(D=D, z=z, chunk=64)
    ckpt = binding.ssm_scan_fwd(x, dt, A, B, C, **how)[2]
    fused = binding.ssm_conv_scan_fwd(sx, c, dt, A, B, C, bias=bias, **how)[2]
    dout = dy.view(n, L, d)
    tok = dict(x_new=_rand(21, 512, d, 1), c=c, dt=0.1 * _rand(22, 512, d).abs(), A=A,
               B=_rand(23, 512, 1, N), C=_rand(24, 512, 1, N), D=D)

    # decode's states are updated in place: fresh ones for every call of the tests, made beforehand
    states = iter([(torch.zeros(512, d, K - 1, device="cuda"), torch.zeros(512, d, 1, N, device="cuda"))
                   for _ in range(7)])

    def decode(**k):
        conv, state = next(states)
        return binding.ssm_decode_step(conv_state=conv, state=state, **tok, **k)

    def plain(f):  # without the workspace, which holds nothing defined
        return lambda **k: {n: t for n, t in f(**k).items() if n != "_ws" and t is not None}

    return {
        "conv_fwd": lambda **k: binding.ssm_conv_fwd(sx, c, bias, want_state=True, **k),
        "conv_bwd": lambda **k: binding.ssm_conv_bwd(sx, c, dout, bias, **k),
        "scan_fwd": lambda **k: binding.ssm_scan_fwd(x, dt, A, B, C, **how, **k),
        "scan_bwd": plain(lambda **k: binding.ssm_scan_bwd(x, dt, A, B, C, dy, ckpt=ckpt, **how, **k)),
        "conv_scan_fwd": lambda **k: binding.ssm_conv_scan_fwd(sx, c, dt, A, B, C, bias=bias, **how,
                                                               **k),
        "conv_scan_bwd": plain(lambda **k: binding.ssm_conv_scan_bwd(
            sx, c, dt, A, B, C, dy, bias=bias, ckpt=fused, **how, **k)),
        "decode_step": decode,
    }


BLOCK = ("add_norm_fwd", "add_norm_bwd", "gated_norm_fwd", "gated_norm_bwd", "ckpt8_save",
         "ckpt8_load", "ckpt8_wgrad")
SCAN = ("conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "conv_scan_fwd", "conv_scan_bwd", "decode_step")
CALLS = [("block", n) for n in BLOCK] + [("scan", n) for n in SCAN]


@pytest.fixture(scope="module")
def calls():
    c = {"block": _block_calls(), "scan": _scan_calls()}
    torch.cuda.synchronize()
    return c


def _temporaries(like):
    """Tensors as large as those in ``like``, the only ones whose blocks become free when dropped."""
    gc.collect()
    torch.cuda.empty_cache()
    return [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda")
            for t in like]


def _spans(ts):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in ts]


@pytest.mark.parametrize("kind,name", CALLS)
def test_results_lie_in_no_memory_freed_on_the_current_stream(calls, kind, name):
    call, side = calls[kind][name], torch.cuda.Stream()
    want = _tensors(call())
    temps = _temporaries(want)
    torch.cuda.synchronize()
    freed = _spans(temps)
    del temps
    got = _tensors(call(stream=side))
    torch.cuda.synchronize()
    for a, b in _spans(got):
        assert not any(a < y and x < b for x, y in freed)
    for p, q in zip(want, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("kind,name", CALLS)
def test_a_call_leaves_memory_with_pending_readers_alone(calls, kind, name):
    """The current stream still has to read temporaries that were dropped; results and workspace of a
    call on another stream go elsewhere.  Twice as many temporaries as results, for the workspaces."""
    call, side = calls[kind][name], torch.cuda.Stream()
    want = [t.clone() for t in _tensors(call())]
    temps = _temporaries(want + want)
    copies = [torch.zeros_like(t) for t in temps]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t, c in zip(temps, copies):
        c.copy_(t)
    del temps, t
    got = _tensors(call(stream=side))
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    for p, q in zip(want, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("kind,name", CALLS)
def test_results_freed_with_readers_pending_on_the_current_stream(calls, kind, name):
    """Results of a call on another stream, read on the current one and dropped: that stream's next
    call does not write over them before they have been read."""
    call, side = calls[kind][name], torch.cuda.Stream()
    want = [t.clone() for t in _tensors(call())]
    copies = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    got = _tensors(call(stream=side))
    spans = _spans(got)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    for t, c in zip(got, copies):
        c.copy_(t)
    del got, t
    again = _tensors(call(stream=side))
    assert not any(a < y and x < b for a, b in _spans(again) for x, y in spans)
    torch.cuda.synchronize()
    for p, q in zip(want, copies):
        assert torch.equal(p, q)


@pytest.mark.parametrize("name", BLOCK)
def test_a_stream_of_another_gpu_is_refused(calls, name):
    """Found on the host, before anything is allocated or enqueued."""
    other = SimpleNamespace(cuda_stream=0, stream_id=0, device_type=1,
                            device_index=torch.cuda.current_device() + 1)
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="stream must be one of cuda"):
        calls["block"][name](stream=other)
    assert torch.cuda.memory_allocated() == before
