"""The layer norm and the head on a stream other than the current one: where their results and workspaces
come from, with work pending on either stream (test_gpu_streams says why)."""
import gc
from types import SimpleNamespace

import pytest
import torch

from bwd_ssm_conv_gb300 import block, head
from test_gpu_streams import BUSY, _rand, _spans, _temporaries, _tensors

pytestmark = pytest.mark.gpu
ROWS, COLS, VOCAB = 1024, 1024, 1500
CALLS = ("add_layer_norm_fwd", "add_layer_norm_bwd", "ce_fwd", "ce_bwd", "distill_fwd", "distill_bwd",
         "ce_fwd_few")


@pytest.fixture(scope="module")
def calls():
    x, y = _rand(0, ROWS, COLS), _rand(1, ROWS, COLS)
    w, W = _rand(2, COLS), 0.03 * _rand(3, VOCAB, COLS)
    a = block.ssm_add_layer_norm_fwd(x, w, w, y, w, save8=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    t = torch.randint(VOCAB, (ROWS,), generator=g, device="cuda")
    t[::5] = -100
    e = torch.randint(VOCAB, (ROWS, 9), generator=g, device="cuda"), _rand(5, ROWS, 9)
    up = _rand(6, ROWS)
    ce = head.ssm_head_ce_fwd(x, W, t)
    kd = head.ssm_head_distill_fwd(x, W, *e)
    c = {
        "add_layer_norm_fwd": lambda **k: block.ssm_add_layer_norm_fwd(x, w, w, y, w, save8=True,
                                                                       save_out8=True, **k),
        "add_layer_norm_bwd": lambda **k: block.ssm_add_layer_norm_bwd(
            x, a.res8, a.mean, a.rstd, w, d_res_out=y, scale=w, x=x, **k),
        "ce_fwd": lambda **k: head.ssm_head_ce_fwd(x, W, t, **k),
        "ce_bwd": lambda **k: head.ssm_head_ce_bwd(x, W, t, ce.lse, up, **k),
        "distill_fwd": lambda **k: head.ssm_head_distill_fwd(x, W, *e, **k),
        "distill_bwd": lambda **k: head.ssm_head_distill_bwd(x, W, *e, kd.lse, up, **k),
        "ce_fwd_few": lambda **k: head.ssm_head_ce_fwd(x[1:2], W, t[1:2], **k),
    }
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("name", CALLS)
def test_results_lie_in_no_memory_freed_on_the_current_stream(calls, name):
    call, side = calls[name], torch.cuda.Stream()
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


@pytest.mark.parametrize("name", CALLS)
def test_a_call_leaves_memory_with_pending_readers_alone(calls, name):
    call, side = calls[name], torch.cuda.Stream()
    want = [t.clone() for t in _tensors(call())]
    temps = _temporaries(want + want)
    # and as large as any of the workspaces, which is where most of a call's writes go
    temps.append(torch.full((1 << 26,), 7, dtype=torch.uint8, device="cuda"))
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


@pytest.mark.parametrize("name", CALLS)
def test_results_freed_with_readers_pending_on_the_current_stream(calls, name):
    call, side = calls[name], torch.cuda.Stream()
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


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_gpu_is_refused(calls, name):
    other = SimpleNamespace(cuda_stream=0, stream_id=0, device_type=1,
                            device_index=torch.cuda.current_device() + 1)
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="stream must be one of cuda"):
        calls[name](stream=other)
    assert torch.cuda.memory_allocated() == before


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_freed_with_its_results(calls, name):
    calls[name]()
    gc.collect()
    before = torch.cuda.memory_allocated()
    kept = calls[name]()
    assert torch.cuda.memory_allocated() > before
    del kept
    for _ in range(5):
        calls[name]()
    assert torch.cuda.memory_allocated() == before
