"""The 64-bit references of the layer norm and of the head's losses against differences, and the C ABI's
and the binding's refusals, without a GPU."""
import math

import pytest
import torch

import head_ref as ref
from bwd_ssm_conv_gb300 import binding, block
from bwd_ssm_conv_gb300.build import build
from test_block_ref import FAKE, INV, UNS, WS, _call, _desc, _difference, _fake, _fake8

f64 = torch.float64


@pytest.fixture(scope="module")
def L():
    build()
    return block.lib()


# ---- layer norm -----------------------------------------------------------------------------------

@pytest.mark.parametrize("with_scale,with_residual", [(True, True), (False, True), (True, False)])
def test_layer_norm_gradient_is_that_of_its_forward(with_scale, with_residual):
    g = torch.Generator().manual_seed(1)
    R, C = 3, 5
    x, d_out, d_s = (torch.randn(R, C, generator=g, dtype=f64) for _ in range(3))
    w, b = (torch.randn(C, generator=g, dtype=f64) for _ in range(2))
    res = torch.randn(R, C, generator=g, dtype=f64) if with_residual else None
    scale = torch.rand(C, generator=g, dtype=f64) if with_scale else None

    def loss():
        (out, s, _, _), _ = ref.layer_norm(x, res, scale, w, b, 1e-3)
        return (out * d_out).sum() + (s * d_s).sum()

    (_, s, mean, rstd), _ = ref.layer_norm(x, res, scale, w, b, 1e-3)
    (d_res, d_x, d_w, d_b, d_scale), _ = ref.layer_norm_bwd(d_out, s, mean, rstd, d_s, scale, w, x)
    for got, v in ((d_x, x), (d_w, w), (d_b, b)) + (((d_res, res),) if with_residual else ()) + \
            (((d_scale, scale),) if with_scale else ()):
        assert torch.allclose(got, _difference(loss, v), rtol=0, atol=1e-7)


LN_FWD = ("x ld_x residual ld_residual scale w b out ld_out res_out ld_res_out mean rstd res_q res_e "
          "x_q x_e out_q out_e").split()
LN_BWD = ("d_out ld_d_out d_res_out ld_d_res_out res ld_res res_q res_e x ld_x x_q x_e mean rstd "
          "scale w d_res ld_d_res d_x ld_d_x d_w d_b d_scale").split()
NEED = ("d_out", "res", "mean", "rstd", "d_x", "d_w")


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(cols=0), INV), (dict(io=7), INV), (dict(group=32), INV),
    (dict(eps=0.0), INV), (dict(eps=math.nan), INV), (dict(flags=1), INV),
    (dict(io=0, res_io=1), INV), (dict(cols=32769), UNS), (dict(rows=1 << 40), UNS),
])
def test_layer_norm_refuses_bad_descriptors(L, kw, code):
    d = _desc(**kw)
    assert _call(L.ssm_add_layer_norm_fwd, LN_FWD, ("x", "out"), d) == code
    assert _call(L.ssm_add_layer_norm_bwd, LN_BWD, NEED, d, ws=(FAKE, 1 << 30)) == code


def test_layer_norm_refusals(L):
    def f(**over):
        return _call(L.ssm_add_layer_norm_fwd, LN_FWD, ("x", "out"), _desc(), **over)
    assert f(x=None) == INV and f(out=None) == INV
    for n in ("w", "b", "mean", "rstd", "scale"):
        assert f(**{n: FAKE + 2}) == INV, n
    assert f(ld_out=63) == INV and f(ld_x=1 << 40) == UNS and f(res_q=FAKE) == INV

    def b(ws=(FAKE, 1 << 30), **over):
        return _call(L.ssm_add_layer_norm_bwd, LN_BWD, NEED, _desc(), ws=ws, **over)
    for n in ("d_out", "res", "mean", "rstd"):
        assert b(**{n: None}) == INV, n
    assert b(d_x=None, d_w=None) == INV
    assert b(d_scale=FAKE, scale=FAKE) == INV and b(d_scale=FAKE, x=FAKE) == INV
    for n in ("mean", "rstd", "d_w", "d_b", "d_x"):
        assert b(**{n: FAKE + 2}) == INV, n
    assert b(res_q=FAKE, res_e=FAKE) == INV
    # on a machine without a GPU the workspace's size cannot be known: an error in either case
    assert b(ws=(None, 0)) != 0 and b(ws=(FAKE + 8, 1 << 30)) != 0
    assert b(ws=(None, 0)) in (WS, binding.SSM_ERR_CUDA)


def _layer_norm_calls():
    def t():
        return _fake(4, 64)

    def v():
        return _fake(64)
    ws = _fake(1 << 16, dtype=torch.uint8)
    return {
        "fwd": (lambda a: block.ssm_add_layer_norm_fwd(
            a["x"], a["w"], a["b"], a["residual"], a["scale"], out=(a["out"], a["res_out"])),
            dict(x=t(), w=v(), b=v(), residual=t(), scale=v(), out=t(), res_out=t())),
        "bwd": (lambda a: block.ssm_add_layer_norm_bwd(
            a["d_out"], a["res"], a["mean"], a["rstd"], a["w"], a["d_res_out"], a["scale"], a["x"],
            ws=a["ws"], out={n: a[n] for n in ("d_res", "d_x", "d_w", "d_scale", "d_b")}),
            dict(d_out=t(), res=t(), mean=_fake(4), rstd=_fake(4), w=v(), d_res_out=t(), scale=v(),
                 x=t(), ws=ws, d_res=t(), d_x=t(), d_w=v(), d_scale=v(), d_b=v())),
        "bwd8": (lambda a: block.ssm_add_layer_norm_bwd(
            a["d_out"], a["res"], a["mean"], a["rstd"], scale=a["scale"], x=a["x"]),
            dict(d_out=t(), res=_fake8(4, 64), mean=_fake(4), rstd=_fake(4), scale=v(),
                 x=_fake8(4, 64))),
    }


@pytest.mark.parametrize("name", list(_layer_norm_calls()))
def test_layer_norm_refuses_tensors_of_two_gpus_by_name(name):
    call, args = _layer_norm_calls()[name]
    first = next(iter(args))
    for n, t in args.items():
        other = _fake8(4, 64, 0, 1) if isinstance(t, tuple) else _fake(*t.shape, dtype=t.dtype, gpu=1)
        wrong = n if n != first else "|".join(args)
        with pytest.raises(ValueError, match=f"^({wrong}) must be a CUDA tensor on cuda"):
            call({**args, n: other})


def test_layer_norm_names_the_argument_that_is_not_a_tensor():
    t = torch.zeros(4, 64)
    for call, name in ((lambda: block.ssm_add_layer_norm_fwd(3), "x"),
                       (lambda: block.ssm_add_layer_norm_fwd(t, b=2.0), "b"),
                       (lambda: block.ssm_add_layer_norm_bwd(t, t, None, t), "mean")):
        with pytest.raises(TypeError, match=name):
            call()


# ---- the head ---------------------------------------------------------------------------------------

def test_ce_gradient_is_that_of_its_forward():
    g = torch.Generator().manual_seed(2)
    h, w = torch.randn(4, 3, generator=g, dtype=f64), torch.randn(6, 3, generator=g, dtype=f64)
    target, up = torch.tensor([2, -100, 5, 0]), torch.randn(4, generator=g, dtype=f64)
    rows = ref.ce_rows(target, 6)

    def loss():
        return (ref.head(h, w, *rows)[0][0] * up).sum()

    want = torch.nn.functional.cross_entropy(h @ w.t(), target, reduction="none")
    (l, lse), _ = ref.head(h, w, *rows)
    assert torch.allclose(l, want, rtol=0, atol=1e-12)
    (d_h, d_w), _ = ref.head_bwd(h, w, rows[0], rows[1], lse, up)
    for got, v in ((d_h, h), (d_w, w)):
        assert torch.allclose(got, _difference(loss, v), rtol=0, atol=1e-7)


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_is_that_of_its_forward(tau):
    g = torch.Generator().manual_seed(3)
    h, w = torch.randn(4, 3, generator=g, dtype=f64), torch.randn(7, 3, generator=g, dtype=f64)
    t_idx = torch.tensor([[1, 4, 2], [-1, -1, -1], [6, -1, 6], [0, 3, 5]])
    t_logit, up = torch.randn(4, 3, generator=g), torch.randn(4, generator=g, dtype=f64)
    t_logit[3, 1] = -math.inf
    rows = ref._p_of(t_idx, t_logit, tau, 7)

    def loss():
        return (ref.head(h, w, *rows, tau=tau)[0][0] * up).sum()

    (l, lse), _ = ref.head(h, w, *rows, tau=tau)
    assert float(l[1]) == 0.0 and float(lse[1]) == 0.0
    # two entries of one word: a divergence from what they are together, up to their own entropy
    p = torch.softmax(t_logit[0].double() / tau, 0)
    q = torch.log_softmax(h[0] @ w.t() / tau, 0)[t_idx[0]]
    assert math.isclose(float(l[0]), tau * tau * float((p * (p.log() - q)).sum()), abs_tol=1e-12)
    (d_h, d_w), _ = ref.head_bwd(h, w, rows[0], rows[1], lse, up, tau=tau)
    for got, v in ((d_h, h), (d_w, w)):
        assert torch.allclose(got, _difference(loss, v), rtol=0, atol=1e-7)


from bwd_ssm_conv_gb300 import head  # noqa: E402


@pytest.fixture(scope="module")
def H():
    build()
    return head.lib()


CE_FWD = "h ld_h w ld_w target loss lse".split()
CE_BWD = "h ld_h w ld_w target lse d_loss d_h ld_d_h d_w".split()
KD_FWD = "h ld_h w ld_w t_idx t_logit loss lse".split()
KD_BWD = "h ld_h w ld_w t_idx t_logit lse d_loss d_h ld_d_h d_w".split()


def _calls(H, **kw):
    """Each entry point with fake pointers: name -> call(**overrides), and the arguments it needs."""
    base = dict(rows=4, cols=64, vocab=300, io=0, entries=0, entry_io=0, temperature=1.0,
                ignore_index=-100, flags=0)
    out = {}
    for name, names, optional, entries in (("ce_fwd", CE_FWD, ("lse",), 0),
                                           ("ce_bwd", CE_BWD, ("d_h", "d_w"), 0),
                                           ("distill_fwd", KD_FWD, ("lse",), 3),
                                           ("distill_bwd", KD_BWD, ("d_h", "d_w"), 3)):
        d = head.HeadDesc(**{**base, "entries": entries, **kw})
        need = tuple(n for n in names if not n.startswith("ld_"))

        def call(names=names, need=need, d=d, fn=getattr(H, "ssm_head_" + name), ws=(FAKE, 1 << 50),
                 **over):
            return _call(fn, names, need, d, ws=ws, **over)
        out[name] = call, need, optional
    return out


def test_every_declared_function_of_the_head_is_bound(H):
    for name in head.EXPORTED:
        assert hasattr(H, name), name


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=-1), INV), (dict(cols=0), INV), (dict(vocab=0), INV),
    (dict(vocab=-5), INV), (dict(io=2), INV), (dict(flags=1), INV), (dict(rows=(1 << 24) + 1), UNS),
    (dict(cols=65537), UNS), (dict(vocab=(1 << 22) + 1), UNS),
    (dict(rows=1 << 24, vocab=(1 << 16) + 1), UNS),
])
def test_head_refuses_bad_descriptors(H, kw, code):
    for name, (call, _, _) in _calls(H, **kw).items():
        assert call() == code, name
    d = head.HeadDesc(**{**dict(rows=4, cols=64, vocab=300, temperature=1.0), **kw})
    assert H.ssm_head_workspace_size(d, 0, 1) == 0


def test_head_refuses_bad_entries_and_temperatures(H):
    for kw, code in ((dict(entries=0), INV), (dict(entries=-1), INV), (dict(entries=129), UNS),
                     (dict(entry_io=3), INV), (dict(temperature=0.0), INV),
                     (dict(temperature=-1.0), INV), (dict(temperature=math.inf), INV),
                     (dict(temperature=math.nan), INV), (dict(temperature=9e-7), UNS),
                     (dict(temperature=1.1e6), UNS)):
        for name in ("distill_fwd", "distill_bwd"):
            assert _calls(H, **kw)[name][0]() == code, (name, kw)
    for name in ("ce_fwd", "ce_bwd"):
        assert _calls(H, entries=3)[name][0]() == INV, name
    d = head.HeadDesc(rows=4, cols=64, vocab=300, temperature=1.0)
    assert H.ssm_head_workspace_size(d, 4, 1) == 0 and H.ssm_head_workspace_size(d, -1, 1) == 0
    assert H.ssm_head_workspace_size(None, 0, 1) == 0


def test_head_refuses_bad_pointers_and_strides(H):
    for name, (call, need, optional) in _calls(H).items():
        for n in need:
            if n not in optional:
                assert call(**{n: None}) == INV, (name, n)
            wide = 8 if n in ("target", "t_idx") else 4
            assert call(**{n: FAKE + wide // 2}) == INV, (name, n)
        assert call(ld_h=63) == INV and call(ld_w=-64) == INV
        assert call(ld_h=1 << 40) == UNS and call(ld_w=1 << 40) == UNS
        if "d_h" in need:
            assert call(ld_d_h=63) == INV and call(ld_d_h=1 << 40) == UNS
            assert call(d_h=None, d_w=None) == INV
        # on a machine without a GPU the workspace's size cannot be known: an error in either case
        for ws in ((None, 0), (FAKE, 16), (FAKE + 8, 1 << 50)):
            assert call(ws=ws) in (WS, binding.SSM_ERR_CUDA)


def _words(*shape, gpu=0):
    return _fake(*shape, dtype=torch.int64, gpu=gpu)


def _head_calls():
    def v():
        return _fake(4)
    h, w, ws = _fake(4, 64), _fake(300, 64), _fake(1 << 16, dtype=torch.uint8)
    grads = dict(lse=v(), d_loss=v(), ws=ws, d_h=_fake(4, 64), d_w=_fake(300, 64))

    def g(a):
        return dict(ws=a["ws"], out={n: a[n] for n in ("d_h", "d_w")})
    return {
        "ce_fwd": (lambda a: head.ssm_head_ce_fwd(a["h"], a["w"], a["target"], ws=a["ws"],
                                                  out=(a["loss"], a["lse"])),
                   dict(h=h, w=w, target=_words(4), ws=ws, loss=v(), lse=v())),
        "ce_bwd": (lambda a: head.ssm_head_ce_bwd(a["h"], a["w"], a["target"], a["lse"], a["d_loss"],
                                                  **g(a)),
                   dict(h=h, w=w, target=_words(4), **grads)),
        "distill_fwd": (lambda a: head.ssm_head_distill_fwd(a["h"], a["w"], a["t_idx"], a["t_logit"],
                                                            ws=a["ws"], out=(a["loss"], a["lse"])),
                        dict(h=h, w=w, t_idx=_words(4, 3), t_logit=_fake(4, 3), ws=ws, loss=v(),
                             lse=v())),
        "distill_bwd": (lambda a: head.ssm_head_distill_bwd(a["h"], a["w"], a["t_idx"], a["t_logit"],
                                                            a["lse"], a["d_loss"], **g(a)),
                        dict(h=h, w=w, t_idx=_words(4, 3), t_logit=_fake(4, 3), **grads)),
    }


@pytest.mark.parametrize("name", list(_head_calls()))
def test_head_refuses_tensors_of_two_gpus_by_name(name):
    call, args = _head_calls()[name]
    for n, t in args.items():
        wrong = n if n != "h" else "|".join(args)
        with pytest.raises(ValueError, match=f"^({wrong}) must be a CUDA tensor on cuda"):
            call({**args, n: _fake(*t.shape, dtype=t.dtype, gpu=1)})


@pytest.mark.parametrize("name", list(_head_calls()))
def test_head_names_the_argument_that_is_not_a_tensor(name):
    call, args = _head_calls()[name]
    for n in args:
        optional = n in ("ws", "d_h", "d_w") or n == "lse" and name.endswith("fwd")
        for bad in ("text", None)[:1 if optional else 2]:
            with pytest.raises(TypeError, match="out" if n in ("d_h", "d_w") else n):
                call({**args, n: bad})
    with pytest.raises(ValueError, match="two dimensions"):
        call({**args, "w": _fake(300)})
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        call({**args, "h": _fake(4, 64, dtype=torch.float16)})
    with pytest.raises(ValueError, match="h must be a CUDA"):
        call({n: torch.empty(t.shape, dtype=t.dtype) for n, t in args.items()})
