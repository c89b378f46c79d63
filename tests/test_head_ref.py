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
