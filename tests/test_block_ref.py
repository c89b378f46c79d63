"""The 64-bit reference of the norms, the 8-bit format and the C ABI's refusals, without a GPU."""
import ctypes
import math

import pytest
import torch

import block_ref as ref
from bwd_ssm_conv_gb300 import binding, block
from bwd_ssm_conv_gb300.build import build

f64 = torch.float64
INV, UNS, WS = binding.SSM_ERR_INVALID_ARG, binding.SSM_ERR_UNSUPPORTED, binding.SSM_ERR_WORKSPACE
FAKE = 1 << 20  # a non-null, aligned pointer value: never dereferenced by these tests


# ---- the formulas' gradients against differences of the forward --------------------------------
# Central differences at step 1e-5 in 64 bits: the error is step^2 times a third derivative of
# order one plus 1e-16 / step, both near 1e-10; 1e-7 leaves three orders for larger derivatives.

def _difference(loss, v):
    g = torch.zeros_like(v)
    flat, out = v.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        at = float(flat[i])
        flat[i] = at + 1e-5
        up = float(loss())
        flat[i] = at - 1e-5
        out[i] = (up - float(loss())) / 2e-5
        flat[i] = at
    return g


@pytest.mark.parametrize("with_scale,with_residual", [(True, True), (False, True), (True, False)])
def test_add_norm_gradient_is_that_of_its_forward(with_scale, with_residual):
    g = torch.Generator().manual_seed(1)
    R, C = 3, 5
    x, w, d_out, d_s = (torch.randn(*s, generator=g, dtype=f64) for s in ((R, C), (C,), (R, C), (R, C)))
    res = torch.randn(R, C, generator=g, dtype=f64) if with_residual else None
    scale = torch.rand(C, generator=g, dtype=f64) if with_scale else None

    def loss():
        out, s, _ = ref.add_norm(x, res, scale, w, 1e-3)
        return (out * d_out).sum() + (s * d_s).sum()

    _, s, rstd = ref.add_norm(x, res, scale, w, 1e-3)
    d_res, d_x, d_w, d_scale = ref.add_norm_bwd(d_out, s, rstd, d_s, scale, w, x)
    for got, v in ((d_x, x), (d_w, w)) + (((d_res, res),) if with_residual else ()) + \
            (((d_scale, scale),) if with_scale else ()):
        assert torch.allclose(got, _difference(loss, v), rtol=0, atol=1e-7)


@pytest.mark.parametrize("group,norm_first", [(0, False), (0, True), (3, False), (3, True)])
def test_gated_norm_gradient_is_that_of_its_forward(group, norm_first):
    g = torch.Generator().manual_seed(2)
    R, C = 2, 6
    y, z, w, d = (torch.randn(*s, generator=g, dtype=f64) for s in ((R, C), (R, C), (C,), (R, C)))

    def loss():
        return (ref.gated_norm(y, z, w, group, 1e-3, norm_first)[0] * d).sum()

    _, rstd = ref.gated_norm(y, z, w, group, 1e-3, norm_first)
    for got, v in zip(ref.gated_norm_bwd(d, y, z, rstd, w, group, norm_first), (y, z, w)):
        assert torch.allclose(got, _difference(loss, v), rtol=0, atol=1e-7)


def test_kept_value_is_within_a_step_of_the_value():
    g = torch.Generator().manual_seed(3)
    v = torch.randn(8, 100, generator=g, dtype=f64) * torch.exp2(torch.randint(-140, 120, (8, 1), generator=g).to(f64))
    q, e = ref.quantise(v)
    got = ref.kept(q, e)
    step = torch.exp2(e.to(f64) - 133.0).repeat_interleave(32, 1)[:, :100]
    bound = torch.where(v.abs() > 127 * step, step, step / 2)
    assert bool(((got - v).abs() <= bound).all())
    assert torch.equal(got.to(torch.bfloat16).to(f64), got)  # bf16 holds it exactly


# ---- refusals ------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def L():
    build()
    return block.lib()


def _desc(**kw):
    base = dict(rows=4, cols=64, group=0, io=0, res_io=0, flags=0, eps=1e-5)
    base.update(kw)
    return block.NormDesc(**base)


ADD_FWD = ("x ld_x residual ld_residual scale w out ld_out res_out ld_res_out rstd res_q res_e x_q "
           "x_e out_q out_e").split()
ADD_BWD = ("d_out ld_d_out d_res_out ld_d_res_out res ld_res res_q res_e x ld_x x_q x_e rstd scale "
           "w d_res ld_d_res d_x ld_d_x d_w d_scale").split()
GATED_FWD = "y ld_y z ld_z w out ld_out rstd y_q y_e z_q z_e out_q out_e".split()
GATED_BWD = ("d_out ld_d_out y ld_y y_q y_e z ld_z z_q z_e rstd w d_y ld_d_y d_z ld_d_z "
             "d_w").split()


def _call(fn, names, required, desc, ws=None, **over):
    args = [over.get(n, 0 if n.startswith("ld_") else FAKE if n in required else None) for n in names]
    return fn(desc, *args, *([] if ws is None else ws), None)


def test_every_declared_function_is_bound(L):
    for name in block.EXPORTED:
        assert hasattr(L, name), name


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(rows=-3), INV), (dict(cols=0), INV), (dict(io=7), INV),
    (dict(group=-1), INV), (dict(group=128), INV), (dict(group=24), INV), (dict(eps=0.0), INV),
    (dict(eps=-1.0), INV), (dict(eps=math.inf), INV), (dict(eps=math.nan), INV),
    (dict(flags=2), INV), (dict(cols=32769), UNS), (dict(rows=1 << 40), UNS),
])
def test_norms_refuse_bad_descriptors(L, kw, code):
    d = _desc(**kw)
    assert _call(L.ssm_add_norm_fwd, ADD_FWD, ("x", "out"), d) == code
    assert _call(L.ssm_add_norm_bwd, ADD_BWD, ("d_out", "res", "rstd", "d_x"), d,
                 ws=(FAKE, 1 << 30)) == code
    assert _call(L.ssm_gated_norm_fwd, GATED_FWD, ("y", "z", "out"), d) == code
    assert _call(L.ssm_gated_norm_bwd, GATED_BWD, ("d_out", "y", "z", "rstd", "d_y", "d_z"), d,
                 ws=(FAKE, 1 << 30)) == code
    assert L.ssm_norm_bwd_workspace_size(d, 1) == 0


def test_add_norm_fwd_refusals(L):
    def f(desc=None, **over):
        return _call(L.ssm_add_norm_fwd, ADD_FWD, ("x", "out"), desc or _desc(), **over)
    assert f(x=None) == INV and f(out=None) == INV
    assert f(_desc(group=32)) == INV                  # one norm per row
    assert f(_desc(io=0, res_io=1)) == INV            # a stream narrower than the activations
    assert f(x=FAKE + 2) == INV and f(w=FAKE + 2) == INV and f(rstd=FAKE + 1) == INV
    assert f(ld_x=63) == INV and f(residual=FAKE, ld_residual=-64) == INV
    assert f(ld_x=1 << 40) == UNS
    for a, b in (("res_q", "res_e"), ("x_q", "x_e"), ("out_q", "out_e")):
        assert f(**{a: FAKE}) == INV and f(**{b: FAKE}) == INV


def test_add_norm_bwd_refusals(L):
    need = ("d_out", "res", "rstd", "d_x", "d_w")

    def f(desc=None, ws=(FAKE, 1 << 30), **over):
        return _call(L.ssm_add_norm_bwd, ADD_BWD, need, desc or _desc(), ws=ws, **over)
    assert f(d_out=None) == INV and f(rstd=None) == INV and f(res=None) == INV
    assert f(d_x=None, d_w=None) == INV               # nothing to compute
    assert f(res_q=FAKE, res_e=FAKE) == INV           # s given twice
    assert f(res=None, res_q=FAKE) == INV
    assert f(x=FAKE, x_q=FAKE, x_e=FAKE) == INV
    assert f(d_scale=FAKE, scale=FAKE) == INV         # d_scale needs x
    assert f(d_scale=FAKE, x=FAKE) == INV             # ... and scale
    assert f(d_x=FAKE + 2) == INV and f(ld_d_x=8) == INV


def test_gated_norm_refusals(L):
    def f(**over):
        return _call(L.ssm_gated_norm_fwd, GATED_FWD, ("y", "z", "out"), _desc(), **over)
    assert f(y=None) == INV and f(z=None) == INV and f(out=None) == INV
    assert f(z=FAKE + 2) == INV and f(ld_z=32) == INV and f(z_q=FAKE) == INV
    need = ("d_out", "y", "z", "rstd", "d_y", "d_z")

    def b(ws=(FAKE, 1 << 30), **over):
        return _call(L.ssm_gated_norm_bwd, GATED_BWD, need, _desc(), ws=ws, **over)
    for n in need:
        assert b(**{n: None}) == INV, n
    assert b(y_q=FAKE, y_e=FAKE) == INV                       # y given twice
    assert b(y=None, y_q=FAKE, y_e=FAKE) == INV               # a checkpoint of y, a tensor z
    assert b(y=None, z=None, y_q=FAKE, y_e=FAKE, z_q=FAKE) == INV


def test_ckpt8_and_wgrad_refusals(L):
    def save(x=FAKE, ld=0, q=FAKE, e=FAKE, rows=4, cols=64, io=0):
        return L.ssm_ckpt8_save(x, ld, q, e, rows, cols, io, None)
    assert save(x=None) == INV and save(q=None) == INV and save(e=None) == INV
    assert save(rows=0) == INV and save(cols=0) == INV and save(io=5) == INV
    assert save(ld=63) == INV and save(x=FAKE + 2) == INV
    assert save(cols=(1 << 20) + 1) == UNS and save(rows=1 << 40) == UNS
    assert L.ssm_ckpt8_load(None, FAKE, FAKE, 0, 4, 64, 0, None) == INV
    assert L.ssm_ckpt8_load(FAKE, FAKE, FAKE + 1, 0, 4, 64, 1, None) == INV

    def wgrad(g=FAKE, ld=0, q=FAKE, e=FAKE, d_W=FAKE, t=4, m=64, k=64, io=0, flags=0, ws=FAKE,
              n=1 << 40):
        return L.ssm_ckpt8_wgrad(g, ld, q, e, d_W, t, m, k, io, flags, ws, n, None)
    for name in ("g", "q", "e", "d_W"):
        assert wgrad(**{name: None}) == INV, name
    assert wgrad(t=0) == INV and wgrad(m=0) == INV and wgrad(k=-1) == INV and wgrad(io=2) == INV
    assert wgrad(flags=2) == INV and wgrad(ld=63) == INV and wgrad(d_W=FAKE + 2) == INV
    assert wgrad(m=(1 << 20) + 1) == UNS and wgrad(t=(1 << 29) + 1) == UNS
    assert L.ssm_ckpt8_wgrad_workspace_size(0, 64, 64, 0, 1) == 0


def test_binding_refuses_what_the_library_cannot_see():
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        block.ssm_add_norm_fwd(t, out=(t, None))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        block.ssm_ckpt8_save(t.double())
    with pytest.raises(ValueError, match="accumulate"):
        block.ssm_ckpt8_wgrad(t, block.Ckpt8(t.to(torch.int8), t[:, :2].to(torch.uint8)),
                              accumulate=True)


def test_binding_names_the_argument_that_is_not_a_tensor():
    t = torch.zeros(4, 64)
    c = block.Ckpt8(t.to(torch.int8), t[:, :2].to(torch.uint8))
    for call, name in ((lambda: block.ssm_add_norm_fwd([1.0]), "x"),
                       (lambda: block.ssm_add_norm_fwd(t, w=2.0), "w"),
                       (lambda: block.ssm_add_norm_bwd(t, None, t), "res"),
                       (lambda: block.ssm_gated_norm_fwd(t, None), "z"),
                       (lambda: block.ssm_gated_norm_bwd(t, t, None, t), "z"),
                       (lambda: block.ssm_ckpt8_load(t), "c"),
                       (lambda: block.ssm_ckpt8_save(t, out=t), "out|x"),
                       (lambda: block.ssm_ckpt8_wgrad(t, t), "x8"),
                       (lambda: block.ssm_ckpt8_wgrad(None, c), "g")):
        with pytest.raises((TypeError, ValueError), match=name):
            call()
    with pytest.raises(ValueError, match="dimension"):
        block.ssm_ckpt8_save(torch.tensor(1.0))
    with pytest.raises(TypeError, match="dtype"):
        block.ssm_add_norm_fwd(t, res_dtype="float32")
    with pytest.raises(ValueError, match="pair"):
        block.ssm_ckpt8_load((c.q,))


# ---- devices: tensors that only look like those of two GPUs, so that nothing can run ---------------

def _fake(*shape, dtype=torch.float32, gpu=0):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=f"cuda:{gpu}")


def _fake8(rows, cols, gpu_q=0, gpu_e=0):
    return block.Ckpt8(_fake(rows, cols, dtype=torch.int8, gpu=gpu_q),
                       _fake(rows, -(-cols // 32), dtype=torch.uint8, gpu=gpu_e))


def _device_calls():
    """(call, its tensor arguments by the name that the error gives them)"""
    def t():
        return _fake(4, 64)

    def v():
        return _fake(64)
    ws = _fake(1 << 16, dtype=torch.uint8)
    return {
        "add_norm_fwd": (lambda a: block.ssm_add_norm_fwd(
            a["x"], a["w"], a["residual"], a["scale"], out=(a["out"], a["res_out"])),
            dict(x=t(), w=v(), residual=t(), scale=v(), out=t(), res_out=t())),
        "add_norm_bwd": (lambda a: block.ssm_add_norm_bwd(
            a["d_out"], a["res"], a["rstd"], a["w"], a["d_res_out"], a["scale"], a["x"], ws=a["ws"],
            out={n: a[n] for n in ("d_res", "d_x", "d_w", "d_scale")}),
            dict(d_out=t(), res=t(), rstd=_fake(4), w=v(), d_res_out=t(), scale=v(), x=t(), ws=ws,
                 d_res=t(), d_x=t(), d_w=v(), d_scale=v())),
        "add_norm_bwd8": (lambda a: block.ssm_add_norm_bwd(
            a["d_out"], a["res"], a["rstd"], scale=a["scale"], x=a["x"]),
            dict(d_out=t(), res=_fake8(4, 64), rstd=_fake(4), scale=v(), x=_fake8(4, 64))),
        "gated_norm_fwd": (lambda a: block.ssm_gated_norm_fwd(a["y"], a["z"], a["w"], out=a["out"]),
                           dict(y=t(), z=t(), w=v(), out=t())),
        "gated_norm_bwd": (lambda a: block.ssm_gated_norm_bwd(
            a["d_out"], a["y"], a["z"], a["rstd"], a["w"], ws=a["ws"],
            out={n: a[n] for n in ("d_y", "d_z", "d_w")}),
            dict(d_out=t(), y=t(), z=t(), rstd=_fake(4), w=v(), ws=ws, d_y=t(), d_z=t(), d_w=v())),
        "gated_norm_bwd8": (lambda a: block.ssm_gated_norm_bwd(a["d_out"], a["y"], a["z"], a["rstd"]),
                            dict(d_out=t(), y=_fake8(4, 64), z=_fake8(4, 64), rstd=_fake(4))),
        "ckpt8_save": (lambda a: block.ssm_ckpt8_save(a["x"], out=a["out"]),
                       dict(x=t(), out=_fake8(4, 64))),
        "ckpt8_load": (lambda a: block.ssm_ckpt8_load(a["c"], out=a["out"]),
                       dict(c=_fake8(4, 64), out=t())),
        "ckpt8_wgrad": (lambda a: block.ssm_ckpt8_wgrad(a["g"], a["x8"], ws=a["ws"], out=a["out"]),
                        dict(g=t(), x8=_fake8(4, 64), ws=ws, out=_fake(64, 64))),
    }


@pytest.mark.parametrize("name", list(_device_calls()))
def test_binding_refuses_tensors_of_two_gpus_by_name(name):
    call, args = _device_calls()[name]
    first = next(iter(args))
    for n, t in args.items():
        if isinstance(t, tuple):
            others = [_fake8(4, 64, 0, 1)] + ([_fake8(4, 64, 1, 1)] if n != first else [])
        else:
            others = [_fake(*t.shape, dtype=t.dtype, gpu=1)]
        for other in others:
            # the first tensor's GPU is the call's: with that one elsewhere, the next is refused
            wrong = n if n != first or isinstance(t, tuple) else "|".join(args)
            with pytest.raises(ValueError, match=f"^({wrong}) must be a CUDA tensor on cuda"):
                call({**args, n: other})
