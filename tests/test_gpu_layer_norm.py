"""The residual add and layer norm against its 64-bit form (head_ref, where the bounds are derived), on
the GPU."""
import pytest
import torch

import block_ref as ref
import head_ref
from bwd_ssm_conv_gb300 import SsmError, block
from head_ref import within

pytestmark = pytest.mark.gpu
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
OUTS = ("d_res", "d_x", "d_w", "d_b", "d_scale")


def _rand(g, *shape, dtype=torch.float32, std=1.0, at=0.0):
    return (at + torch.randn(*shape, generator=g) * std).to(dtype)


def _nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _inputs(rows, cols, io, res, seed, at=0.0):
    g = torch.Generator().manual_seed(seed)
    return dict(x=_rand(g, rows, cols, dtype=DT[io]),
                residual=_rand(g, rows, cols, dtype=DT[res], at=at),
                scale=torch.rand(cols, generator=g) + 0.1, w=1.0 + 0.2 * _rand(g, cols),
                b=0.3 * _rand(g, cols), d_out=_rand(g, rows, cols, dtype=DT[io]),
                d_s=_rand(g, rows, cols, dtype=DT[res]))


def _check_fwd(a, i, eps=EPS):
    want, bound = head_ref.layer_norm(i["x"], i.get("residual"), i.get("scale"), i.get("w"),
                                      i.get("b"), eps)
    for name, got, v, e in zip(("out", "s", "mean", "rstd"), (a.out, a.res_out, a.mean, a.rstd),
                               want, bound):
        if got is not None:
            within(name, got, v, e)


def _check_bwd(got, i, s, mean, rstd, x, d_s="d_s"):
    want, bound = head_ref.layer_norm_bwd(i["d_out"], s, mean.cpu(), rstd.cpu(), i.get(d_s),
                                          i.get("scale"), i.get("w"), x)
    for name, v, e in zip(OUTS, want, bound):
        if got[name] is not None:
            within(name, got[name], v, e)


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
SIZES = [  # (rows, cols): one column to the widest; odd widths; rows beyond the resident blocks
    (1, 1), (3, 7), (5, 8), (2, 24), (9, 32), (4, 33), (700, 40), (6, 96), (1, 256), (33, 264),
    (5, 520), (37, 768), (2, 1003), (1, 1536), (64, 2056), (3, 4104), (2, 4608), (2, 8200),
    (2, 8193), (2, 32768), (1, 32767), (6001, 72), (2000, 99), (900, 1536),
]


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_add_layer_norm(rows, cols, io, res):
    i = _inputs(rows, cols, io, res, seed=rows * 7 + cols, at=3.0)
    c = {k: v.cuda() for k, v in i.items()}
    shape = (rows, cols)
    a = block.ssm_add_layer_norm_fwd(c["x"], c["w"], c["b"], c["residual"], c["scale"], eps=EPS,
                                     save8=True, save_x8=True, save_out8=True,
                                     out=(_nan(shape, DT[io]), _nan(shape, DT[res])))
    _check_fwd(a, i)
    # the stream holds the bits of an unfused add; the checkpoints hold what is stored
    s32 = (i["residual"].float() + i["scale"] * i["x"].float()).to(DT[res])
    assert torch.equal(a.res_out.cpu(), s32)
    for name, c8, of in (("res8", a.res8, s32), ("x8", a.x8, i["x"]), ("out8", a.out8, a.out.cpu())):
        q, e = ref.quantise(of)
        assert torch.equal(c8.q.cpu(), q) and torch.equal(c8.e.cpu(), e), name
    # backward from the stream, then from 8 bits
    for saved, x, s_in, x_in in ((a.res_out, c["x"], s32, i["x"]),
                                 (a.res8, a.x8, ref.through8(s32), ref.through8(i["x"]))):
        into = dict(d_res=_nan(shape, DT[res]), d_x=_nan(shape, DT[io]),
                    **{n: _nan((cols,), torch.float32) for n in OUTS[2:]})
        got = block.ssm_add_layer_norm_bwd(c["d_out"], saved, a.mean, a.rstd, c["w"],
                                           d_res_out=c["d_s"], scale=c["scale"], x=x, out=into)
        _check_bwd(got, i, s_in, a.mean, a.rstd, x_in)


def test_without_its_optional_parts():
    i = _inputs(11, 136, "bf16", "f32", seed=5)
    c = {k: v.cuda() for k, v in i.items()}
    bare = dict(x=i["x"], d_out=i["d_out"])
    a = block.ssm_add_layer_norm_fwd(c["x"], eps=EPS)
    _check_fwd(a, bare)
    assert torch.equal(a.res_out, c["x"]) and a.res8 is None
    got = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd)
    _check_bwd(got, bare, i["x"], a.mean, a.rstd, None)
    assert torch.equal(got["d_x"], got["d_res"]) and got["d_w"] is None and got["d_scale"] is None
    none = block.ssm_add_layer_norm_fwd(c["x"], b=c["b"], want_stats=False, want_res=False)
    assert none.mean is None and none.rstd is None and none.res_out is None
    _check_fwd(none, dict(x=i["x"], b=i["b"]))
    # each column sum by itself, and without any
    how = dict(want_dres=False, want_dx=False)
    only = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, c["w"],
                                        want_db=False, **how)
    _check_bwd(only, dict(bare, w=i["w"]), i["x"], a.mean, a.rstd, None)
    assert only["d_b"] is None and only["d_w"] is not None
    only = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, **how)
    _check_bwd(only, bare, i["x"], a.mean, a.rstd, None)
    assert only["d_b"] is not None and only["d_w"] is None
    two = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, scale=c["scale"],
                                       x=c["x"], **how)
    _check_bwd(two, dict(bare, scale=i["scale"]), i["x"], a.mean, a.rstd, i["x"])
    assert two["d_b"] is not None and two["d_scale"] is not None
    plain = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, want_db=False)
    _check_bwd(plain, bare, i["x"], a.mean, a.rstd, None)


@pytest.mark.parametrize("lead,tail", [(0, 8), (8, 0), (3, 2), (1, 7)])  # aligned slices, and not
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_and_misaligned_rows(lead, tail, io):
    rows, cols = 19, 264
    i = _inputs(rows, cols, io, io, seed=17)

    def strided(t):
        wide = _nan((rows, lead + cols + tail), t.dtype)
        wide[:, lead:lead + cols] = t.cuda()
        return wide[:, lead:lead + cols]

    c = {k: strided(v) if v.dim() == 2 else v.cuda() for k, v in i.items()}
    zero = torch.zeros(rows, cols, dtype=DT[io])
    into = strided(zero), strided(zero)
    a = block.ssm_add_layer_norm_fwd(c["x"], c["w"], c["b"], c["residual"], c["scale"], eps=EPS, out=into)
    _check_fwd(a, i)
    grads = dict(d_res=strided(zero), d_x=strided(zero),
                 **{n: _nan((cols,), torch.float32) for n in OUTS[2:]})
    got = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, c["w"], d_res_out=c["d_s"],
                                       scale=c["scale"], x=c["x"], out=grads)
    _check_bwd(got, i, a.res_out.cpu(), a.mean, a.rstd, i["x"])
    for t in into + (grads["d_res"], grads["d_x"]):  # nothing outside the slice was written
        wide = t._base
        assert bool(torch.isnan(wide[:, :lead]).all()) and bool(torch.isnan(wide[:, lead + cols:]).all())


@pytest.mark.parametrize("cols", [40, 768, 1003, 4104])
def test_a_mean_far_from_zero_keeps_its_digits(cols):
    """Rows around 1000 with a deviation of 1: the mean of the squares alone has 20 bits of the 24 taken up."""
    i = _inputs(7, cols, "f32", "f32", seed=cols, at=1000.0)
    c = {k: v.cuda() for k, v in i.items()}
    a = block.ssm_add_layer_norm_fwd(c["x"], c["w"], c["b"], c["residual"], eps=EPS)
    _check_fwd(a, {k: v for k, v in i.items() if k != "scale"})
    want = head_ref.layer_norm(i["x"], i["residual"], None, i["w"], i["b"], EPS)[0][0]
    # the bound above allows for the mean's error; the digits themselves: a row's mean is good to
    # 1000 SUM 2^-24 = 3e-3 of a deviation at the very worst
    assert float((a.out.cpu().double() - want).abs().max()) < 1e-2


def test_constant_rows_and_bad_values_stay_in_their_rows():
    """A row of one value has no deviation: eps keeps it finite and out is b; a row with an infinity
    or a NaN spoils itself only."""
    g = torch.Generator().manual_seed(8)
    rows, cols = 6, 128
    x, b, d = _rand(g, rows, cols), _rand(g, cols), _rand(g, rows, cols)
    x[1], x[3, 40], x[4, 70] = 2.0, float("inf"), float("nan")
    a = block.ssm_add_layer_norm_fwd(x.cuda(), b=b.cuda(), eps=EPS)
    assert torch.equal(a.out[1].cpu(), b) and bool(torch.isfinite(a.out[[0, 1, 2, 5]]).all())
    assert bool(torch.isnan(a.out[[3, 4]]).all())
    got = block.ssm_add_layer_norm_bwd(d.cuda(), a.res_out, a.mean, a.rstd)
    assert bool(torch.isfinite(got["d_x"][[0, 1, 2, 5]]).all())


def test_in_place_on_another_stream_and_in_a_graph():
    i = _inputs(300, 264, "bf16", "bf16", seed=9)
    c = {k: v.cuda() for k, v in i.items()}

    def once(stream=None):
        a = block.ssm_add_layer_norm_fwd(c["x"], c["w"], c["b"], c["residual"], c["scale"],
                                         stream=stream)
        g = block.ssm_add_layer_norm_bwd(c["d_out"], a.res_out, a.mean, a.rstd, c["w"], c["d_s"],
                                         c["scale"], c["x"], stream=stream)
        return [a.out, a.res_out, a.mean, a.rstd] + [g[n] for n in OUTS]

    first = once()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = once(side)
    side.synchronize()
    for p, q in zip(first, again):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for t in held:
        t.zero_()
    for _ in range(2):
        graph.replay()
    for p, q in zip(first, held):
        assert torch.equal(p, q)
    x2, r2 = c["x"].clone(), c["residual"].clone()
    a = block.ssm_add_layer_norm_fwd(x2, c["w"], c["b"], r2, c["scale"], out=(x2, r2))
    assert torch.equal(a.out, first[0]) and torch.equal(a.res_out, first[1])
    d2, u2 = c["d_out"].clone(), c["d_s"].clone()
    sums = {n: _nan((264,), torch.float32) for n in OUTS[2:]}
    block.ssm_add_layer_norm_bwd(d2, r2, a.mean, a.rstd, c["w"], u2, c["scale"], c["x"],
                                 out=dict(d_res=u2, d_x=d2, **sums))
    for p, q in zip(first[4:], (u2, d2, sums["d_w"], sums["d_b"], sums["d_scale"])):
        assert torch.equal(p, q)


def test_more_dimensions_and_shape_checks():
    x = torch.randn(2, 3, 64, device="cuda")
    a = block.ssm_add_layer_norm_fwd(x, save_out8=True)
    assert a.mean.shape == a.rstd.shape == (2, 3) and a.out8.e.shape == (2, 3, 2)
    with pytest.raises(ValueError, match="b must be"):
        block.ssm_add_layer_norm_fwd(x, b=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="mean must be"):
        block.ssm_add_layer_norm_bwd(x, a.res_out, a.mean[:1].contiguous(), a.rstd)
    with pytest.raises(SsmError):
        block.ssm_add_layer_norm_fwd(x, eps=0.0)
    with pytest.raises(ValueError, match="workspace"):
        block.ssm_add_layer_norm_bwd(x, a.res_out, a.mean, a.rstd,
                                     ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
