"""The norms before and after the scan against their 64-bit forms (block_ref), on the GPU.

Tolerances (floored relative error, conftest.max_rel_err): with fp32 I/O the framework's gates,
1e-4 forward and 1e-3 for gradients, whose subtraction d_out w - n mean(...) cancels; with bf16
I/O one rounding to 8 bits, 2^-9, doubled to 2^-8 for values that fp32 errors carry over a
rounding boundary.  Parameter gradients are fp32 sums in either case: 1e-3."""
import pytest
import torch

import block_ref as ref
from bwd_ssm_conv_gb300 import SsmError, block
from gpu_util import TOL_F32_FWD, TOL_F32_GRAD, assert_close

pytestmark = pytest.mark.gpu
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def tol(dtype, grad):
    return 2.0 ** -8 if dtype == torch.bfloat16 else (TOL_F32_GRAD if grad else TOL_F32_FWD)


def close(name, got, want, grad=False):
    assert_close(name, got, want.numpy(), tol(got.dtype, grad))


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _strided(t, lead, tail):
    """The same values on the GPU as a slice [lead : lead + cols] of wider rows."""
    rows, cols = t.shape
    wide = torch.full((rows, lead + cols + tail), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, lead:lead + cols] = t.cuda()
    return wide[:, lead:lead + cols]


def _nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
SIZES = [  # (rows, cols): one column to the widest; odd widths; rows beyond the resident blocks
    (1, 1), (3, 7), (5, 8), (2, 24), (9, 32), (4, 33), (700, 40), (6, 96), (1, 256), (33, 264),
    (5, 520), (37, 768), (2, 1003), (1, 1536), (64, 2056), (3, 4104), (2, 8200), (2, 8193),
    (2, 32768), (1, 32767), (6001, 72),
]


def _add_inputs(rows, cols, io, res, seed):
    g = torch.Generator().manual_seed(seed)
    return dict(x=_rand(g, rows, cols, dtype=DT[io]), residual=_rand(g, rows, cols, dtype=DT[res]),
                scale=torch.rand(cols, generator=g) + 0.1, w=1.0 + 0.2 * _rand(g, cols),
                d_out=_rand(g, rows, cols, dtype=DT[io]), d_s=_rand(g, rows, cols, dtype=DT[res]))


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_add_norm(rows, cols, io, res):
    i = _add_inputs(rows, cols, io, res, seed=rows * 7 + cols)
    c = {k: v.cuda() for k, v in i.items()}
    out, s, rstd = ref.add_norm(i["x"], i["residual"], i["scale"], i["w"], EPS)
    a = block.ssm_add_norm_fwd(c["x"], c["w"], c["residual"], c["scale"], eps=EPS, save8=True,
                               save_x8=True, save_out8=True,
                               out=(_nan(out.shape, DT[io]), _nan(out.shape, DT[res])))
    close("out", a.out, out)
    close("s", a.res_out, s)
    close("rstd", a.rstd, rstd)
    # the stream is a product and a sum, each rounded once in fp32, then rounded to its type; the
    # checkpoints hold exactly what is stored
    s32 = (i["residual"].float() + i["scale"] * i["x"].float()).to(DT[res])
    assert torch.equal(a.res_out.cpu(), s32)
    for name, c8, of in (("res8", a.res8, s32), ("x8", a.x8, i["x"]), ("out8", a.out8, a.out.cpu())):
        q, e = ref.quantise(of)
        assert torch.equal(c8.q.cpu(), q) and torch.equal(c8.e.cpu(), e), name
    # backward from the stream, then from 8 bits
    for saved, x, s_in, x_in in ((a.res_out, c["x"], s32, i["x"]),
                                 (a.res8, a.x8, ref.through8(s32), ref.through8(i["x"]))):
        want = ref.add_norm_bwd(i["d_out"], s_in, a.rstd.cpu(), i["d_s"], i["scale"], i["w"], x_in)
        into = dict(d_res=_nan(out.shape, DT[res]), d_x=_nan(out.shape, DT[io]),
                    d_w=_nan((cols,), torch.float32), d_scale=_nan((cols,), torch.float32))
        got = block.ssm_add_norm_bwd(c["d_out"], saved, a.rstd, c["w"], d_res_out=c["d_s"],
                                     scale=c["scale"], x=x, out=into)
        for k, v in zip(("d_res", "d_x", "d_w", "d_scale"), want):
            close(k, got[k], v, grad=True)


def test_add_norm_without_its_optional_parts():
    i = _add_inputs(11, 136, "bf16", "f32", seed=5)
    c = {k: v.cuda() for k, v in i.items()}
    out, s, rstd = ref.add_norm(i["x"], None, None, None, EPS)
    a = block.ssm_add_norm_fwd(c["x"], eps=EPS)
    close("out", a.out, out)
    assert torch.equal(a.res_out, c["x"]) and a.res8 is None
    want = ref.add_norm_bwd(i["d_out"], s, a.rstd.cpu(), None, None, None, None)
    got = block.ssm_add_norm_bwd(c["d_out"], a.res_out, a.rstd)
    close("d_res", got["d_res"], want[0], grad=True)
    assert torch.equal(got["d_x"], got["d_res"]) and got["d_w"] is None and got["d_scale"] is None
    only = block.ssm_add_norm_bwd(c["d_out"], a.res_out, a.rstd, c["w"], want_dres=False,
                                  want_dx=False)
    close("d_w", only["d_w"], want[2], grad=True)


@pytest.mark.parametrize("lead,tail", [(0, 8), (8, 0), (3, 2), (1, 7)])  # aligned slices, and not
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_and_misaligned_rows(lead, tail, io):
    rows, cols = 19, 264
    i = _add_inputs(rows, cols, io, io, seed=17)
    c = {k: (_strided(v, lead, tail) if v.dim() == 2 else v.cuda()) for k, v in i.items()}
    out, s, _ = ref.add_norm(i["x"], i["residual"], i["scale"], i["w"], EPS)
    into = tuple(_strided(torch.zeros(rows, cols, dtype=DT[io]), lead, tail) for _ in range(2))
    a = block.ssm_add_norm_fwd(c["x"], c["w"], c["residual"], c["scale"], eps=EPS, out=into)
    close("out", a.out, out)
    close("s", a.res_out, s)
    want = ref.add_norm_bwd(i["d_out"], a.res_out.cpu(), a.rstd.cpu(), i["d_s"], i["scale"], i["w"], i["x"])
    got = block.ssm_add_norm_bwd(c["d_out"], a.res_out, a.rstd, c["w"], d_res_out=c["d_s"],
                                 scale=c["scale"], x=c["x"])
    for k, v in zip(("d_res", "d_x", "d_w", "d_scale"), want):
        close(k, got[k], v, grad=True)
    y = block.ssm_gated_norm_fwd(c["x"], c["d_out"], c["w"], group=88, out=into[0])
    close("gated", y.out, ref.gated_norm(i["x"], i["d_out"], i["w"], 88, EPS, False)[0])
    for t in into:  # nothing outside the slice was written
        wide = t._base
        assert bool(torch.isnan(wide[:, :lead]).all()) and bool(torch.isnan(wide[:, lead + cols:]).all())


GATED = [  # (rows, cols, group)
    (1, 1, 0), (3, 7, 0), (4, 33, 0), (16, 1536, 0), (300, 96, 0), (2, 8200, 0), (1, 32768, 0),
    (5, 512, 64), (130, 96, 32), (3, 1536, 768), (7, 480, 96), (2, 2048, 256), (9, 144, 48),
    (4, 60, 20), (3, 35, 5), (2, 24, 8), (3, 1000, 1), (1, 16384, 8192), (701, 128, 32),
]


@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,group", GATED)
def test_gated_norm(rows, cols, group, io, norm_first):
    g = torch.Generator().manual_seed(rows + cols + group)
    y, z, d = (_rand(g, rows, cols, dtype=DT[io]) for _ in range(3))
    w = 1.0 + 0.2 * _rand(g, cols)
    how = dict(group=group, norm_first=norm_first)
    out, rstd = ref.gated_norm(y, z, w, group, EPS, norm_first)
    zc = _strided(z, cols, 0)  # the gate's half of an input projection
    a = block.ssm_gated_norm_fwd(y.cuda(), zc, w.cuda(), eps=EPS, save8=True, save_out8=True,
                                 out=_nan(out.shape, DT[io]), **how)
    close("out", a.out, out)
    close("rstd", a.rstd, rstd)
    for name, c8, of in (("y8", a.y8, y), ("z8", a.z8, z), ("out8", a.out8, a.out.cpu())):
        q, e = ref.quantise(of)
        assert torch.equal(c8.q.cpu(), q) and torch.equal(c8.e.cpu(), e), name
    for yg, zg, yr, zr in ((y.cuda(), zc, y, z), (a.y8, a.z8, ref.through8(y), ref.through8(z))):
        want = ref.gated_norm_bwd(d, yr, zr, a.rstd.cpu(), w, group, norm_first)
        wide = _nan((rows, 2 * cols), DT[io])  # d_z into the projection's gradient
        into = dict(d_y=_nan(out.shape, DT[io]), d_z=wide[:, cols:], d_w=_nan((cols,), torch.float32))
        got = block.ssm_gated_norm_bwd(d.cuda(), yg, zg, a.rstd, w.cuda(), out=into, **how)
        for k, v in zip(("d_y", "d_z", "d_w"), want):
            close(k, got[k], v, grad=True)
        assert bool(torch.isnan(wide[:, :cols]).all())


def _gated_fwd_c(y, z, group, keep):
    """ssm_gated_norm_fwd through the C ABI with the checkpoints named in ``keep`` only; buffers for
    all three, filled with 99."""
    rows, cols = y.shape
    out = _nan((rows, cols), y.dtype)
    kept = {n: (torch.full((rows, cols), 99, dtype=torch.int8, device="cuda"),
                torch.full((rows, -(-cols // 32)), 99, dtype=torch.uint8, device="cuda"))
            for n in ("y", "z", "out")}
    pairs = [p.data_ptr() if n in keep else None for n in kept for p in kept[n]]
    d = block.NormDesc(rows, cols, group, block._IO[y.dtype], 0, 0, EPS)
    rc = block.lib().ssm_gated_norm_fwd(d, y.data_ptr(), 0, z.data_ptr(), 0, None, out.data_ptr(), 0,
                                        None, *pairs, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    return out, kept


@pytest.mark.parametrize("keep", [(), ("y",), ("z",), ("out",), ("y", "z"), ("z", "out")])
@pytest.mark.parametrize("io", ["f32", "bf16"])
# eight columns at a time, blocks of 32 that straddle groups, single columns, rows without groups
@pytest.mark.parametrize("rows,cols,group", [(9, 192, 64), (9, 144, 48), (5, 99, 33), (7, 264, 0),
                                             (3, 1003, 0), (2, 8200, 0)])
def test_gated_norm_keeps_each_checkpoint_by_itself(rows, cols, group, io, keep):
    g = torch.Generator().manual_seed(31)
    y, z = (_rand(g, rows, cols, dtype=DT[io]) for _ in range(2))
    out, kept = _gated_fwd_c(y.cuda(), z.cuda(), group, keep)
    close("out", out, ref.gated_norm(y, z, None, group, EPS, False)[0])
    for name, of in (("y", y), ("z", z), ("out", out.cpu())):
        q, e = (t.cpu() for t in kept[name])
        if name in keep:
            want_q, want_e = ref.quantise(of)
            assert torch.equal(q, want_q) and torch.equal(e, want_e), name
        else:
            assert bool((q == 99).all()) and bool((e == 99).all()), name


def test_zero_rows_and_bad_values_stay_in_their_rows():
    """An all-zero row gives zeros (eps keeps it finite); a row with an infinity or a NaN spoils
    its own outputs and its 8-bit block only."""
    g = torch.Generator().manual_seed(8)
    rows, cols = 6, 128
    x = _rand(g, rows, cols)
    x[1] = 0.0
    x[3, 40] = float("inf")
    x[4, 70] = float("nan")
    a = block.ssm_add_norm_fwd(x.cuda(), eps=EPS, save8=True)
    assert bool((a.out[1] == 0).all()) and bool(torch.isfinite(a.out[[0, 1, 2, 5]]).all())
    assert bool(torch.isnan(a.out[4]).all())
    e = a.res8.e.cpu()
    assert (e == 255).nonzero().tolist() == [[3, 1], [4, 2]]
    d = _rand(g, rows, cols)
    got = block.ssm_add_norm_bwd(d.cuda(), a.res8, a.rstd)
    assert bool(torch.isfinite(got["d_x"][[0, 1, 2, 5]]).all())
    b = block.ssm_gated_norm_fwd(x.cuda(), torch.full_like(x, -200.0).cuda(), norm_first=False)
    assert bool((b.out[0] == 0).all())  # a closed gate: silu(-200) is -0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [99, 264, 1003, 4608, 8193, 8200])  # every way a row is read
def test_backwards_of_checkpoints_with_zeros_for_padding(cols, io):
    """Rows and blocks of zeros, scale bytes and all, are zeros to the backwards too."""
    g = torch.Generator().manual_seed(cols)
    rows = 9
    s, x, y, z, d = (_rand(g, rows, cols, dtype=DT[io]) for _ in range(5))
    w, scale, rstd = 1.0 + 0.2 * _rand(g, cols), torch.rand(cols, generator=g), torch.rand(rows, generator=g) + 0.5
    kept = []
    for i, v in enumerate((s, x, y, z)):
        q, e = ref.quantise(v)
        q[2 + i:5], e[2 + i:5] = 0, 0
        q[7, -(cols % 32 or 32):], e[7, -1] = 0, 5
        kept.append((q, e))
    s8, x8, y8, z8 = (block.Ckpt8(q.cuda(), e.cuda()) for q, e in kept)
    s, x, y, z = (ref.kept(q, e) for q, e in kept)
    got = block.ssm_add_norm_bwd(d.cuda(), s8, rstd.cuda(), w.cuda(), scale=scale.cuda(), x=x8)
    want = ref.add_norm_bwd(d, s, rstd, None, scale, w, x)
    for k, v in zip(("d_res", "d_x", "d_w", "d_scale"), want):
        close(k, got[k], v, grad=True)
    got = block.ssm_gated_norm_bwd(d.cuda(), y8, z8, rstd[:, None].cuda(), w.cuda())
    for k, v in zip(("d_y", "d_z", "d_w"), ref.gated_norm_bwd(d, y, z, rstd[:, None], w, 0, False)):
        close(k, got[k], v, grad=True)


def test_outputs_in_place_of_inputs():
    g = torch.Generator().manual_seed(9)
    x, r, d = (_rand(g, 40, 200).cuda() for _ in range(3))
    a = block.ssm_add_norm_fwd(x, residual=r)
    x2, r2 = x.clone(), r.clone()
    b = block.ssm_add_norm_fwd(x2, residual=r2, out=(x2, r2))
    assert torch.equal(a.out, b.out) and torch.equal(a.res_out, b.res_out)
    g1 = block.ssm_add_norm_bwd(d, a.res_out, a.rstd)
    d2 = d.clone()
    g2 = block.ssm_add_norm_bwd(d2, a.res_out, a.rstd,
                                out=dict(d_res=None, d_x=d2, d_w=None, d_scale=None))
    assert torch.equal(g1["d_x"], g2["d_x"])


def test_same_bits_every_time_and_on_another_stream():
    g = torch.Generator().manual_seed(10)
    y, z, d = (_rand(g, 3000, 768, dtype=torch.bfloat16).cuda() for _ in range(3))
    w = _rand(g, 768).cuda()

    def once(stream=None):
        a = block.ssm_gated_norm_fwd(y, z, w, save8=True, stream=stream)
        b = block.ssm_gated_norm_bwd(d, a.y8, a.z8, a.rstd, w, stream=stream)
        return (a.out, b["d_y"], b["d_z"], b["d_w"])

    first = once()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (None, side):
        again = once(s)
        if s is not None:
            torch.empty(3000, 768, dtype=torch.bfloat16, device="cuda").zero_()  # takes no live memory
            s.synchronize()
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_more_than_two_dimensions_and_shape_checks():
    g = torch.Generator().manual_seed(11)
    x = _rand(g, 2, 3, 64).cuda()
    a = block.ssm_add_norm_fwd(x, save_out8=True)
    close("out", a.out.view(6, 64), ref.add_norm(x.cpu().view(6, 64), None, None, None, EPS)[0])
    assert a.rstd.shape == (2, 3) and a.out8.e.shape == (2, 3, 2)
    with pytest.raises(ValueError, match="residual"):
        block.ssm_add_norm_fwd(x, residual=x[:1])
    with pytest.raises(ValueError, match="one stride"):
        block.ssm_add_norm_fwd(_rand(g, 3, 2, 64).cuda().transpose(0, 1))
    with pytest.raises(ValueError, match="dense"):
        block.ssm_add_norm_fwd(_rand(g, 64, 3).cuda().t())
    with pytest.raises(ValueError, match="w must be"):
        block.ssm_add_norm_fwd(x, w=torch.ones(63, device="cuda"))
    with pytest.raises(TypeError, match="z must be"):
        block.ssm_gated_norm_fwd(x, x.bfloat16())
    with pytest.raises(ValueError, match="workspace"):
        block.ssm_add_norm_bwd(x, a.res_out, a.rstd, torch.ones(64, device="cuda"),
                               ws=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_rows_past_32_bit_offsets():
    rows, cols = 1_100_000, 2048  # 2.25e9 elements
    g = torch.Generator().manual_seed(12)
    last = _rand(g, 4, cols, dtype=torch.bfloat16)
    y = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    y[-4:], z[-4:] = last.cuda(), last.flip(0).cuda()
    a = block.ssm_gated_norm_fwd(y, z, eps=EPS, save8=True)
    close("out", a.out[-4:], ref.gated_norm(last, last.flip(0), None, 0, EPS, False)[0])
    assert torch.equal(a.y8.q[-4:].cpu(), ref.quantise(last)[0])
    b = block.ssm_gated_norm_bwd(y, a.y8, a.z8, a.rstd, out=dict(d_y=y, d_z=z, d_w=None))
    y8, z8 = ref.through8(last), ref.through8(last.flip(0))
    want = ref.gated_norm_bwd(last, y8, z8, a.rstd[-4:].cpu(), None, 0, False)
    close("d_y", b["d_y"][-4:], want[0], grad=True)
    close("d_z", b["d_z"][-4:], want[1], grad=True)


def test_what_a_call_makes_is_freed_with_its_results():
    x = torch.randn(40, 96, device="cuda")
    w = torch.ones(96, device="cuda")

    def step():
        a = block.ssm_add_norm_fwd(x, w, x, w, save8=True, save_x8=True, save_out8=True)
        g = block.ssm_add_norm_bwd(x, a.res8, a.rstd, w, d_res_out=x, scale=w, x=a.x8)
        b = block.ssm_gated_norm_fwd(x, x, w, save8=True, save_out8=True)
        h = block.ssm_gated_norm_bwd(x, b.y8, b.z8, b.rstd, w)
        d = block.ssm_ckpt8_wgrad(x, b.out8)
        e = block.ssm_ckpt8_load(block.ssm_ckpt8_save(x))
        with pytest.raises(ValueError):
            block.ssm_add_norm_fwd(x, w[:5])
        with pytest.raises(SsmError):
            block.ssm_gated_norm_fwd(x, x, w, group=7)
        return a, g, b, h, d, e

    step()
    before = torch.cuda.memory_allocated()
    kept = step()
    assert torch.cuda.memory_allocated() > before
    assert type(kept[0].res8) is block.Ckpt8 and type(kept[0]) is block.AddNorm
    del kept
    for _ in range(20):
        step()
    assert torch.cuda.memory_allocated() == before
