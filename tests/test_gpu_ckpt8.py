"""8-bit activation checkpoints and the weight gradient that reads them, against block_ref."""
import pytest
import torch

import block_ref as ref
from bwd_ssm_conv_gb300 import binding, block

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _check(x, xc, dtype):
    q, e = ref.quantise(x)
    c = block.ssm_ckpt8_save(xc, out=block.Ckpt8(torch.full(q.shape, 99, dtype=torch.int8, device="cuda"),
                                                 torch.full(e.shape, 99, dtype=torch.uint8, device="cuda")))
    assert torch.equal(c.q.cpu(), q) and torch.equal(c.e.cpu(), e)
    want = ref.kept(q, e)
    for dt in DT.values():  # both types hold every kept value exactly
        got = block.ssm_ckpt8_load(c, dt)
        assert got.dtype == dt
        assert torch.allclose(got.cpu().double(), want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 31), (4, 32), (7, 33), (9, 72),
                                       (3, 517), (2, 1024), (33, 1536), (1, 40000), (1000, 64)])
def test_save_and_load(rows, cols, io):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(cols, generator=g))).to(DT[io])
    _check(x, x.cuda(), io)


def test_edges_of_the_format():
    x = torch.randn(16, 96, generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 40] = float("nan")
    x[3, 64] = -float("inf")
    x[4] = 1e-40                       # subnormal: the scale stops at 2^-120
    x[5] *= 2.0 ** -119                # around the smallest scale
    x[6] = torch.finfo(torch.float32).max * torch.sign(x[6])
    x[7] = 127.5 / 64                  # past the last value: limited to 127
    x[8, ::2], x[8, 1::2] = -127.9 / 64, 1.0
    x[9] = (torch.arange(96) % 64 + 0.5) / 64  # ties, to even
    x[9, ::32] = 1.0
    x[10] = 2.0 ** torch.arange(-40, 56).float()
    x[11] = -(2.0 ** torch.arange(-126, -30).float())
    x[12] = float("nan")
    _check(x, x.cuda(), "f32")
    _check(x.bfloat16(), x.bfloat16().cuda(), "bf16")


@pytest.mark.parametrize("cols", [32, 33, 64])  # one column and eight at a time
def test_every_scale_byte_reads_as_its_power_of_two(cols):
    g = torch.Generator().manual_seed(21)
    q = torch.randint(-127, 128, (256, cols), generator=g).to(torch.int8)
    q[:, ::5] = 0
    e = torch.arange(256)[:, None].expand(256, -(-cols // 32)).to(torch.uint8).contiguous()
    want = ref.kept(q, e)
    for dt in DT.values():  # both types hold q 2^(e - 133) exactly, as subnormals where e is small
        got = block.ssm_ckpt8_load(block.Ckpt8(q.cuda(), e.cuda()), dt).cpu().double()
        assert torch.allclose(got, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("lead,tail", [(8, 8), (1, 2)])
def test_strided_rows(lead, tail):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(21, 104, generator=g)
    wide = torch.zeros(21, lead + 104 + tail, device="cuda")
    wide[:, lead:lead + 104] = x.cuda()
    view = wide[:, lead:lead + 104]
    _check(x, view, "f32")
    c = block.ssm_ckpt8_save(view)
    wide.fill_(7.0)
    block.ssm_ckpt8_load(c, out=view)
    assert torch.equal(view.cpu().double(), ref.through8(x))
    assert bool((wide[:, :lead] == 7).all()) and bool((wide[:, lead + 104:] == 7).all())


def test_offsets_past_32_bits():
    rows, cols = 2_200_000, 1024
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(3, cols, generator=torch.Generator().manual_seed(3)).bfloat16()
    x[-3:] = last.cuda()
    c = block.ssm_ckpt8_save(x)
    q, e = ref.quantise(last)
    assert torch.equal(c.q[-3:].cpu(), q) and torch.equal(c.e[-3:].cpu(), e)
    assert torch.equal(block.ssm_ckpt8_load(c, out=x)[-3:].cpu().double(), ref.kept(q, e))


# ---- the weight gradient --------------------------------------------------------------------------

SIZES = [  # (tokens, m, k)
    (1, 1, 1), (1, 8, 32), (2, 64, 64), (3, 5, 33), (63, 128, 256), (64, 128, 128), (65, 136, 264),
    (127, 16, 2048), (500, 80, 96), (1000, 768, 1536), (129, 1000, 31), (4097, 64, 512),
    (31, 2056, 72), (2049, 130, 300), (1024, 264, 1032), (40000, 40, 72),
]


def _exact_case(tokens, m, k, dtype, seed):
    """Integer g in +-4 and checkpoints of few distinct scales: every product and every partial
    sum in any order is an integer multiple of 2^-9 below 2^24 times it, so that fp32 sums are
    exact and the result must be equal."""
    g = torch.Generator().manual_seed(seed)
    top = max(1, min(4, 2 ** 20 // (tokens * 16)))
    gv = torch.randint(-top, top + 1, (tokens, m), generator=g).to(dtype)
    q = torch.randint(-4, 5, (tokens, k), generator=g).to(torch.int8)
    e = torch.randint(124, 126, (tokens, -(-k // 32)), generator=g).to(torch.uint8)
    return gv, q, e


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,m,k", SIZES)
def test_wgrad_is_exact_where_fp32_is(tokens, m, k, io):
    gv, q, e = _exact_case(tokens, m, k, DT[io], seed=tokens + m + k)
    want = gv.double().t() @ ref.kept(q, e)
    out = torch.full((m, k), float("nan"), device="cuda")
    got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda()), out=out)
    assert torch.equal(got.cpu().double(), want)
    # added to what is there
    start = torch.randint(-8, 9, (m, k), generator=torch.Generator().manual_seed(5)).float()
    out = start.cuda()
    block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda()), out=out, accumulate=True)
    assert torch.equal(out.cpu().double(), want + start.double())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,m,k", [(700, 200, 96), (5000, 128, 320), (8192, 256, 256)])
def test_wgrad_of_random_values(tokens, m, k, io):
    """Bound: a sum of T terms in fp32, in any order and with any rounding of each addition, is
    within T 2^-23 sum |terms|; with blocked sums far less: a hundredth of it is asked for, and
    never less than 64 additions' worth."""
    g = torch.Generator().manual_seed(6)
    gv = torch.randn(tokens, m, generator=g).to(DT[io])
    x = torch.randn(tokens, k, generator=g) * torch.exp(torch.randn(k, generator=g))
    q, e = ref.quantise(x)
    X = ref.kept(q, e)
    got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda())).cpu().double()
    want, size = gv.double().t() @ X, gv.double().abs().t() @ X.abs()
    assert bool(((got - want).abs() <= max(64, tokens / 100) * 2.0 ** -23 * size).all())


def test_wgrad_of_a_strided_gradient_with_a_bad_block():
    g = torch.Generator().manual_seed(7)
    wide = torch.randn(200, 300, generator=g).bfloat16()
    x = torch.randn(200, 128, generator=g)
    x[77, 40] = float("inf")
    c = block.ssm_ckpt8_save(x.cuda())
    for lead in (0, 8, 3):
        got = block.ssm_ckpt8_wgrad(wide.cuda()[:, lead:lead + 144], c).cpu().double()
        X = ref.through8(x)
        fine = [j for j in range(128) if not 32 <= j < 64]
        want = wide[:, lead:lead + 144].double().t() @ X[:, fine]
        assert torch.allclose(got[:, fine], want, rtol=0, atol=64 * 2.0 ** -23 * 200 * 4 * 4)
        assert bool(torch.isnan(got[:, 32:64]).all())  # the infinity's block is NaN, no other


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wgrad_same_bits_every_time_status_and_workspace(io):
    g = torch.Generator().manual_seed(8)
    gv = torch.randn(3000, 136, generator=g).to(DT[io]).cuda()
    c = block.ssm_ckpt8_save(torch.randn(3000, 264, generator=g).cuda())
    ws = torch.full((block.ssm_ckpt8_wgrad_workspace_size(3000, 136, 264, block._IO[gv.dtype]),),
                    0xff, dtype=torch.uint8, device="cuda")
    first = block.ssm_ckpt8_wgrad(gv, c, ws=ws)
    assert binding.ssm_scan_status(ws) == binding.SSM_OK
    side = torch.cuda.Stream()
    again = block.ssm_ckpt8_wgrad(gv, c, stream=side)
    side.synchronize()
    assert torch.equal(first, again)
    with pytest.raises(ValueError, match="workspace"):
        block.ssm_ckpt8_wgrad(gv, c, ws=ws[:128])
    with pytest.raises(ValueError, match="x8 must hold"):
        block.ssm_ckpt8_wgrad(gv[:-1], c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wgrad_of_long_sums_of_one_sign(io):
    """Where every addition could lose up to 2^-23 of the sum to one side, 32768 tokens of positive
    terms accumulated 16 at a time would lose up to 2048 2^-23 = 2.4e-4.  The accumulator is emptied
    every 1024 tokens into sums rounded to nearest: at most 64 2^-23 = 7.7e-6 in each part, and 96
    additions of parts at 2^-24 (three terms of g), 5.8e-6."""
    g = torch.Generator().manual_seed(9)
    gv = (1.0 + torch.rand(32768, 136, generator=g)).to(DT[io])
    q = torch.randint(64, 128, (32768, 272), generator=g).to(torch.int8)
    e = torch.full((32768, 9), 127, dtype=torch.uint8)
    got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda())).cpu().double()
    want = gv.double().t() @ ref.kept(q, e)
    assert float(((got - want).abs() / want).max()) < 1.4e-5


def test_wgrad_of_large_and_not_finite_gradients():
    """fp32 g at the ends of its range is split exactly; infinities and NaN reach their columns."""
    gv = torch.ones(70, 24)
    gv[3, 1], gv[5, 2] = torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max
    gv[7, 3], gv[9, 4] = float("inf"), float("nan")
    gv[:, 5] = 2.0 ** -120 * (1.0 + 2.0 ** -23)
    c = block.ssm_ckpt8_save(torch.full((70, 32), 0.25).cuda())
    got = block.ssm_ckpt8_wgrad(gv.cuda(), c).cpu()
    want = gv.double().t() @ torch.full((70, 32), 0.25, dtype=torch.float64)
    fine = [i for i in range(24) if i not in (3, 4)]
    assert torch.allclose(got[fine].double(), want[fine], rtol=1e-5, atol=0)
    assert bool(torch.isinf(got[3]).all()) and bool(torch.isnan(got[4]).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,m,k", [(70, 24, 96), (300, 136, 264), (65, 8, 33), (1500, 264, 72)])
def test_wgrad_of_checkpoints_with_rows_of_zeros(tokens, m, k, io):
    """Zeros for padding, scale bytes and all, add nothing: the same bits as zeros with any scale."""
    gv, q, e = _exact_case(tokens, m, k, DT[io], seed=22)
    q[tokens // 3:tokens // 2], e[tokens // 3:tokens // 2] = 0, 0
    e[:, 0][q[:, :32].abs().sum(1) == 0] = 0
    q[-1], e[-1] = 0, 5
    want = gv.double().t() @ ref.kept(q, e)
    got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda()))
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_wgrad_of_the_smallest_scales(io):
    """q 2^(e - 133) with e of 0 .. 4, subnormal steps, times 2^100: products are multiples of 2^-33
    below 2^-22, sums of 64 of them below 2^-16, so that fp32 holds every partial sum exactly."""
    g = torch.Generator().manual_seed(23)
    gv = ((torch.randint(0, 2, (64, 40), generator=g) * 2 - 1) * 2.0 ** 100).to(DT[io])
    q = torch.randint(-127, 128, (64, 96), generator=g).to(torch.int8)
    e = torch.randint(0, 5, (64, 3), generator=g).to(torch.uint8)
    got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda())).cpu().double()
    assert torch.equal(got, gv.double().t() @ ref.kept(q, e))


def test_wgrad_of_every_scale_byte():
    """One token: d_W is g times the kept values, in one product each, exact within fp32's normal
    numbers (g = 2^60 for the small half of the scales)."""
    g = torch.Generator().manual_seed(24)
    for power, first in ((60, 0), (0, 128)):
        q = torch.randint(-127, 128, (1, 128 * 32), generator=g).to(torch.int8)
        e = torch.arange(first, first + 128)[None].to(torch.uint8)
        gv = torch.full((1, 8), 2.0 ** power).bfloat16()
        got = block.ssm_ckpt8_wgrad(gv.cuda(), block.Ckpt8(q.cuda(), e.cuda())).cpu().double()
        want = gv.double().t() @ ref.kept(q, e)
        assert torch.allclose(got, want, rtol=0, atol=0, equal_nan=True)


def _off(t, elements):
    """The same values on the GPU, ``elements`` past an aligned address."""
    wide = torch.zeros(t.numel() + elements, dtype=t.dtype, device="cuda")
    wide[elements:] = t.reshape(-1).cuda()
    return wide[elements:].view(t.shape)


# (type of g, m, k, row stride of g, offsets of g and q in elements, what the size query is told)
ALIGNED = [("f32", 12, 512, 0, 0, 0, 1), ("f32", 12, 512, 516, 0, 0, 1), ("f32", 64, 512, 0, 3, 0, 1),
           ("f32", 40, 48, 41, 1, 0, 1), ("bf16", 64, 512, 72, 0, 0, 1), ("bf16", 64, 512, 0, 8, 16, 1),
           ("bf16", 64, 512, 68, 0, 0, 0), ("bf16", 64, 512, 0, 1, 0, 0), ("bf16", 64, 512, 0, 0, 5, 0),
           ("f32", 64, 512, 0, 0, 8, 0), ("bf16", 20, 33, 0, 0, 0, 0)]


@pytest.mark.parametrize("io,m,k,ld,off_g,off_q,aligned", ALIGNED)
def test_wgrad_takes_the_workspace_that_the_header_asks_for(io, m, k, ld, off_g, off_q, aligned):
    tokens = 300
    gv, q, e = _exact_case(tokens, m, k, DT[io], seed=25)
    rows = torch.zeros(tokens, ld or m, dtype=gv.dtype)
    rows[:, :m] = gv
    g, q8, e8 = _off(rows, off_g), _off(q, off_q), e.cuda()
    L = block.lib()
    n = L.ssm_ckpt8_wgrad_workspace_size(tokens, m, k, block._IO[gv.dtype], aligned)
    ws = torch.full((n + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    out = torch.full((m, k), float("nan"), device="cuda")
    rc = L.ssm_ckpt8_wgrad(g.data_ptr(), ld, q8.data_ptr(), e8.data_ptr(), out.data_ptr(), tokens, m, k,
                           block._IO[gv.dtype], 0, ws.data_ptr(), n,
                           torch.cuda.current_stream().cuda_stream)
    assert rc == binding.SSM_OK
    assert torch.equal(out.cpu().double(), gv.double().t() @ ref.kept(q, e))
    assert bool((ws[n:] == 0x5a).all())
    # and through the binding, which asks for as much
    got = block.ssm_ckpt8_wgrad(g[:, :m], block.Ckpt8(q8, e8), ws=ws[:n])
    assert torch.equal(got, out)
