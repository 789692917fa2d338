"""Edges of the 8-bit checkpoint operators: the tails of the activation
functions, roundings counted one by one, every code in the weight gradient,
and sizes of more than one launch.

u(dtype) is half a step of a type relative to the value, as in
test_gpu_ckpt8.py, whose definitions in 64 bits are used here too."""
import math

import pytest
import torch

import ckpt8_ref as ref
from gpu_util import say
from test_gpu_ckpt8 import LEAST, U, assert_close, gen, randn, to_ck

pytestmark = pytest.mark.gpu

FORMATS = [ref.INT8, ref.E4M3]


@pytest.fixture(scope="module")
def tlc():
    from gradient_compression_distributed_lc_amd import tlc
    return tlc


# In 16 bits x*x is exact (at most 22 bits), so P(x) = exp(-x^2/2) * h(|x|) is
# off by the exponent's two roundings (constant and product: x^2/2 * 1.5 *
# 2^-24), and by less than 12 * 2^-24 for the hardware's exp2 and reciprocal,
# the fit (1.4 * 2^-24) and the polynomial's roundings.
def tail_bound(x64):
    return (0.75 * x64 * x64 + 12) * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gelu_in_the_negative_tail_is_right_relative_to_its_value(tlc, dtype):
    """Every value of the type between -13 and -3: f and f' fall to 1e-37 there, and each keeps the type's precision."""
    x = torch.arange(-13.0, -3.0, 2.0 ** -9).to(dtype).unique()
    x = torch.nn.functional.pad(x, (0, -x.numel() % 32), value=-3.0).view(-1, 32)  # sorted: a group is a short range
    rows, cols = x.shape
    for fmt in FORMATS:
        say(f"case gelu tail {rows}x{cols} {dtype} format {fmt}")
        b = torch.full_like(x, 2.0)
        y, ca, cb = tlc.ckpt8_act(x.cuda(), ref.GELU, fmt, b=b.cuda())
        want = ref.act(ref.GELU, x.double())[0] * 2
        assert_close(y, want, (U[dtype] * 1.01 + tail_bound(x.double())) * want.abs() + LEAST[dtype], "y")
        # the gradients and y in 8 bits, at the checkpoint's values
        dy = torch.ones(rows, cols, dtype=torch.float32, device="cuda").to(dtype)
        da, db, cy = tlc.ckpt8_act_grad(dy, ref.GELU, ca, cb, want_y=True)
        a = ref.decode(*ref.encode(x.double(), fmt), fmt, cols)
        f, slope = ref.act(ref.GELU, a)
        assert_close(db, f, (U[dtype] * 1.01 + tail_bound(a)) * f.abs() + LEAST[dtype], "db")
        # f' = P + x*phi: |x*phi| is above nine times P, so what either is off by counts 10/8 of the sum at most
        want = 2 * slope
        assert_close(da, want, (U[dtype] * 1.01 + 1.25 * (tail_bound(a) + 4 * 2.0 ** -24)) * want.abs() + LEAST[dtype],
                     "da")
        y64 = 2 * f
        codes, scales = ref.encode(y64, fmt)
        got_scales = cy.scales.cpu()
        assert torch.equal(got_scales, scales)
        s = torch.exp2(scales[:, :1].double() - 127)
        half = s / 2 if fmt == ref.INT8 else torch.maximum(y64.abs() * 2.0 ** -4, s * 2.0 ** -10)
        got = ref.decode(cy.codes.cpu(), got_scales, fmt, cols)
        assert ((got - y64).abs() <= half * 1.0001 + tail_bound(a) * y64.abs()).all(), "y in 8 bits"


# P falls as e^-k: k = x^2/2 (gelu), -u (gelu_tanh), -x (silu).  An exponent of
# at most 8 roundings moves it by 8k * 2^-24 of itself, and what else is done to
# it is below 16 roundings; f' has two parts, and for x <= -3 their sum is at
# least 1/1.6 of the larger.  Where P is below 2^-126 it may be 0: |x| <= 88
# times that.


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", [ref.GELU, ref.GELU_TANH, ref.SILU])
def test_activations_in_the_negative_tail(tlc, kind, dtype):
    low = {ref.GELU: -13.0, ref.GELU_TANH: -10.0, ref.SILU: -87.0}[kind]
    x = torch.linspace(low, -3.0, 4096).to(dtype).view(-1, 32)
    rows, cols = x.shape
    floor = 2.0 ** -119 + LEAST[dtype]

    def act(a):
        """f and f' as ref.act has them, but without tanh's cancellation, and the exponent k."""
        if kind != ref.GELU_TANH:
            return (*ref.act(kind, a), a * a / 2 if kind == ref.GELU else -a)
        k = 2 * math.sqrt(2 / math.pi)
        u = k * (a + 0.044715 * a ** 3)
        p, q = torch.sigmoid(u), torch.sigmoid(-u)
        return a * p, p + a * p * q * k * (1 + 0.134145 * a * a), -u

    for fmt in FORMATS:
        say(f"case tail of {kind} {rows}x{cols} {dtype} format {fmt}")
        y, c, _ = tlc.ckpt8_act(x.cuda(), kind, fmt)
        want, _, k = act(x.double())
        assert_close(y, want, (U[dtype] * 1.01 + (16 + 8 * k) * 2.0 ** -24) * want.abs() + floor, "y")
        ones = tlc.ckpt8_pack(torch.ones(rows, cols, device="cuda"), fmt)
        da, db, _ = tlc.ckpt8_act_grad(torch.ones_like(x).cuda(), kind, c, ones)
        f, slope, k = act(ref.decode(*ref.encode(x.double(), fmt), fmt, cols))
        off = (16 + 8 * k) * 2.0 ** -24
        assert_close(db, f, (U[dtype] * 1.01 + off) * f.abs() + floor, "db")
        assert_close(da, slope, (U[dtype] * 1.01 + 1.6 * off) * slope.abs() + floor, "da")


def test_gelu_tanh_gradient_in_fp32_counts_roundings(tlc):
    """f' = p + x*u'*p*q with p and q the logistic function of u and -u, both without a cancellation: u (below 4
    roundings) moves p by p*q*|u| of them and p*q by as much of itself, and the products round a few times more.
    1 - p taken from p rounded to 24 bits would be off by x*u'*2^-25, hundreds of roundings of the result."""
    x = torch.cat([torch.linspace(-9, 9, 2048), torch.linspace(-40, 40, 2048)]).view(-1, 32)
    k, e = math.sqrt(2 / math.pi), 2.0 ** -24
    for fmt in FORMATS:
        say(f"case gelu_tanh gradient {tuple(x.shape)} format {fmt}")
        c = tlc.ckpt8_pack(x.cuda(), fmt)
        a = ref.decode(*ref.encode(x.double(), fmt), fmt, 32)
        da, _, _ = tlc.ckpt8_act_grad(torch.ones_like(x).cuda(), ref.GELU_TANH, c)
        u = 2 * k * (a + 0.044715 * a ** 3)
        p, q = torch.sigmoid(u), torch.sigmoid(-u)
        part = a * 2 * k * (1 + 3 * 0.044715 * a * a) * p * q
        want = p + part
        bound = e * (want.abs() + p * (4 + 4 * u.abs() * q) + part.abs() * (12 + 8 * u.abs())) + 2.0 ** -126
        assert_close(da, want, bound, "da")


def test_norm_output_in_fp32_is_rounded_once(tlc):
    """y = sum*rstd*weight from 64 bits: off by half a step, with a weight and without."""
    for k, (rows, cols) in enumerate([(1, 1), (7, 33), (64, 515), (9, 4096), (5, 9000)]):
        say(f"case norm fp32 {rows}x{cols}")
        g = gen(500 + k)
        x, r, w = randn(g, rows, cols), randn(g, rows, cols, scale=3.0), 1 + randn(g, cols, scale=0.3)
        total = x + r
        _, n = ref.norm(total.double(), float(torch.tensor(1e-5)))
        for fmt in (None, *FORMATS):
            for weight in (w, None):
                _, y, _, _ = tlc.ckpt8_norm(x.cuda(), None if weight is None else weight.cuda(), 1e-5, fmt,
                                            residual=r.cuda())
                want = n if weight is None else n * weight.double()
                assert_close(y, want, want.abs() * 2.0 ** -24 * 1.0001 + LEAST[torch.float32], "y")


# ---- every code in the weight gradient ----------------------------------------


def one_hot(rows, n, dtype):
    dy = torch.zeros(rows, n, dtype=dtype)
    dy[torch.arange(rows), torch.arange(rows) % n] = 1.0
    return dy


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_weight_gradient_reads_every_code_at_every_scale(tlc, fmt, dtype):
    """dy of one 1 a row: dw is the checkpoint's values themselves, from every code at the least, the largest and all
    scales between, in the small tile and in the large one."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127] if fmt == ref.E4M3 else codes[codes != 128]
    codes = torch.nn.functional.pad(codes, (0, 256 - codes.numel())).view(1, 256)
    lo, hi = ref.LOW[fmt] + 127, ref.HIGH[fmt] + 127
    scales = torch.arange(lo, hi + 1, dtype=torch.uint8)
    rows = scales.numel()
    for n, wide in ((rows, 1), (4096, 16)):
        say(f"case weight_grad codes {rows}x{n}x{256 * wide} {dtype} format {fmt}")
        all_codes, all_scales = codes.repeat(rows, wide), scales.view(-1, 1).repeat(1, 8 * wide)
        want = ref.decode(all_codes, all_scales, fmt, 256 * wide)
        got = tlc.ckpt8_weight_grad(one_hot(rows, n, dtype).cuda(), to_ck(tlc, all_codes, all_scales, 256 * wide, fmt))
        assert torch.equal(got[:rows].cpu().double(), want)
        assert not got[rows:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", FORMATS)
def test_weight_gradient_of_groups_that_are_not_finite(tlc, fmt, dtype):
    """A group with scale byte 255 makes its columns of dw NaN, whatever dy is there; the others are as without it.
    The small tile, in one part and in slices, and the large one."""
    for rows, n, cols in ((70, 40, 100), (5000, 130, 260), (330, 4096, 4096)):
        say(f"case weight_grad not finite {rows}x{n}x{cols} {dtype} format {fmt}")
        x = torch.randint(-7, 8, (rows, cols), generator=gen(1)).float()
        dy = torch.randint(-3, 4, (rows, n), generator=gen(2)).to(dtype).cuda()
        want = tlc.ckpt8_weight_grad(dy, tlc.ckpt8_pack(x.cuda(), fmt))
        nan = torch.zeros(cols, dtype=torch.bool)
        for row, col, v in ((11, 50, math.inf), (rows - 1, cols - 1, math.nan), (40, 2, -math.inf)):
            x[row, col] = v
            nan[col // 32 * 32:col // 32 * 32 + 32] = True
        c = tlc.ckpt8_pack(x.cuda(), fmt)
        assert int((c.scales == 255).sum()) == 3
        got = tlc.ckpt8_weight_grad(dy, c)
        nan = nan.cuda()
        assert torch.isnan(got[:, nan]).all()
        assert torch.equal(got[:, ~nan], want[:, ~nan])


# ---- more than one launch ---------------------------------------------------
#
# HIP refuses a launch of 2^32 threads; the elementwise calls give a thread two
# units of eight columns (one in the gated gradient), the norm a row of up to
# 512 columns to a wavefront, the weight gradient a tile to 512 threads.


def ends(n, k=1000):
    """The first and last k rows, and k around the middle."""
    return [slice(0, k), slice(n // 2 - k, n // 2), slice(n - k, n)]


def rows_of(c, at):
    return type(c)(c.codes[at], c.scales[at], c.cols, c.format)


def test_elementwise_calls_of_more_than_one_launch(tlc):
    rows = 2 ** 31 - 1  # four units a row
    say(f"case elementwise {rows}x1")
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    for at in ends(rows):
        x[at] = torch.linspace(-3, 3, 1000, device="cuda").to(torch.bfloat16).unsqueeze(1)
    c = tlc.ckpt8_pack(x, ref.INT8)
    for at in ends(rows):
        alone = tlc.ckpt8_pack(x[at], ref.INT8)
        assert torch.equal(c.codes[at], alone.codes) and torch.equal(c.scales[at], alone.scales)
    y = tlc.ckpt8_unpack(c)
    for at in ends(rows):
        assert torch.equal(y[at], tlc.ckpt8_unpack(rows_of(c, at)))
    tlc.ckpt8_act_grad(x, ref.SILU, c, da=y)
    for at in ends(rows):
        assert torch.equal(y[at], tlc.ckpt8_act_grad(x[at], ref.SILU, rows_of(c, at))[0])
    c.codes.zero_()
    tlc.ckpt8_act(x, ref.SILU, ref.INT8, y=y, a_out=c)
    for at in ends(rows):
        want, alone, _ = tlc.ckpt8_act(x[at], ref.SILU, ref.INT8)
        assert torch.equal(y[at], want) and torch.equal(c.codes[at], alone.codes)


def test_gated_gradient_of_more_than_one_launch(tlc):
    rows = 2 ** 30 + 5
    say(f"case gated gradient {rows}x1")
    a = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    for at in ends(rows):
        a[at] = torch.linspace(-3, 3, 1000, device="cuda").to(torch.bfloat16).unsqueeze(1)
    c = tlc.ckpt8_pack(a, ref.E4M3)
    da, db, cy = tlc.ckpt8_act_grad(a, ref.GELU, c, c, want_y=True)
    for at in ends(rows):
        want = tlc.ckpt8_act_grad(a[at], ref.GELU, rows_of(c, at), rows_of(c, at), want_y=True)
        assert torch.equal(da[at], want[0]) and torch.equal(db[at], want[1])
        assert torch.equal(cy.codes[at], want[2].codes) and torch.equal(cy.scales[at], want[2].scales)


def test_norm_of_more_than_one_launch(tlc):
    rows, cols = 2 ** 26 + 5, 2
    say(f"case norm {rows}x{cols}")
    x = torch.ones(rows, cols, device="cuda")
    r = torch.ones(rows, cols, device="cuda")
    for at in ends(rows):
        r[at] = randn(gen(at.stop % 7), 1000, cols).cuda()
    w = torch.tensor([0.5, 3.0], device="cuda")
    total, y, c, rstd = tlc.ckpt8_norm(x, w, 1e-5, ref.INT8, residual=r)
    for at in ends(rows):
        t1, y1, c1, r1 = tlc.ckpt8_norm(x[at], w, 1e-5, ref.INT8, residual=r[at])
        assert torch.equal(total[at], t1) and torch.equal(y[at], y1) and torch.equal(rstd[at], r1)
        assert torch.equal(c.codes[at], c1.codes) and torch.equal(c.scales[at], c1.scales)
    # its gradient walks over the rows with a bounded number of blocks
    dx, _ = tlc.ckpt8_norm_grad(r, c, rstd, w)
    for at in ends(rows):
        assert torch.equal(dx[at], tlc.ckpt8_norm_grad(r[at], rows_of(c, at), rstd[at], w)[0])


def test_weight_gradient_of_more_than_one_launch(tlc):
    cols = 2 ** 30 + 300  # 2^23 + 3 tiles of 128
    say(f"case weight_grad 1x1x{cols}")
    x = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    for at in ends(cols):
        x[0, at] = torch.randint(-7, 8, (1000,), generator=gen(at.stop % 7)).cuda().to(torch.bfloat16)
    c = tlc.ckpt8_pack(x, ref.INT8)
    dy = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = tlc.ckpt8_weight_grad(dy, c)
    for at in ends(cols):
        assert torch.equal(dw[0, at], 3 * x[0, at].float())
    assert float(dw.min()) == -21.0 and float(dw.max()) == 21.0
    # no rows: the same matrix is set to 0
    none = tlc.Checkpoint8(c.codes[:0], c.scales[:0], cols, ref.INT8)
    tlc.ckpt8_weight_grad(dy[:0], none, dw=dw)
    assert not dw.any()
