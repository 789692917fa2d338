"""The 8-bit checkpoint operators on the GPU against their definitions in 64
bits: bit for bit where the result is defined so (codes, scales, decoded
values, exact sums), otherwise within bounds derived from the roundings.

u(dtype) is half a step of a type relative to the value: 2^-8 (bf16), 2^-11
(fp16), 2^-24 (fp32); a stored result is off by u of its value, plus half the
least step of the type near zero."""
import math

import pytest
import torch

import ckpt8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
FORMATS = [ref.INT8, ref.E4M3]
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def tlc():
    from gradient_compression_distributed_lc_amd import tlc
    return tlc


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def strided(t: torch.Tensor, pad: int, offset: int = 0) -> torch.Tensor:
    """t on the GPU as a view with rows `pad` further apart, starting `offset` elements in; the gaps hold NaN."""
    rows, cols = t.shape
    flat = torch.full((offset + rows * (cols + pad),), math.nan, dtype=t.dtype, device="cuda")
    v = flat[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def gaps(v: torch.Tensor) -> torch.Tensor:
    """What lies between the rows of a view made by strided()."""
    rows, cols = v.shape
    return torch.as_strided(v, (rows, v.stride(0) - cols), (v.stride(0), 1), v.storage_offset() + cols)


def to_ck(tlc, codes, scales, cols, fmt):
    return tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, fmt)


def assert_ck(c, codes, scales, label):
    assert torch.equal(c.scales.cpu(), scales), (label, "scales")
    got = c.codes.cpu()
    if not torch.equal(got, codes):
        at = (got != codes).nonzero()[0].tolist()
        raise AssertionError(f"{label}: code at {at}: got {int(got[tuple(at)])}, want {int(codes[tuple(at)])}")


def assert_close(got, want, bound, label):
    got = got.cpu().double()
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{label}: at {at}: got {float(got[tuple(at)])!r}, want {float(want[tuple(at)])!r}, "
                             f"bound {float(bound.expand_as(want)[tuple(at)]):.3g} ({int(bad.sum())} values)")


# ---- the format -------------------------------------------------------------

SHAPES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (4, 128), (7, 129), (1, 4096), (65, 515), (130, 1000), (257, 8),
          (600, 40), (3, 16391)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_pack_and_unpack(tlc, fmt, dtype):
    for k, (rows, cols) in enumerate(SHAPES):
        say(f"case pack {rows}x{cols} {dtype} format {fmt}")
        x = randn(gen(k), rows, cols, dtype=dtype, scale=10.0 ** (k % 7 - 3))
        codes, scales = ref.encode(x.double(), fmt)
        c = tlc.ckpt8_pack(x.cuda(), fmt)
        assert_ck(c, codes, scales, (rows, cols))
        # rows further apart, starting at an odd element
        assert_ck(tlc.ckpt8_pack(strided(x, 3, 1), fmt), codes, scales, (rows, cols, "strided"))
        want = ref.decode(codes, scales, fmt, cols)
        for out in DTYPES:
            y = strided(torch.zeros(rows, cols, dtype=out), 5, 1)
            got = tlc.ckpt8_unpack(c, y=y)
            assert got is y
            assert torch.equal(y.cpu().double(), want.to(out).double()), (rows, cols, out)
            assert torch.isnan(gaps(y)).all(), "a gap between rows was written"


@pytest.mark.parametrize("fmt", FORMATS)
def test_group_borders_and_special_values(tlc, fmt):
    """Each row one group: largest magnitudes at, just below and just above every border of the scale, zeros of both
    signs, denormals, the type's limits, infinities and NaN anywhere in the group."""
    top = ref.LARGEST[fmt]
    limit = torch.finfo(torch.float32).max
    rows = []
    for k in list(range(-149, 128, 3)) + [-127, -126, -125, 119, 120, 121, 126, 127]:
        for m in (1.0, top / 2.0 ** math.floor(math.log2(top))):
            for nudge in (-1, 0, 1):
                v = torch.tensor(m * 2.0 ** k, dtype=torch.float64).float()
                if nudge and torch.isfinite(v):
                    v = torch.nextafter(v, torch.tensor(math.inf if nudge > 0 else 0.0))
                rows.append(torch.cat([v.view(1), v.view(1) * torch.linspace(-1, 1, 31)]))
    for a in (0.0, -0.0, 2.0 ** -149, -2.0 ** -140, limit, -limit, math.inf, -math.inf, math.nan):
        for at in (0, 7, 8, 31):
            for rest in (0.0, 1.5, -limit):
                r = torch.full((32,), rest)
                r[at] = a
                rows.append(r)
    x = torch.stack([r for r in rows if not (r.numel() != 32)])
    say(f"case borders: {x.shape[0]} groups")
    codes, scales = ref.encode(x.double(), fmt)
    if fmt == ref.INT8:  # a zero has no sign there; in e4m3 it keeps it
        assert (codes != 128).all()
    c = tlc.ckpt8_pack(x.cuda(), fmt)
    assert_ck(c, codes, scales, "borders")
    want = ref.decode(codes, scales, fmt, 32)
    for dtype in (torch.float32, torch.bfloat16):
        got = tlc.ckpt8_unpack(c, dtype).cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0)), "decoded values are exact"
    assert torch.isfinite(want[scales[:, 0] != 255]).all()
    # the same groups in 16 bits
    for dtype in (torch.float16, torch.bfloat16):
        h = x.to(dtype)
        assert_ck(tlc.ckpt8_pack(h.cuda(), fmt), *ref.encode(h.double(), fmt), dtype)


@pytest.mark.parametrize("fmt", FORMATS)
def test_unpack_every_code(tlc, fmt):
    codes = torch.arange(256, dtype=torch.uint8)
    if fmt == ref.E4M3:
        codes = codes[(codes & 127) != 127]
    else:
        codes = codes[codes != 128]
    codes = torch.nn.functional.pad(codes, (0, -codes.numel() % 32)).view(-1, 32).repeat(4, 1)
    scales = torch.zeros(codes.shape[0], 4, dtype=torch.uint8)
    lo, hi = ref.LOW[fmt] + 127, ref.HIGH[fmt] + 127
    scales[:, 0] = torch.tensor([lo, 90, 130, hi], dtype=torch.uint8).repeat_interleave(codes.shape[0] // 4)
    got = tlc.ckpt8_unpack(to_ck(tlc, codes, scales, 32, fmt), torch.float32)
    assert torch.equal(got.cpu().double(), ref.decode(codes, scales, fmt, 32))


# ---- activation functions ---------------------------------------------------
#
# P (f = x*P) in fp32 is off by less than 2^-20: 7.5e-8 of the rational form and
# a few roundings of 2^-24 to 2^-22.  So y is off by u|y| + 2^-20 |x b|.  The
# slope adds x*P', whose parts are below 1, and x*(1-P)*u' where 1-P is off by
# 2^-24 while x*u' is below 40: below 2^-18 in all.


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", [ref.GELU, ref.GELU_TANH, ref.SILU])
def test_act_and_gradient(tlc, kind, gated, dtype):
    for k, (rows, cols) in enumerate([(1, 1), (3, 33), (66, 257), (9, 1031), (40, 4096)]):
        fmt = FORMATS[k % 2]
        say(f"case act {kind} gated {gated} {rows}x{cols} {dtype} format {fmt}")
        g = gen(10 * k + kind)
        fused = randn(g, rows, 2 * cols, dtype=dtype, scale=3.0)
        fused[0, 0] = 0.0
        if cols > 8:
            fused[0, 1:5] = torch.tensor([30.0, -30.0, 1000.0, -1000.0])
        dy = randn(g, rows, cols, dtype=dtype)
        d = fused.cuda()
        a, b = d[:, :cols], d[:, cols:] if gated else None
        a64, b64 = fused[:, :cols].double(), fused[:, cols:].double() if gated else torch.ones(1, dtype=torch.float64)
        y = strided(torch.zeros(rows, cols, dtype=dtype), 2, 1)
        got, ca, cb = tlc.ckpt8_act(a, kind, fmt, b=b, y=y)
        f, _ = ref.act(kind, a64)
        want = f * b64
        assert_close(got, want, U[dtype] * want.abs() * 1.01 + 2.0 ** -20 * (a64 * b64).abs() + LEAST[dtype], "y")
        assert torch.isnan(gaps(y)).all()
        codes, scales = ref.encode(a64, fmt)
        assert_ck(ca, codes, scales, "a")
        av, bv = ref.decode(codes, scales, fmt, cols), torch.ones(1, dtype=torch.float64)
        if gated:
            codes, scales = ref.encode(b64, fmt)
            assert_ck(cb, codes, scales, "b")
            bv = ref.decode(codes, scales, fmt, cols)
        else:
            assert cb is None
        # the gradient, from the checkpoints
        da = strided(torch.zeros(rows, cols, dtype=dtype), 1, 1)
        got_a, got_b, cy = tlc.ckpt8_act_grad(strided(dy, 3, 1), kind, ca, cb, da=da, want_y=True)
        dy64 = dy.double()
        f, slope = ref.act(kind, av)
        want = dy64 * bv * slope
        assert_close(got_a, want, U[dtype] * want.abs() * 1.01 + 2.0 ** -18 * (dy64 * bv).abs() + LEAST[dtype], "da")
        assert torch.isnan(gaps(da)).all()
        if gated:
            want = dy64 * f
            assert_close(got_b, want, U[dtype] * want.abs() * 1.01 + 2.0 ** -20 * (dy64 * av).abs() + LEAST[dtype],
                         "db")
        else:
            assert got_b is None
        # y again in 8 bits: within half a step of its group, plus what fp32 is off
        y64 = f * bv
        groups = -(-cols // 32)
        padded = torch.nn.functional.pad(y64, (0, groups * 32 - cols)).view(rows, groups, 32)
        noise = torch.nn.functional.pad(2.0 ** -20 * (av * bv).abs(), (0, groups * 32 - cols)).view(rows, groups, 32)
        got_y = torch.nn.functional.pad(ref.decode(cy.codes.cpu(), cy.scales.cpu(), fmt, cols),
                                        (0, groups * 32 - cols)).view(rows, groups, 32)
        amax = padded.abs().amax(2, keepdim=True)
        least = torch.full_like(amax, 2.0 ** (ref.LOW[fmt] + (0 if fmt == ref.INT8 else -9)))
        if fmt == ref.INT8:  # a step is at most amax/63.5 (127 codes, scale less than twice the least that fits)
            half = amax / 63.5 / 2
        else:  # u of e4m3, or half a step of 2^-9 at a scale below amax/224
            half = torch.maximum(padded.abs() * 2.0 ** -4, amax / 224 * 2.0 ** -10)
        half = torch.maximum(half, least)
        assert ((got_y - padded).abs() <= half * 1.001 + noise * 1.1).all(), "y in 8 bits"
        # not asked for
        assert tlc.ckpt8_act_grad(dy.cuda(), kind, ca, cb)[2] is None


def test_act_gradient_against_differences(tlc):
    """da and db are the slopes of the 64-bit loss sum(dy * f(a)*b) at the checkpoint's values."""
    rows, cols, h = 5, 96, 1e-5
    for kind in (ref.GELU, ref.GELU_TANH, ref.SILU):
        g = gen(kind)
        a, b, dy = (randn(g, rows, cols, scale=2.0) for _ in range(3))
        _, ca, cb = tlc.ckpt8_act(a.cuda(), kind, ref.INT8, b=b.cuda())
        da, db, _ = tlc.ckpt8_act_grad(dy.cuda(), kind, ca, cb)
        av, bv = (tlc.ckpt8_unpack(c, torch.float32).cpu().double() for c in (ca, cb))
        d = dy.double()
        up, down = ref.act(kind, av + h)[0], ref.act(kind, av - h)[0]
        # the difference quotient is off by h^2/6 of a third derivative below 4, and 2^-52/h
        bound = (d * bv).abs() * (2.0 ** -18 + h * h + 2.0 ** -50 / h) + 1e-9
        assert_close(da, d * bv * (up - down) / (2 * h), bound, f"da {kind}")
        assert_close(db, d * ref.act(kind, av)[0], (d * av).abs() * 2.0 ** -20 + 1e-9, f"db {kind}")


def test_act_gradient_in_place_and_nan_groups(tlc):
    rows, cols = 9, 100
    g = gen(3)
    a, b, dy = (randn(g, rows, cols, dtype=torch.bfloat16) for _ in range(3))
    a[2, 40] = math.nan
    a[3, 70] = math.inf
    _, ca, cb = tlc.ckpt8_act(a.cuda(), ref.SILU, ref.INT8, b=b.cuda())
    want_a, want_b, _ = tlc.ckpt8_act_grad(dy.cuda(), ref.SILU, ca, cb)
    d = dy.cuda()
    got_a, got_b, _ = tlc.ckpt8_act_grad(d, ref.SILU, ca, cb, da=d)
    assert got_a.data_ptr() == d.data_ptr()
    assert torch.equal(got_a.nan_to_num(9.0), want_a.nan_to_num(9.0))
    assert torch.equal(got_b.nan_to_num(9.0), want_b.nan_to_num(9.0))
    nan = torch.zeros(rows, cols, dtype=torch.bool)
    nan[2, 32:64] = True   # the whole group of a value that is not finite
    nan[3, 64:96] = True
    for kind in (ref.GELU, ref.GELU_TANH, ref.SILU):
        da, db, _ = tlc.ckpt8_act_grad(dy.cuda(), kind, ca, cb)
        assert torch.equal(torch.isnan(da).cpu(), nan) and torch.equal(torch.isnan(db).cpu(), nan), kind


# ---- norm -------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 7), (2, 32), (5, 100), (70, 512), (33, 515), (6, 1023), (9, 2048), (4, 4096), (3, 5000),
               (2, 8192), (2, 8200), (2, 12001), (1, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_norm(tlc, fmt, dtype):
    eps = 1e-5
    for k, (rows, cols) in enumerate(NORM_SHAPES):
        say(f"case norm {rows}x{cols} {dtype} format {fmt}")
        g = gen(100 + k)
        x, r = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype, scale=4.0)
        w = (1 + randn(g, cols, scale=0.3)).to((torch.float32, dtype)[k % 2])
        total = (x.float() + r.float()).to(dtype)
        rstd, n = ref.norm(total.double(), float(torch.tensor(eps)))
        for weighted in (False, True):
            t = strided(torch.zeros(rows, cols, dtype=dtype), 1, 1)
            y = strided(torch.zeros(rows, cols, dtype=dtype), 2, 1)
            got_t, got_y, c, got_r = tlc.ckpt8_norm(strided(x, 1, 1), w.cuda(), eps, fmt, residual=strided(r, 3, 1),
                                                    weighted=weighted, total=t, y=y)
            assert torch.equal(got_t.cpu(), total)
            assert torch.isnan(gaps(t)).all() and torch.isnan(gaps(y)).all()
            # fp64 up to one rounding; the mean's order of addition is 2^-40 at most
            assert_close(got_r, rstd, rstd * 2.0 ** -24 * 1.001, "rstd")
            want = n * w.double()
            # n to fp32, times the weight in fp32, to the type
            assert_close(got_y, want, want.abs() * (U[dtype] + 3 * 2.0 ** -24) * 1.01 + LEAST[dtype], "y")
            assert_ck(c, *ref.encode(want if weighted else n, fmt), (rows, cols, weighted))
        # no residual, no weight: the sum is x itself
        rstd, n = ref.norm(x.double(), float(torch.tensor(eps)))
        xd = x.cuda()
        got_t, got_y, c, _ = tlc.ckpt8_norm(xd, None, eps, fmt)
        assert got_t is xd
        assert_ck(c, *ref.encode(n, fmt), (rows, cols, "plain"))
        assert_close(got_y, n, n.abs() * (U[dtype] + 2.0 ** -23) * 1.01 + LEAST[dtype], "y plain")


def test_norm_outputs_that_are_not_asked_for_and_in_place(tlc):
    x, r = randn(gen(1), 40, 300, dtype=torch.bfloat16), randn(gen(2), 40, 300, dtype=torch.bfloat16)
    w = randn(gen(3), 300)
    want = tlc.ckpt8_norm(x.cuda(), w.cuda(), 1e-6, ref.INT8, residual=r.cuda())
    for place in ("x", "residual"):
        xd, rd = x.cuda(), r.cuda()
        got = tlc.ckpt8_norm(xd, w.cuda(), 1e-6, ref.INT8, residual=rd, total=xd if place == "x" else rd)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2].codes, want[2].codes) and torch.equal(got[3], want[3])
    t, y, c, _ = tlc.ckpt8_norm(x.cuda(), w.cuda(), 1e-6, None, residual=r.cuda())
    assert c is None and torch.equal(y, want[1]) and torch.equal(t, want[0])
    t, y, c, _ = tlc.ckpt8_norm(x.cuda(), w.cuda(), 1e-6, ref.INT8, residual=r.cuda(), want_y=False)
    assert y is None and torch.equal(c.codes, want[2].codes)


def test_norm_rows_of_zeros_and_rows_that_are_not_finite(tlc):
    x = randn(gen(4), 6, 96)
    x[0] = 0.0
    x[1, 5] = math.nan
    x[2, 40] = math.inf
    x[3] = 1e-30  # squares vanish in fp32, not in fp64
    x[4] = 1e25   # squares overflow fp32, not fp64
    for fmt in FORMATS:
        _, y, c, rstd = tlc.ckpt8_norm(x.cuda(), None, 1e-12, fmt)
        y, rstd = y.cpu(), rstd.cpu()
        assert (y[0] == 0).all() and (c.scales[0].cpu() == 0).all() and (c.codes[0].cpu() == 0).all()
        assert math.isclose(float(rstd[0]), 1e6, rel_tol=1e-6)
        assert torch.isnan(y[1]).all() and (c.scales[1, :3].cpu() == 255).all()
        # an infinite value: rstd is 0, the finite values 0 and the infinite one NaN
        assert float(rstd[2]) == 0.0 and torch.isnan(y[2, 40]) and int(torch.isnan(y[2]).sum()) == 1
        assert c.scales[2, :3].cpu().tolist() == [0, 255, 0]
        _, n = ref.norm(x[3:].double(), float(torch.tensor(1e-12)))
        codes, scales = ref.encode(n, fmt)
        assert torch.equal(c.codes[3:].cpu(), codes) and torch.equal(c.scales[3:].cpu(), scales)


def test_norm_weight_past_the_largest_scale(tlc):
    """Weighted values past the largest scale are held to the largest code; infinite ones make NaN groups."""
    x = torch.ones(2, 64)
    w = torch.full((64,), 1.0)
    w[3], w[40] = 3.3e38, math.inf
    for fmt in FORMATS:
        _, _, c, _ = tlc.ckpt8_norm(x.cuda(), w.cuda(), 1e-20, fmt, weighted=True)
        _, n = ref.norm(x.double(), float(torch.tensor(1e-20)))
        assert_ck(c, *ref.encode(n * w.double(), fmt), fmt)


# dx = dsum + rstd*(g - n*m), m = mean(g n): g, n, m, the products and the sums
# are fp32: off by (6 + cols/64) roundings of 2^-24 of the largest parts at most;
# dw: a sum of `rows` products in fp32.


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("saved", ["checkpoint", "sum"])
def test_norm_gradient(tlc, saved, dtype):
    for k, (rows, cols) in enumerate(NORM_SHAPES + [(0, 40), (1100, 36), (2500, 130)]):
        fmt = FORMATS[k % 2]
        say(f"case norm_grad {rows}x{cols} {dtype} {saved} format {fmt}")
        g = gen(200 + k)
        total = randn(g, rows, cols, dtype=dtype, scale=3.0)
        dy, dt = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype)
        w = (1 + randn(g, cols, scale=0.3)).to((torch.float32, dtype)[k // 2 % 2]) if k % 4 else None
        _, _, c, rstd = tlc.ckpt8_norm(total.cuda(), None, 1e-5, fmt)
        r64 = rstd.cpu().double()
        if saved == "checkpoint":
            n = ref.decode(c.codes.cpu(), c.scales.cpu(), fmt, cols)
            given = c
        else:
            n = total.double() * r64.unsqueeze(1)
            given = strided(total, 1, 1)
        w64 = w.double() if w is not None else torch.ones(cols, dtype=torch.float64)
        dx = strided(torch.zeros(rows, cols, dtype=dtype), 3, 1)
        base = randn(g, cols)
        got_dx, got_dw = tlc.ckpt8_norm_grad(strided(dy, 1, 1), given, rstd, None if w is None else w.cuda(),
                                             dtotal=strided(dt, 5, 1) if k % 2 else None, dx=dx)
        want_dx, want_dw = ref.norm_grad(dy.double(), n, r64, w64, dt.double() if k % 2 else None)
        gn = (dy.double() * w64).abs()
        part = r64.unsqueeze(1) * (gn + n.abs() * (gn * n.abs()).mean(1, keepdim=True)) + (dt.double().abs() if k % 2
                                                                                          else 0.0)
        assert_close(got_dx, want_dx, U[dtype] * want_dx.abs() * 1.01 + (6 + cols / 64) * 2.0 ** -24 * part
                     + LEAST[dtype], "dx")
        assert torch.isnan(gaps(dx)).all()
        terms = (dy.double().abs() * n.abs()).sum(0)
        bound = (rows + 4) * 2.0 ** -24 * terms + 2.0 ** -149
        assert_close(got_dw, want_dw, bound, "dw")
        again = base.cuda()
        tlc.ckpt8_norm_grad(dy.cuda(), given, rstd, None if w is None else w.cuda(), dw=again, accumulate=True)
        assert_close(again, want_dw + base.double(), bound + 2.0 ** -24 * (want_dw + base.double()).abs() * 1.01,
                     "dw added")
        only_dx, none = tlc.ckpt8_norm_grad(dy.cuda(), given, rstd, None if w is None else w.cuda(), want_dw=False,
                                            dtotal=dt.cuda() if k % 2 else None)
        assert none is None and torch.equal(only_dx, got_dx)


def test_norm_gradient_against_differences(tlc):
    """dx and dw are the slopes of the 64-bit loss sum(dy*norm(x)*w) + sum(dtotal*x)."""
    rows, cols, h, eps = 4, 70, 1e-5, 1e-3
    g = gen(9)
    x, dy, dt = (randn(g, rows, cols) for _ in range(3))
    w = 1 + randn(g, cols, scale=0.3)
    _, _, _, rstd = tlc.ckpt8_norm(x.cuda(), None, eps, None)
    dx, dw = tlc.ckpt8_norm_grad(dy.cuda(), x.cuda(), rstd, w.cuda(), dtotal=dt.cuda())
    x64, e = x.double(), float(torch.tensor(eps))

    def loss(x, w):
        return float((dy.double() * ref.norm(x, e)[1] * w).sum() + (dt.double() * x).sum())

    for r, c in [(0, 0), (1, 31), (2, 33), (3, 69)]:
        d = torch.zeros(rows, cols, dtype=torch.float64)
        d[r, c] = h
        slope = (loss(x64 + d, w.double()) - loss(x64 - d, w.double())) / (2 * h)
        assert abs(float(dx[r, c]) - slope) < 1e-5, (r, c)
        d = torch.zeros(cols, dtype=torch.float64)
        d[c] = h
        slope = (loss(x64, w.double() + d) - loss(x64, w.double() - d)) / (2 * h)
        assert abs(float(dw[c]) - slope) < 1e-5, c


def test_norm_gradient_in_place(tlc):
    total, dy, dt = (randn(gen(k), 30, 200, dtype=torch.bfloat16) for k in range(3))
    _, _, c, rstd = tlc.ckpt8_norm(total.cuda(), None, 1e-5, ref.INT8)
    want, dw = tlc.ckpt8_norm_grad(dy.cuda(), c, rstd, dtotal=dt.cuda())
    for place in ("dy", "dtotal"):
        a, b = dy.cuda(), dt.cuda()
        got, dw2 = tlc.ckpt8_norm_grad(a, c, rstd, dtotal=b, dx=a if place == "dy" else b)
        assert torch.equal(got, want) and torch.equal(dw, dw2)


# ---- weight gradient --------------------------------------------------------

WEIGHT_SHAPES = [(1, 1, 1), (1, 40, 33), (31, 3, 129), (32, 128, 128), (33, 129, 127), (64, 16, 512), (100, 300, 96),
                 (257, 64, 40), (500, 130, 260), (1030, 257, 515), (2300, 128, 64), (777, 515, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_weight_gradient_of_whole_numbers_is_exact(tlc, fmt, dtype):
    """Small whole numbers: every sum is below 2^24 and has one right value, whatever its order."""
    for k, (rows, n, cols) in enumerate(WEIGHT_SHAPES):
        say(f"case weight_grad exact {rows}x{n}x{cols} {dtype} format {fmt}")
        g = gen(300 + k)
        dy = torch.randint(-9, 10, (rows, n), generator=g).to(dtype)
        x = torch.randint(-7, 8, (rows, cols), generator=g).double()
        codes, scales = ref.encode(x, fmt)
        x = ref.decode(codes, scales, fmt, cols)
        want = dy.double().t() @ x
        dw = strided(torch.zeros(n, cols), 3, 1)
        got = tlc.ckpt8_weight_grad(strided(dy, 3, 1), to_ck(tlc, codes, scales, cols, fmt), dw=dw)
        assert torch.equal(got.cpu().double(), want), (rows, n, cols)
        assert torch.isnan(gaps(dw)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_weight_gradient(tlc, fmt, dtype):
    """Products are exact (below 2^-126 aside) and sums fp32, in the matrix cores and between slices: each addition
    rounds or cuts once, at most 2^-23 of the sum of magnitudes."""
    for k, (rows, n, cols) in enumerate(WEIGHT_SHAPES):
        say(f"case weight_grad {rows}x{n}x{cols} {dtype} format {fmt}")
        g = gen(400 + k)
        dy = randn(g, rows, n, dtype=dtype, scale=0.01)
        codes, scales = ref.encode(randn(g, rows, cols, scale=3.0).double(), fmt)
        x = ref.decode(codes, scales, fmt, cols)
        cs = (1 + randn(g, cols, scale=0.3)).to((torch.float32, dtype)[k % 2])
        want, sizes = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
        bound = rows * 2.0 ** -23 * sizes + 2.0 ** -149
        c = to_ck(tlc, codes, scales, cols, fmt)
        assert_close(tlc.ckpt8_weight_grad(dy.cuda(), c), want, bound, "dw")
        got = tlc.ckpt8_weight_grad(dy.cuda(), c, col_scale=cs.cuda())
        c64 = cs.double()
        assert_close(got, want * c64, bound * c64.abs() * 1.01 + 2.0 ** -24 * (want * c64).abs(), "dw scaled")
        base = randn(g, n, cols)
        dw = base.cuda()
        tlc.ckpt8_weight_grad(dy.cuda(), c, dw=dw, accumulate=True)
        assert_close(dw, want + base.double(), bound * 1.01 + 2.0 ** -24 * (want + base.double()).abs() * 1.01,
                     "dw added")
        # the same bits every time
        assert torch.equal(tlc.ckpt8_weight_grad(dy.cuda(), c), tlc.ckpt8_weight_grad(dy.cuda(), c))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_weight_gradient_of_many_tiles_is_exact(tlc, fmt, dtype):
    """Sizes that take the larger tile, alone and in slices, with and without ragged edges; whole numbers, so that
    every sum has one right value (below 2^24)."""
    sizes = [(300, 4000, 4100), (2000, 2100, 2000), (330, 4096, 4096), (700, 2048, 2048), (4096, 2100, 2050),
             (2100, 4000, 4000)]
    for k, (rows, n, cols) in enumerate(sizes):
        say(f"case weight_grad many tiles {rows}x{n}x{cols} {dtype} format {fmt}")
        g = torch.Generator(device="cuda").manual_seed(k)
        dy = torch.randint(-9, 10, (rows, n + 5), generator=g, device="cuda").to(dtype)[:, 3:n + 3]
        x = torch.randint(-7, 8, (rows, cols), generator=g, device="cuda").float()
        c = tlc.ckpt8_pack(x, fmt)
        x = tlc.ckpt8_unpack(c, torch.float32).double()
        want = dy.double().t().contiguous() @ x
        assert torch.equal(tlc.ckpt8_weight_grad(dy, c).double(), want)
        scale = torch.tensor([0.5, 1.0, 2.0, -1.0], device="cuda").repeat(-(-cols // 4))[:cols]
        dw = torch.ones(n, cols + 1, device="cuda")[:, :cols]
        tlc.ckpt8_weight_grad(dy, c, col_scale=scale.to((torch.float32, dtype)[k % 2]), dw=dw, accumulate=True)
        assert torch.equal(dw.double(), want * scale.double() + 1)


def test_norm_of_wide_rows_in_every_variant(tlc):
    """Past 8192 columns, every type with either type of weight and either format."""
    rows, cols = 3, 9001
    for dtype in DTYPES:
        for wt in {torch.float32, dtype}:
            for fmt in FORMATS:
                g = gen(5)
                x, dy = randn(g, rows, cols, dtype=dtype, scale=2.0), randn(g, rows, cols, dtype=dtype)
                w = (1 + randn(g, cols, scale=0.3)).to(wt)
                _, y, c, rstd = tlc.ckpt8_norm(x.cuda(), w.cuda(), 1e-5, fmt)
                r64, n = ref.norm(x.double(), float(torch.tensor(1e-5)))
                assert_ck(c, *ref.encode(n, fmt), (dtype, wt, fmt))
                want = n * w.double()
                assert_close(y, want, want.abs() * (U[dtype] + 3 * 2.0 ** -24) * 1.01 + LEAST[dtype], "y")
                for saved, nv in ((c, ref.decode(c.codes.cpu(), c.scales.cpu(), fmt, cols)), (x.cuda(), None)):
                    r = rstd.cpu().double()
                    nv = x.double() * r.unsqueeze(1) if nv is None else nv
                    dx, dw = tlc.ckpt8_norm_grad(dy.cuda(), saved, rstd, w.cuda())
                    want, want_dw = ref.norm_grad(dy.double(), nv, r, w.double())
                    gn = (dy.double() * w.double()).abs()
                    part = r.unsqueeze(1) * (gn + nv.abs() * (gn * nv.abs()).mean(1, keepdim=True))
                    assert_close(dx, want, U[dtype] * want.abs() * 1.01 + (6 + cols / 64) * 2.0 ** -24 * part
                                 + LEAST[dtype], "dx")
                    assert_close(dw, want_dw, (rows + 4) * 2.0 ** -24 * (dy.double() * nv).abs().sum(0) + 2.0 ** -149,
                                 "dw")


def test_offsets_past_32_bits(tlc):
    """More than 2^32 values: the last rows of the whole are what they are alone."""
    rows, cols, last = 1_100_000, 4096, 300
    say(f"case offsets {rows}x{cols}")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x[-last:] = torch.randint(-7, 8, (last, cols), generator=g, device="cuda").to(torch.bfloat16)
    for fmt in FORMATS:
        c, alone = tlc.ckpt8_pack(x, fmt), tlc.ckpt8_pack(x[-last:], fmt)
        assert torch.equal(c.codes[-last:], alone.codes) and torch.equal(c.scales[-last:], alone.scales)
        y = tlc.ckpt8_unpack(c)
        assert torch.equal(y[-last:], x[-last:]) and torch.equal(y[:last], x[:last])
        del y
    da = tlc.ckpt8_act_grad(x, ref.SILU, c)[0]
    assert torch.equal(da[-last:], tlc.ckpt8_act_grad(x[-last:], ref.SILU, alone)[0])
    del da
    _, y, n8, rstd = tlc.ckpt8_norm(x, None, 1e-5, ref.INT8)
    _, y_alone, n8_alone, rstd_alone = tlc.ckpt8_norm(x[-last:], None, 1e-5, ref.INT8)
    assert torch.equal(y[-last:], y_alone) and torch.equal(n8.codes[-last:], n8_alone.codes)
    assert torch.equal(rstd[-last:], rstd_alone)
    dx, _ = tlc.ckpt8_norm_grad(x, n8, rstd)
    assert torch.equal(dx[-last:], tlc.ckpt8_norm_grad(x[-last:], n8_alone, rstd_alone)[0])
    del y, dx, n8
    # a gradient that is 0 but in the last rows: the sums are those rows' alone
    dy = torch.zeros(rows, 16, dtype=torch.bfloat16, device="cuda")
    dy[-last:] = torch.randint(-9, 10, (last, 16), generator=g, device="cuda").to(torch.bfloat16)
    want = dy[-last:].double().t().contiguous() @ x[-last:].double()
    assert torch.equal(tlc.ckpt8_weight_grad(dy, c).double(), want)


def test_weight_gradient_of_no_rows(tlc):
    for dtype in DTYPES:
        c = tlc.Checkpoint8(torch.empty(0, 64, dtype=torch.uint8, device="cuda"),
                            torch.empty(0, 4, dtype=torch.uint8, device="cuda"), 40, ref.INT8)
        dy = torch.empty(0, 300, dtype=dtype, device="cuda")
        assert (tlc.ckpt8_weight_grad(dy, c) == 0).all()
        dw = torch.ones(300, 40, device="cuda")
        tlc.ckpt8_weight_grad(dy, c, dw=dw, accumulate=True)
        assert (dw == 1).all()
        tlc.ckpt8_weight_grad(dy, c, dw=dw)
        assert (dw == 0).all()


def test_no_rows(tlc):
    for fmt in FORMATS:
        x = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        c = tlc.ckpt8_pack(x, fmt)
        assert c.rows == 0 and tlc.ckpt8_unpack(c).shape == (0, 40)
        y, ca, cb = tlc.ckpt8_act(x, ref.GELU, fmt, b=x)
        da, db, cy = tlc.ckpt8_act_grad(x, ref.GELU, ca, cb, want_y=True)
        assert y.shape == da.shape == db.shape == (0, 40) and cy.rows == 0
        w = torch.ones(40, device="cuda")
        t, y, c, r = tlc.ckpt8_norm(x, w, 1e-5, fmt, residual=x)
        assert t.shape == y.shape == (0, 40) and r.shape == (0,)
        dw = torch.full((40,), 3.0, device="cuda")
        tlc.ckpt8_norm_grad(x, c, r, w, dw=dw, accumulate=True)
        assert (dw == 3).all()
        tlc.ckpt8_norm_grad(x, c, r, w, dw=dw)
        assert (dw == 0).all()


def test_weight_gradient_with_values_that_are_not_finite(tlc):
    """A NaN group or a NaN or infinite dy reaches the columns and rows it multiplies, and no others."""
    rows, n, cols = 70, 40, 100
    for dtype in DTYPES:
        x = randn(gen(5), rows, cols)
        x[11, 50] = math.inf  # group 32..63 of row 11
        c = tlc.ckpt8_pack(x.cuda(), ref.INT8)
        dy = randn(gen(6), rows, n, dtype=dtype)
        dy[3, 7], dy[4, 9] = math.nan, math.inf
        got = tlc.ckpt8_weight_grad(dy.cuda(), c).cpu()
        nan = torch.zeros(n, cols, dtype=torch.bool)
        nan[:, 32:64] = True
        nan[7] = True
        assert torch.isnan(got[nan]).all()
        rest = torch.ones(n, cols, dtype=torch.bool)
        rest[:, 32:64] = False
        rest[7], rest[9] = False, False
        assert torch.isfinite(got[rest]).all()
        assert not torch.isfinite(got[9]).any()


# ---- streams, graphs, refusals ----------------------------------------------


def step(tlc, x, r, w, dy, dt, dw_flat, ws=None):
    """A norm, a gated activation and their gradients, as a training step strings them together."""
    cols = x.shape[1]
    half = cols // 2
    total, y, c, rstd = tlc.ckpt8_norm(x, w, 1e-5, ref.INT8, residual=r)
    h, ca, cb = tlc.ckpt8_act(y[:, :half], ref.SILU, ref.E4M3, b=y[:, half:2 * half])
    dyy = torch.zeros_like(y)
    tlc.ckpt8_act_grad(dy, ref.SILU, ca, cb, da=dyy[:, :half], db=dyy[:, half:2 * half])
    dx, dw = tlc.ckpt8_norm_grad(dyy, c, rstd, w, dtotal=dt)
    tlc.ckpt8_weight_grad(dyy, c, col_scale=w, dw=dw_flat.view(cols, cols))
    return total, h, dx, dw


def test_on_another_stream(tlc):
    rows, cols = 300, 256
    args = [randn(gen(k), rows, cols, dtype=torch.bfloat16).cuda() for k in range(2)]
    w = randn(gen(2), cols).cuda()
    dy = randn(gen(3), rows, cols // 2, dtype=torch.bfloat16).cuda()
    x8 = tlc.ckpt8_pack(args[0], ref.INT8)
    want = [tlc.ckpt8_unpack(x8), tlc.ckpt8_weight_grad(dy, x8), *tlc.ckpt8_norm(args[0], w, 1e-5, None)[1:2]]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = [tlc.ckpt8_unpack(x8, stream=s), tlc.ckpt8_weight_grad(dy, x8, stream=s),
               *tlc.ckpt8_norm(args[0], w, 1e-5, None, stream=s)[1:2]]
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # two streams at once, each with a workspace of its own
    t = torch.cuda.Stream()
    got = [tlc.ckpt8_weight_grad(dy, x8, stream=q) for q in (s, t, s, t)]
    torch.cuda.synchronize()
    for a in got:
        assert torch.equal(a, want[1])


def test_captured_and_replayed(tlc):
    rows, cols = 600, 256
    ins = [randn(gen(k), rows, cols, dtype=torch.bfloat16).cuda() for k in range(3)]
    w = randn(gen(4), cols).cuda()
    dy = randn(gen(5), rows, cols // 2, dtype=torch.bfloat16).cuda()
    flat = torch.zeros(cols * cols, device="cuda")
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step(tlc, ins[0], ins[1], w, dy, ins[2], flat)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(tlc, ins[0], ins[1], w, dy, ins[2], flat)
    for k in range(4):
        for j, v in enumerate(ins):
            v.copy_(randn(gen(50 + 10 * k + j), rows, cols, dtype=torch.bfloat16))
        dy.copy_(randn(gen(70 + k), rows, cols // 2, dtype=torch.bfloat16))
        flat.fill_(math.nan)
        for o in outs:
            o.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (*outs, flat)]
        eager_flat = torch.zeros(cols * cols, device="cuda")
        want = step(tlc, ins[0], ins[1], w, dy, ins[2], eager_flat)
        for a, b in zip(got, (*want, eager_flat)):
            assert torch.equal(a, b), k


def test_refusals(tlc):
    x = torch.zeros(4, 40, dtype=torch.bfloat16, device="cuda")
    c = tlc.ckpt8_pack(x, ref.INT8)
    r = torch.ones(4, device="cuda")
    w = torch.ones(40, device="cuda")
    bad = tlc.Checkpoint8(c.codes[:, :40], c.scales, 40, ref.INT8)
    refused = [
        lambda: tlc.ckpt8_pack(x, 3),
        lambda: tlc.ckpt8_pack(x.double(), ref.INT8),
        lambda: tlc.ckpt8_pack(x.cpu(), ref.INT8),
        lambda: tlc.ckpt8_pack(x.t(), ref.INT8),
        lambda: tlc.ckpt8_pack(x[0], ref.INT8),
        lambda: tlc.ckpt8_pack(x[:1].expand(4, 40), ref.INT8),
        lambda: tlc.ckpt8_pack(x, ref.INT8, out=tlc.ckpt8_pack(x, ref.E4M3)),
        lambda: tlc.ckpt8_pack(x, ref.INT8, out=tlc.ckpt8_pack(x[:3], ref.INT8)),
        lambda: tlc.ckpt8_unpack(bad),
        lambda: tlc.ckpt8_unpack(tlc.Checkpoint8(c.codes, c.scales, 65, ref.INT8)),
        lambda: tlc.ckpt8_unpack(tlc.Checkpoint8(c.codes, c.scales[:3], 40, ref.INT8)),
        lambda: tlc.ckpt8_unpack(c, torch.float64),
        lambda: tlc.ckpt8_unpack(c, y=x[:3]),
        lambda: tlc.ckpt8_act(x, 4, ref.INT8),
        lambda: tlc.ckpt8_act(x, ref.GELU, ref.INT8, b=x[:3]),
        lambda: tlc.ckpt8_act(x, ref.GELU, ref.INT8, b=x.float()),
        lambda: tlc.ckpt8_act(x, ref.GELU, ref.INT8, b_out=c),
        lambda: tlc.ckpt8_act_grad(x[:3], ref.GELU, c),
        lambda: tlc.ckpt8_act_grad(x, ref.GELU, c, db=x),
        lambda: tlc.ckpt8_act_grad(x, ref.GELU, c, tlc.ckpt8_pack(x, ref.E4M3)),
        lambda: tlc.ckpt8_act_grad(x, 0, c),
        lambda: tlc.ckpt8_norm(x, w[:39], 1e-5, ref.INT8),
        lambda: tlc.ckpt8_norm(x, w.half(), 1e-5, ref.INT8),
        lambda: tlc.ckpt8_norm_grad(x, c, r, w.half()),
        lambda: tlc.ckpt8_weight_grad(x, c, col_scale=w.half()),
        lambda: tlc.ckpt8_norm(x, w, 0.0, ref.INT8),
        lambda: tlc.ckpt8_norm(x, w, math.nan, ref.INT8),
        lambda: tlc.ckpt8_norm(x, w, -1.0, ref.INT8),
        lambda: tlc.ckpt8_norm(x, w, 1e-5, ref.INT8, total=x),
        lambda: tlc.ckpt8_norm(x, None, 1e-5, ref.INT8, weighted=True),
        lambda: tlc.ckpt8_norm(x, w, 1e-5, None, want_y=False),
        lambda: tlc.ckpt8_norm(torch.zeros(1, 16385, device="cuda"), None, 1e-5, ref.INT8),
        lambda: tlc.ckpt8_norm_grad(x, c, r[:3], w),
        lambda: tlc.ckpt8_norm_grad(x, c, r.half(), w),
        lambda: tlc.ckpt8_norm_grad(x, x.float(), r, w),
        lambda: tlc.ckpt8_norm_grad(x, c, r, w, accumulate=True),
        lambda: tlc.ckpt8_norm_grad(x, c, r, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: tlc.ckpt8_weight_grad(x[:3], c),
        lambda: tlc.ckpt8_weight_grad(x, c, col_scale=w[:39]),
        lambda: tlc.ckpt8_weight_grad(x, c, dw=torch.zeros(40, 41, device="cuda")),
        lambda: tlc.ckpt8_weight_grad(x, c, dw=torch.zeros(40, 40, device="cuda", dtype=torch.bfloat16)),
        lambda: tlc.ckpt8_weight_grad(x, c, accumulate=True),
        lambda: tlc.ckpt8_weight_grad(x, c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for k, call in enumerate(refused):
        with pytest.raises((ValueError, tlc.TLCError)):
            call()
            raise AssertionError(f"call {k} was taken")
    torch.cuda.synchronize()


# ---- together ---------------------------------------------------------------


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_gradients_into_a_compressed_bucket(tlc, fmt, dtype):
    """A block (norm, gated feed-forward) whose backward pass keeps only checkpoints: its gradients go straight into a
    flat bucket, agree with the 64-bit gradients at the checkpoints' values, and leave through the gradient codec as
    the same numbers handed over as an array do."""
    rows, cols, wide = 200, 96, 160
    g = gen(fmt)
    x, r, dout = (randn(g, rows, cols, dtype=dtype) for _ in range(3))
    nw = (1 + randn(g, cols, scale=0.2))
    w1, w2 = randn(g, 2 * wide, cols, dtype=dtype, scale=cols ** -0.5), randn(g, cols, wide, dtype=dtype,
                                                                             scale=wide ** -0.5)
    sizes = [cols, 2 * wide * cols, cols * wide]
    group = tlc.Group(sizes)
    bucket = torch.full((group.total,), math.nan, device="cuda")
    o = group.elem_offsets
    d_nw, d_w1, d_w2 = bucket[:o[1]], bucket[o[1]:o[2]].view(2 * wide, cols), bucket[o[2]:].view(cols, wide)

    def product(a, b):
        return (a.float() @ b.float()).to(dtype)

    # forward: kept are n8, a8, b8 and rstd
    total, y, n8, rstd = tlc.ckpt8_norm(x.cuda(), nw.cuda(), 1e-5, fmt, residual=r.cuda())
    ab = product(y, w1.cuda().t())
    h, a8, b8 = tlc.ckpt8_act(ab[:, :wide], ref.SILU, fmt, b=ab[:, wide:])
    # backward
    dout_d = dout.cuda()
    dh = product(dout_d, w2.cuda())
    dab = torch.empty(rows, 2 * wide, dtype=dtype, device="cuda")
    _, _, h8 = tlc.ckpt8_act_grad(dh, ref.SILU, a8, b8, da=dab[:, :wide], db=dab[:, wide:], want_y=True)
    tlc.ckpt8_weight_grad(dout_d, h8, dw=d_w2)
    tlc.ckpt8_weight_grad(dab, n8, col_scale=nw.cuda(), dw=d_w1)
    dy = product(dab, w1.cuda())
    dx, _ = tlc.ckpt8_norm_grad(dy, n8, rstd, nw.cuda(), dtotal=dout_d, dw=d_nw)
    torch.cuda.synchronize()

    # the same from the definitions, step by step from what each step was given
    def values(c):
        return ref.decode(c.codes.cpu(), c.scales.cpu(), c.format, c.cols)

    n, a, b, h64 = values(n8), values(a8), values(b8), values(h8)
    f, slope = ref.act(ref.SILU, a)
    dh64 = dh.cpu().double()
    assert_close(dab[:, :wide], dh64 * b * slope, U[dtype] * (dh64 * b * slope).abs() * 1.01
                 + 2.0 ** -18 * (dh64 * b).abs() + LEAST[dtype], "da")
    assert_close(dab[:, wide:], dh64 * f, U[dtype] * (dh64 * f).abs() * 1.01 + 2.0 ** -20 * (dh64 * a).abs()
                 + LEAST[dtype], "db")
    dab64, dout64, nw64 = dab.cpu().double(), dout.double(), nw.double()
    assert_close(d_w2, dout64.t() @ h64, rows * 2.0 ** -23 * (dout64.abs().t() @ h64.abs()) + 1e-30, "dw2")
    sizes64 = (dab64.abs().t() @ n.abs()) * nw64.abs()
    assert_close(d_w1, (dab64.t() @ n) * nw64, (rows + 1) * 2.0 ** -23 * sizes64 + 1e-30, "dw1")
    dy64 = dy.cpu().double()
    assert_close(d_nw, (dy64 * n).sum(0), (rows + 4) * 2.0 ** -24 * (dy64 * n).abs().sum(0) + 1e-30, "dnw")
    assert torch.isfinite(bucket).all() and torch.isfinite(dx.float()).all()
    # the whole against the gradient without checkpoints: as far off as 8 bits are
    full = [t.double().requires_grad_() for t in (nw, w1, w2)]
    t64 = total.cpu().double()
    n64 = ref.norm(t64, float(torch.tensor(1e-5)))[1]
    z = (n64 * full[0]) @ full[1].t()
    out = (torch.nn.functional.silu(z[:, :wide]) * z[:, wide:]) @ full[2].t()
    out.backward(dout64)
    # codes are off by 2^-7.. of the group's largest value (int8) or 2^-4 of the value (e4m3), independently over
    # `rows` products: the sums agree to a few percent of their norm
    for got, want in zip((d_nw, d_w1, d_w2), full):
        off = (got.cpu().double() - want.grad).norm() / want.grad.norm()
        assert off < 2.0 ** -4, float(off)
    # into the codec: as the oracle compresses the same numbers
    import oracle
    import numpy as np
    err = torch.zeros(group.total, device="cuda")
    out_b, lens, scales, status = group.compress(bucket, err, 1.5)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    host = bucket.cpu().numpy()
    for t, size in enumerate(sizes):
        want_st, want_m, _ = oracle.compress(host[o[t]:o[t] + size], np.zeros(size, np.float32), 1.5)
        L = int(lens[t].item())
        assert np.array_equal(out_b[group.offsets[t]:group.offsets[t] + L].cpu().numpy(), want_st)
        assert np.float32(scales[t].item()) == want_m
