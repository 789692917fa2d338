"""8-bit integer products and products grouped by expert on the GPU against
their definitions in 64 bits: bit for bit where the result is defined so (codes,
scales, sums of whole numbers), otherwise within bounds derived from the
roundings.

u(dtype) is half a step of a type relative to the value; a stored result is off
by u of its value, plus half the least step of the type near zero."""
import math

import pytest
import torch

import ckpt8_ref
import products_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
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


def whole(g, *shape, dtype=torch.float32, most=3):
    """Whole numbers: products and sums of them are exact in any order."""
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype)


def strided(t, pad, offset=0):
    """t on the GPU as a view with rows `pad` further apart, starting `offset` elements in; the gaps hold NaN."""
    rows, cols = t.shape[-2:]
    many = t.numel() // (rows * cols) if t.numel() else 1
    flat = torch.full((offset + many * rows * (cols + pad),), math.nan, dtype=t.dtype, device="cuda")
    v = flat[offset:].view(*t.shape[:-1], cols + pad)[..., :cols]
    v.copy_(t)
    return v


def offsets_of(counts, first=0):
    ends = [first]
    for c in counts:
        ends.append(ends[-1] + c)
    return torch.tensor(ends, dtype=torch.int64)


def assert_close(got, want, bound, label):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{label}: at {at}: got {float(got[tuple(at)])!r}, want {float(want[tuple(at)])!r}, "
                             f"bound {float(bound.expand_as(want)[tuple(at)]):.3g} ({int(bad.sum())} values)")


# ---- 8-bit rows and columns --------------------------------------------------

SHAPES = [(1, 1), (1, 33), (5, 128), (3, 129), (77, 1000), (130, 96), (9, 2049), (2, 8193), (2, 16385), (1, 131072),
          (1025, 40), (257, 513)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_rows(tlc, rows, cols, dtype):
    say(f"pack_rows {rows}x{cols} {dtype}")
    x = randn(gen(rows * 7 + cols), rows, cols, dtype=dtype, scale=3.0)
    codes, scales = ref.pack_rows(x)
    for v in (x.cuda(), strided(x, 3, 1)):
        q = tlc.q8_pack_rows(v)
        assert torch.equal(q.scales.cpu(), scales)
        assert torch.equal(q.codes.cpu(), codes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,rows", SHAPES)
def test_pack_columns(tlc, rows, cols, dtype):
    say(f"pack_columns {rows}x{cols} {dtype}")
    x = randn(gen(rows * 5 + cols), rows, cols, dtype=dtype, scale=3.0)
    codes, scales = ref.pack_columns(x)
    for v in (x.cuda(), strided(x, 3, 1)):
        q = tlc.q8_pack_columns(v)
        assert torch.equal(q.scales.cpu(), scales)
        assert torch.equal(q.codes.cpu(), codes)


def special_rows(cols):
    """Rows whose scale or codes are special: zeros, borders between codes, the least and largest numbers, no number."""
    g = gen(3)
    rows = [torch.zeros(cols)]
    steps = torch.arange(cols).remainder(255).float() - 127
    rows += [steps, (steps + 0.5).clamp(-127, 127), steps * 2.0 ** -140, steps * 2.0 ** 120]
    rows += [torch.full((cols,), 2.0 ** -149), torch.full((cols,), torch.finfo(torch.float32).max), torch.full((cols,), -1.4e-45)]
    for v in (127 * 2.0 ** -126, 126.99999 * 2.0 ** -126, 2.0 ** -126):
        r = torch.randn(cols, generator=g) * v / 4
        r[1] = v
        rows.append(r.clamp(-v, v))
    for v in (math.inf, -math.inf, math.nan):
        r = torch.randn(cols, generator=g)
        r[-1] = v
        rows.append(r)
    both = torch.randn(cols, generator=g)
    both[0], both[5] = math.nan, math.inf
    return torch.stack([*rows, both])


@pytest.mark.parametrize("cols", [64, 300, 3000])
def test_pack_special_values(tlc, cols):
    x = special_rows(cols)
    codes, scales = ref.pack_rows(x)
    q, t = tlc.q8_pack_rows(x.cuda()), tlc.q8_pack_columns(x.t().contiguous().cuda())
    for got in (q, t):
        assert torch.equal(got.codes.cpu(), codes)
        assert torch.equal(torch.nan_to_num(got.scales.cpu(), nan=-1.0), torch.nan_to_num(scales, nan=-1.0))


def test_pack_rows_of_more_than_one_launch(tlc):
    """2^26 rows of 64 lanes are 2^32 threads, which HIP takes in two launches."""
    rows = 2 ** 26 + 5
    x = torch.zeros(rows, 1, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 2 ** 25, 2 ** 26 - 8, 2 ** 26 - 4, 2 ** 26, 2 ** 26 + 4], device="cuda")
    x[at, 0] = torch.arange(1, 8, device="cuda").bfloat16()
    q = tlc.q8_pack_rows(x)
    assert (q.codes[at, 0] == 127).all() and not q.codes[at, 1:].any()
    assert torch.equal(q.scales[at].cpu(), torch.arange(1, 8).float() / torch.full((7,), 127.0))
    assert int((q.codes[:, 0] != 0).sum()) == 7


# ---- the product of 8-bit integers -------------------------------------------


def random_codes(g, rows, cols):
    codes = torch.zeros(rows, -(-cols // 128) * 128, dtype=torch.int8)
    codes[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=g).to(torch.int8)
    return codes, torch.exp(torch.randn(rows, generator=g))


def rows8(tlc, codes, scales, cols):
    return tlc.Rows8(codes.cuda(), scales.cuda(), cols)


def check_product8(got, want, dtype, label):
    # the sum's conversion and the two products with the scales: a rounding of 2^-24 each; then the type's
    bound = want.abs() * (3.01 * 2.0 ** -24 + (0 if dtype == torch.float32 else U[dtype] * 1.001)) + LEAST[dtype]
    assert_close(got, want, bound, label)


PRODUCTS = [(1, 1, 1), (1, 8192, 200), (3, 33, 127), (16, 64, 128), (17, 130, 129), (33, 515, 1000), (128, 128, 256),
            (129, 257, 515), (300, 1000, 96), (257, 300, 4096), (700, 384, 384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,k", PRODUCTS)
def test_product8(tlc, rows, n, k, dtype):
    say(f"product8 {rows}x{n}x{k} {dtype}")
    g = gen(rows + n + k)
    (a, sa), (w, sw) = random_codes(g, rows, k), random_codes(g, n, k)
    sa *= 2.0 ** -20  # results inside fp16's range
    want, _ = ref.product8(a, sa, w, sw)
    y = tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), dtype)
    check_product8(y, want, dtype, "y")
    out = strided(torch.zeros(rows, n, dtype=dtype), 5, 1)
    assert tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), dtype, y=out) is out
    assert torch.equal(out, y)
    gaps = torch.as_strided(out, (rows, 5), (n + 5, 1), out.storage_offset() + n)
    assert torch.isnan(gaps).all()


def test_product8_of_long_sums_is_exact(tlc):
    """131072 products of the largest codes: sums next to 2^31, exact before they are rounded to fp32."""
    k = 131072
    a = torch.full((3, k), 127, dtype=torch.int8)
    a[1] = -127
    a[2, ::2] = -127
    a[2, 5] = 126
    w = torch.full((40, k), 127, dtype=torch.int8)
    w[7, :9] = 1
    one = torch.ones
    want = a.double() @ w.double().t()
    y = tlc.q8_product(rows8(tlc, a, one(3), k), rows8(tlc, w, one(40), k), torch.float32)
    assert torch.equal(y.cpu(), want.float())


def test_product8_scales_that_meet_at_the_ends_of_the_range(tlc):
    """Scales of 2^-126 and 2^120: neither product with the sum leaves fp32's range where the result does not."""
    k = 64
    g = gen(9)
    a, _ = random_codes(g, 4, k)
    w, _ = random_codes(g, 6, k)
    sa = torch.tensor([2.0 ** -126, 2.0 ** 120, 2.0 ** -126, 1.0])
    sw = torch.tensor([2.0 ** 120, 2.0 ** -126, 2.0 ** 119, 2.0 ** -100, math.nan, 2.0 ** 10])
    y = tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32).cpu()
    want, sums = ref.product8(a, sa, w, sw)
    fits = torch.isfinite(want) & (want.abs() < 2.0 ** 127) & (want.abs() >= 2.0 ** -126)
    assert fits.sum() >= 8
    assert torch.equal(y[fits].double(), want[fits])  # scales are powers of two, sums below 2^24
    assert torch.isnan(y[:, 4]).all()
    assert torch.isinf(y[1, 0]) and torch.isinf(y[1, 2])
    sa[2] = math.nan
    y = tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32).cpu()
    assert torch.isnan(y[2]).all() and not torch.isnan(y[3, :4]).any()


@pytest.mark.parametrize("rows,n,k", [(5, 40, 64), (200, 300, 515)])
def test_product8_added_to_a_bucket(tlc, rows, n, k):
    g = gen(4)
    (a, _), (w, _) = random_codes(g, rows, k), random_codes(g, n, k)
    sa, sw = torch.ones(rows), torch.ones(n)
    want, _ = ref.product8(a, sa, w, sw)  # below 2^24: exact
    start = whole(g, rows, n, most=1000)
    bucket = strided(start, 2, 3)
    y = tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32, y=bucket, accumulate=True)
    assert y is bucket and torch.equal(y.cpu().double(), want + start.double())


COUNTS = [
    [7],
    [0, 5, 0],
    [1, 1, 1, 1, 1, 1, 1, 1],
    [130, 0, 3, 129, 128, 0, 0, 260],
    [0] * 70 + [3, 0, 40] + [1] * 60,
    [600, 1],
]


@pytest.mark.parametrize("k,n", [(200, 40), (515, 300)])
@pytest.mark.parametrize("counts", COUNTS)
def test_product8_grouped(tlc, counts, k, n):
    say(f"product8 grouped {counts} {k} {n}")
    g = gen(len(counts) + n)
    before, behind = 2, 5
    offsets = offsets_of(counts, before)
    rows = before + sum(counts) + behind
    (a, _), (w, _) = random_codes(g, rows, k), random_codes(g, len(counts) * n, k)
    sa, sw = torch.ones(rows), torch.ones(len(counts) * n)
    y = torch.full((rows, n), math.nan, device="cuda")
    tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32, offsets=offsets.cuda(), y=y)
    got = y.cpu()
    assert torch.isnan(got[:before]).all() and torch.isnan(got[rows - behind:]).all()
    for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
        want, _ = ref.product8(a[b:t], sa[b:t], w[e * n:(e + 1) * n], sw[e * n:(e + 1) * n])
        assert torch.equal(got[b:t].double(), want), e  # below 2^24: exact


# ---- products grouped by expert ----------------------------------------------


def weights(g, experts, n, k, dtype, make=randn):
    return make(g, experts, n, k, dtype=dtype)


LAYOUTS = [
    # pad and offset of rows, of the weight's rows: 16-byte aligned, and at any element
    (0, 0, 0, 0),
    (8, 0, 16, 0),
    (3, 1, 5, 3),
]
EXPERT_SIZES = [(1, 1), (33, 20), (64, 64), (128, 256), (129, 131), (515, 260), (40, 1000)]  # (k, n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k,n", EXPERT_SIZES)
@pytest.mark.parametrize("counts", COUNTS)
def test_expert_products_of_whole_numbers_are_exact(tlc, counts, k, n, dtype):
    say(f"expert products {counts} k={k} n={n} {dtype}")
    g = gen(k + n + len(counts))
    before, behind = 1, 3
    offsets, rows, experts = offsets_of(counts, before), before + sum(counts) + behind, len(counts)
    # fp16 holds whole numbers up to 2048, bf16 up to 256: their results are rounded from the exact sums
    x, dy, w = whole(g, rows, k, dtype=dtype), whole(g, rows, n, dtype=dtype), whole(g, experts, n, k, dtype=dtype)
    off = offsets.cuda()
    for pad, at, wpad, wat in LAYOUTS:
        y = strided(torch.full((rows, n), math.nan, dtype=dtype), pad, at)
        dx = strided(torch.full((rows, k), math.nan, dtype=dtype), pad, at)
        wd = strided(w, wpad, wat)
        tlc.expert_product(strided(x, pad, at), wd, off, y=y)
        tlc.expert_input_grad(strided(dy, pad, at), wd, off, dx=dx)
        y, dx = y.cpu(), dx.cpu()
        for v in (y, dx):
            assert torch.isnan(v[:before]).all() and torch.isnan(v[rows - behind:]).all()
        for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
            we = w[e].double()
            assert torch.equal(y[b:t], (x[b:t].double() @ we.t()).to(dtype)), (e, pad)
            assert torch.equal(dx[b:t], (dy[b:t].double() @ we).to(dtype)), (e, pad)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k,n,experts", [(3, 500, 70, 4), (200, 1024, 257, 3), (333, 515, 1000, 1),
                                              (1000, 640, 320, 7)])
def test_expert_products(tlc, rows, k, n, experts, dtype):
    say(f"expert products {rows} {k} {n} {experts} {dtype}")
    g = gen(rows + k)
    x, dy = randn(g, rows, k, dtype=dtype), randn(g, rows, n, dtype=dtype, scale=0.1)
    w = randn(g, experts, n, k, dtype=dtype, scale=k ** -0.5)
    ends = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g)).values.tolist()
    offsets = torch.tensor([0, *ends, rows], dtype=torch.int64)
    off = offsets.cuda() if experts > 1 else None
    y, dx = tlc.expert_product(x.cuda(), w.cuda(), off), tlc.expert_input_grad(dy.cuda(), w.cuda(), off)
    assert y.dtype == dx.dtype == dtype
    for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
        for got, left, right, terms in ((y, x, w[e].t(), k), (dx, dy, w[e], n)):
            left, right = left[b:t].double(), right.double()
            want, size = left @ right, left.abs() @ right.abs()
            # each of `terms` additions in fp32, and in fp32 each product, rounds by 2^-24 of at most `size`
            bound = 2 * terms * 2.0 ** -24 * size + U[dtype] * want.abs() * 1.01 + LEAST[dtype]
            assert_close(got[b:t], want, bound, (e, terms))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [3, 200])
def test_values_below_the_normal_range(tlc, rows, dtype):
    """Subnormal inputs count with their value, and subnormal results are rounded to their step."""
    k, n = 96, 40
    g = gen(11)
    least = {torch.float32: -149, torch.float16: -24, torch.bfloat16: -133}[dtype]
    x = whole(g, rows, k, most=3).double() * 2.0 ** least
    x, up = x.to(dtype), 2.0 ** (20 if dtype != torch.float16 else 10)
    assert (x != 0).any()
    for factor in (up, 0.25):
        w = (whole(g, 1, n, k, most=3).double() * factor).to(dtype)
        # In 16 bits fp32 holds every product and sum exactly.  In fp32 a quarter of the least step is no fp32 number:
        # each of the k additions rounds to a multiple of 2^-149, by 2^-150 at most.
        inside = k * 2.0 ** -150 if dtype == torch.float32 and factor < 1 else 0.0
        want = (x.double() @ w[0].double().t()).to(dtype).double()
        bound = torch.full_like(want, inside + (2.0 ** -150 if inside else 0.0))  # and the reference's own rounding
        assert_close(tlc.expert_product(x.cuda(), w.cuda()), want, bound, ("y", factor))
        back = w.transpose(1, 2).contiguous().cuda()
        assert_close(tlc.expert_input_grad(x.cuda(), back), want, bound, ("dx", factor))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [1027, 2050, 4099, 8191])
def test_long_reductions(tlc, k, dtype):
    """Few tiles and a long reduction, whose slices end at odd places: the last one may be shorter than 16 bytes."""
    rows, n, counts = 140, 72, [85, 0, 55]
    g = gen(k)
    x, w = whole(g, rows, k, dtype=dtype, most=1), whole(g, 3, n, k, dtype=dtype, most=1)
    off = offsets_of(counts).cuda()
    y = tlc.expert_product(strided(x, 3, 1), strided(w, 1, 0), off)
    # the same numbers as the reduction of the gradient: w transposed, its rows the reduction
    z = tlc.expert_input_grad(x.cuda(), w.transpose(1, 2).contiguous().cuda(), off)
    for e, (b, t) in enumerate(ref.spans(off.tolist(), rows)):
        want = (x[b:t].double() @ w[e].double().t()).to(dtype)
        assert torch.equal(y[b:t].cpu(), want) and torch.equal(z[b:t].cpu(), want), e
    q = [random_codes(g, r, k) for r in (rows, 3 * n)]
    y8 = tlc.q8_product(*[rows8(tlc, c, torch.ones(c.shape[0]), k) for c, _ in q], torch.float32, offsets=off)
    for e, (b, t) in enumerate(ref.spans(off.tolist(), rows)):
        assert torch.equal(y8[b:t].cpu(), (q[0][0][b:t].double() @ q[1][0][e * n:(e + 1) * n].double().t()).float())


# Rows of two experts in one round of large tiles, 240 of them, and in 272, whose last 16 smaller ones compute: with a
# last tile of 4 rows, and of 156.
LARGE = [[1700, 1900], [2460, 1540], [1540, 2460]]


@pytest.mark.parametrize("counts", LARGE)
@pytest.mark.parametrize("k,pad", [(1096, 0), (1096, 3), (1027, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_large_ragged_products_of_whole_numbers_are_exact(tlc, dtype, k, pad, counts):
    """Sizes that take the larger tile (in 16 bits and 8), with a ragged last one in every direction."""
    n, before, behind = 4091, 3, 5
    say(f"large products {dtype} k={k} pad={pad} {counts}")
    g = gen(k + pad)
    offsets, rows = offsets_of(counts, before), before + sum(counts) + behind
    off = offsets.cuda()
    x, w = whole(g, rows, k, dtype=dtype), whole(g, 2, n, k, dtype=dtype)
    back = w.transpose(1, 2).contiguous()
    y = strided(torch.full((rows, n), math.nan, dtype=dtype), pad)
    z = strided(torch.full((rows, n), math.nan, dtype=dtype), pad)
    tlc.expert_product(strided(x, pad), strided(w, pad), off, y=y)
    tlc.expert_input_grad(strided(x, pad), strided(back, pad), off, dx=z)
    for v in (y, z):
        assert torch.isnan(v[:before]).all() and torch.isnan(v[rows - behind:]).all()
        for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
            want = (x[b:t].cuda().float() @ w[e].cuda().float().t()).to(dtype)  # whole numbers below 2^24
            assert torch.equal(v[b:t], want), e


@pytest.mark.parametrize("counts", LARGE)
def test_large_ragged_product8_is_exact(tlc, counts):
    n, k, rows = 4091, 2055, sum(counts)
    g = gen(21)
    off = offsets_of(counts).cuda()
    a, w = [torch.randint(-80, 81, (r, k), generator=g).to(torch.int8) for r in (rows, 2 * n)]
    pads = torch.nn.functional.pad
    q = [tlc.Rows8(pads(c, (0, 2176 - k)).cuda(), torch.ones(c.shape[0], device="cuda"), k) for c in (a, w)]
    y = tlc.q8_product(*q, torch.float32, offsets=off)
    z = torch.zeros_like(y)
    tlc.q8_product(*q, torch.float32, offsets=off, y=z, accumulate=True)
    assert torch.equal(y, z)
    for e, (b, t) in enumerate(ref.spans(off.tolist(), rows)):
        want = a[b:t].cuda().float() @ w[e * n:(e + 1) * n].cuda().float().t()  # 2055 * 80 * 80 is below 2^24
        assert torch.equal(y[b:t], want), e


def test_offsets_that_are_not_in_order(tlc):
    """Offsets that fall, are negative or past the rows: held to the rows and to not falling, nothing else is written."""
    rows, k, n = 300, 96, 40
    g = gen(1)
    x, dy = whole(g, rows, k), whole(g, rows, n)
    x8 = ckpt8_ref.encode(x, ckpt8_ref.INT8)
    for offsets in ([0, 50, 20, 60], [10, 5, 400, 7], [0, -1, 3, 2], [299, 300, 300, 1 << 62], [5, 5, 5, 5],
                    [250, 100, 0, 0]):
        w = whole(g, 3, n, k)
        off = torch.tensor(offsets, dtype=torch.int64).cuda()
        y = torch.full((rows, n), math.nan, device="cuda")
        dx = torch.full((rows, k), math.nan, device="cuda")
        tlc.expert_product(x.cuda(), w.cuda(), off, y=y)
        tlc.expert_input_grad(dy.cuda(), w.cuda(), off, dx=dx)
        dw = tlc.expert_weight_grad(dy.cuda(), tlc.Checkpoint8(x8[0].cuda(), x8[1].cuda(), k, ckpt8_ref.INT8), off)
        want_y, want_dx = torch.full((rows, n), math.nan), torch.full((rows, k), math.nan)
        for e, (b, t) in enumerate(ref.spans(offsets, rows)):
            want_y[b:t], want_dx[b:t] = x[b:t] @ w[e].t(), dy[b:t] @ w[e]
            assert torch.equal(dw[e].cpu(), dy[b:t].t() @ x[b:t]), (offsets, e)
        for got, want in ((y, want_y), (dx, want_dx)):
            assert torch.equal(torch.nan_to_num(got.cpu(), nan=9e9), torch.nan_to_num(want, nan=9e9)), offsets


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_that_are_not_finite_stay_in_their_rows(tlc, dtype):
    """An infinity or NaN in a row of one expert reaches that row's results only, also next to an odd end of a row."""
    rows, k, n = 40, 77, 50
    g = gen(2)
    x, w = whole(g, rows, k, dtype=dtype), whole(g, 2, n, k, dtype=dtype)
    x[5, 3], x[20, k - 1], x[21, 0] = math.nan, math.inf, math.nan
    w[1, 7, 0] = math.nan
    off = offsets_of([18, 22])
    y = tlc.expert_product(x.cuda(), w.cuda(), off.cuda()).cpu()
    bad = torch.zeros(rows, n, dtype=torch.bool)
    bad[5], bad[20], bad[21], bad[18:, 7] = True, True, True, True
    assert torch.isfinite(y[~bad].float()).all()
    assert torch.isnan(y[5]).all() and torch.isnan(y[21]).all() and torch.isnan(y[18:, 7]).all()
    dx = tlc.expert_input_grad(whole(g, rows, n, dtype=dtype).cuda(), w.cuda(), off.cuda()).cpu()
    bad = torch.zeros(rows, k, dtype=torch.bool)
    bad[18:, 0] = True
    assert torch.isfinite(dx[~bad].float()).all() and torch.isnan(dx[bad].float()).all()


@pytest.mark.parametrize("fmt", [ckpt8_ref.INT8, ckpt8_ref.E4M3])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", COUNTS + [[1000, 0, 700, 9]])
def test_expert_weight_gradient_of_whole_numbers_is_exact(tlc, counts, dtype, fmt):
    say(f"expert weight grad {counts} {dtype} {fmt}")
    n, cols = 70, 129
    g = gen(len(counts))
    before, behind = 2, 4
    offsets, rows, experts = offsets_of(counts, before), before + sum(counts) + behind, len(counts)
    dy, x = whole(g, rows, n, dtype=dtype), whole(g, rows, cols)
    codes, scales = ckpt8_ref.encode(x, fmt)
    x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, fmt)
    values = ckpt8_ref.decode(codes, scales, fmt, cols)
    assert torch.equal(values, x.double())
    cs = torch.randint(1, 4, (cols,), generator=g).float()
    want = torch.stack([dy[b:t].double().t() @ values[b:t] * cs.double()
                        for b, t in ref.spans(offsets.tolist(), rows)])
    off = offsets.cuda()
    dw = tlc.expert_weight_grad(strided(dy, 3, 1), x8, off, col_scale=cs.cuda())
    assert torch.equal(dw.cpu().double(), want)
    # added to a strided place of a bucket
    start = whole(g, experts, n, cols, most=50)
    bucket = strided(start, 3, 2)
    tlc.expert_weight_grad(dy.cuda(), x8, off, col_scale=cs.cuda(), dw=bucket, accumulate=True)
    assert torch.equal(bucket.cpu().double(), want + start.double())
    gaps = torch.as_strided(bucket, (experts * n, 3), (cols + 3, 1), bucket.storage_offset() + cols)
    assert torch.isnan(gaps).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_expert_weight_gradient_of_many_tiles_and_slices(tlc, dtype):
    """Sizes that take the larger tile, and sliced rows of few small weights."""
    for counts, n, cols in (([300, 0, 900, 500], 1024, 2048), ([5000, 100, 3000], 128, 256), ([9000], 128, 128)):
        say(f"expert weight grad tiles {counts} {n} {cols} {dtype}")
        g = gen(n)
        offsets, rows = offsets_of(counts), sum(counts)
        dy, x = whole(g, rows, n, dtype=dtype, most=2), whole(g, rows, cols, most=2)
        codes, scales = ckpt8_ref.encode(x, ckpt8_ref.E4M3)
        x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, ckpt8_ref.E4M3)
        dw = tlc.expert_weight_grad(dy.cuda(), x8, offsets.cuda())
        for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
            want = dy[b:t].cuda().float().t() @ x[b:t].cuda()  # whole numbers below 2^24: exact in fp32
            assert torch.equal(dw[e], want), (counts, e)


@pytest.mark.parametrize("n,cols", [(256, 512), (200, 300)])
@pytest.mark.parametrize("experts", [7, 8, 9, 63, 64, 65])
def test_expert_weight_gradient_in_any_order_of_lengths(tlc, experts, n, cols):
    """Longest first, up to a wavefront's lanes of experts: rising, falling, equal, all but one empty, and offsets that turn back."""
    say(f"expert weight grad order {experts} {n} {cols}")
    g = gen(experts)
    e = list(range(experts))
    one = [0] * experts
    one[experts // 2] = 333
    turning = offsets_of([5] * experts)
    turning[experts // 3] = 2**63 - 1 if experts % 2 else 0  # past the rows, or back to the first
    for offsets in [offsets_of(c) for c in (e, e[::-1], [17] * experts, one)] + [turning]:
        rows = max(int(offsets[-1]), 1)
        dy, x = whole(g, rows, n, dtype=torch.bfloat16), whole(g, rows, cols)
        codes, scales = ckpt8_ref.encode(x, ckpt8_ref.INT8)
        x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, ckpt8_ref.INT8)
        dw = tlc.expert_weight_grad(dy.cuda(), x8, offsets.cuda())
        for i, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
            # whole numbers of at most 2^24: exact in fp32
            assert torch.equal(dw[i], dy[b:t].cuda().float().t() @ x[b:t].cuda()), (offsets, i)


def test_no_rows(tlc):
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.ones(3, 8, 16, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert tlc.expert_product(x, w, off).shape == (0, 8)
    assert tlc.expert_input_grad(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), w, off).shape == (0, 16)
    q = tlc.q8_pack_rows(x)
    assert q.rows == 0
    w8 = tlc.q8_pack_rows(w.view(24, 16))
    assert tlc.q8_product(q, w8, offsets=off).shape == (0, 8)
    x8 = tlc.ckpt8_pack(x, ckpt8_ref.INT8)
    dy = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert not tlc.expert_weight_grad(dy, x8, off).any()
    kept = torch.ones(3, 8, 16, device="cuda")
    tlc.expert_weight_grad(dy, x8, off, dw=kept, accumulate=True)
    assert (kept == 1).all()


def test_gradients_against_differences(tlc):
    """sum(g*y) along a direction: the products are linear in each operand, so whole numbers make differences exact."""
    counts, k, n = [30, 0, 45], 40, 24
    g = gen(8)
    off, rows = offsets_of(counts).cuda(), sum(counts)
    x, vx = whole(g, rows, k).cuda(), whole(g, rows, k).cuda()
    w, vw = whole(g, 3, n, k).cuda(), whole(g, 3, n, k).cuda()
    dy = whole(g, rows, n).cuda()

    def loss(x, w):
        return (tlc.expert_product(x, w, off).double() * dy).sum()

    dx = tlc.expert_input_grad(dy, w, off)
    dw = tlc.expert_weight_grad(dy, tlc.ckpt8_pack(x, ckpt8_ref.INT8), off)
    assert torch.equal((dx.double() * vx).sum(), (loss(x + vx, w) - loss(x - vx, w)) / 2)
    assert torch.equal((dw.double() * vw).sum(), (loss(x, w + vw) - loss(x, w - vw)) / 2)


def test_one_weight_for_all_experts_and_large_offsets(tlc):
    """A weight shared by stride 0, and experts that lie more than 2^32 bytes apart."""
    k, n, experts = 8192, 4096, 40
    g = gen(5)
    base = torch.empty(experts, n, k, dtype=torch.float32, device="cuda")  # 5.4 GB
    base[0].copy_(whole(g, n, k))
    base[-1].copy_(whole(g, n, k))
    x, dy = whole(g, 20, k).cuda(), whole(g, 20, n).cuda()
    off = torch.tensor([0] + [7] * (experts - 1) + [20], dtype=torch.int64, device="cuda")
    y, dx = tlc.expert_product(x, base, off), tlc.expert_input_grad(dy, base, off)
    for b, t, e in ((0, 7, 0), (7, 20, experts - 1)):
        we = base[e].cpu()
        assert torch.equal(y[b:t].cpu(), x[b:t].cpu() @ we.t())
        assert torch.equal(dx[b:t].cpu(), dy[b:t].cpu() @ we)
    shared = base[:1].expand(experts, n, k)
    assert torch.equal(tlc.expert_product(x, shared, off), tlc.expert_product(x, base[:1]))


# ---- together ----------------------------------------------------------------


def layer(tlc, x, w1, w2, off, dout, bucket, fmt):
    """A layer of experts, forward and backward, as a training step strings the calls together."""
    experts, wide, cols = w1.shape
    o = experts * wide * cols
    ab = tlc.expert_product(x, w1, off)
    h, a8, _ = tlc.ckpt8_act(ab, ckpt8_ref.SILU, fmt)
    y = tlc.expert_product(h, w2, off)
    x8 = tlc.ckpt8_pack(x, fmt)
    dh = tlc.expert_input_grad(dout, w2, off)
    da, _, h8 = tlc.ckpt8_act_grad(dh, ckpt8_ref.SILU, a8, want_y=True)
    tlc.expert_weight_grad(dout, h8, off, dw=bucket[o:].view(experts, cols, wide))
    tlc.expert_weight_grad(da, x8, off, dw=bucket[:o].view(experts, wide, cols))
    return y, tlc.expert_input_grad(da, w1, off)


def layer_inputs(counts, cols, wide, dtype, seed):
    g = gen(seed)
    rows, experts = sum(counts), len(counts)
    x, dout = randn(g, rows, cols, dtype=dtype).cuda(), randn(g, rows, cols, dtype=dtype, scale=0.1).cuda()
    w1 = randn(g, experts, wide, cols, dtype=dtype, scale=cols ** -0.5).cuda()
    w2 = randn(g, experts, cols, wide, dtype=dtype, scale=wide ** -0.5).cuda()
    return x, w1, w2, offsets_of(counts).cuda(), dout


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_of_experts_into_a_compressed_bucket(tlc, dtype):
    """Experts' gradients go straight into a flat bucket, agree with the 64-bit gradients to what 8 bits keep, and leave
    through the gradient codec as the same numbers handed over as an array do."""
    counts, cols, wide = [60, 0, 133, 7], 96, 160
    x, w1, w2, off, dout = layer_inputs(counts, cols, wide, dtype, 3)
    sizes = [len(counts) * wide * cols] * 2
    group = tlc.Group(sizes)
    bucket = torch.full((group.total,), math.nan, device="cuda")
    y, dx = layer(tlc, x, w1, w2, off, dout, bucket, ckpt8_ref.INT8)
    full = [t.cpu().double().requires_grad_() for t in (x, w1, w2)]
    outs = []
    for e, (b, t) in enumerate(ref.spans(off.tolist(), x.shape[0])):
        outs.append(torch.nn.functional.silu(full[0][b:t] @ full[1][e].t()) @ full[2][e].t())
    out = torch.cat(outs)
    out.backward(dout.cpu().double())
    # bf16 steps of 2^-8 three times over; codes are off by up to 2^-8 of the largest of 32 values: a few percent
    for got, want in ((y, out.detach()), (dx, full[0].grad), (bucket[:sizes[0]].view_as(w1), full[1].grad),
                      (bucket[sizes[0]:].view_as(w2), full[2].grad)):
        off_by = (got.cpu().double() - want).norm() / want.norm()
        assert off_by < 0.05, float(off_by)
    assert not bucket[:sizes[0]].view_as(w1)[1].any()  # the expert without rows
    # the codec on the bucket and on a copy of it
    errors = []
    for values in (bucket, bucket.clone()):
        errors.append(torch.zeros(group.total, device="cuda"))
        group.compress(values, errors[-1], 1.5)
    torch.cuda.synchronize()
    assert errors[0].any() and torch.equal(*errors)


def test_layer_in_8_bit_integers(tlc):
    """A layer's three products in 8-bit integers, and its experts' forward pass, near those of the values."""
    rows, k, n = 257, 300, 200
    g = gen(6)
    x, w, dy = randn(g, rows, k).cuda(), randn(g, n, k, scale=k ** -0.5).cuda(), randn(g, rows, n).cuda()
    y = tlc.q8_product(tlc.q8_pack_rows(x), tlc.q8_pack_rows(w), torch.float32)
    dx = tlc.q8_product(tlc.q8_pack_rows(dy), tlc.q8_pack_columns(w), torch.float32)
    dw = tlc.q8_product(tlc.q8_pack_columns(dy), tlc.q8_pack_columns(x), torch.float32)
    for got, a, b in ((y, x, w.t()), (dx, dy, w), (dw, dy.t(), x)):
        # a code is off by half a scale, the scale being a 127th of the largest of normal numbers (below 5 of them):
        # 0.5/127*5/sqrt(3) = 1.1% of their size on either side, independently: 1.6%
        want = a.double() @ b.double()
        assert ((got.double() - want).norm() / want.norm()).item() < 0.03
    w3 = randn(g, 3, n, k, scale=k ** -0.5).cuda()
    off = offsets_of([100, 0, 150]).cuda()
    x8, w8 = tlc.q8_pack_rows(x), tlc.q8_pack_rows(w3.view(3 * n, k))
    y = tlc.q8_product(x8, w8, torch.float32, offsets=off)
    one = tlc.q8_product(tlc.Rows8(x8.codes[100:250], x8.scales[100:250], k),
                         tlc.Rows8(w8.codes[2 * n:], w8.scales[2 * n:], k), torch.float32)
    assert torch.equal(y[100:250], one)


def step8(tlc, x, w, dy, off, w3, flat):
    y = tlc.q8_product(tlc.q8_pack_rows(x), tlc.q8_pack_rows(w))
    dx = tlc.q8_product(tlc.q8_pack_rows(dy), tlc.q8_pack_columns(w))
    tlc.q8_product(tlc.q8_pack_columns(dy), tlc.q8_pack_columns(x), torch.float32, y=flat.view(w.shape),
                   accumulate=True)
    z = torch.zeros_like(y)
    tlc.q8_product(tlc.q8_pack_rows(x), tlc.q8_pack_rows(w3.view(-1, w3.shape[2])), offsets=off, y=z)
    return y, dx, z


def test_captured_and_replayed(tlc):
    counts, cols, wide = [200, 0, 70, 30], 128, 192
    x, w1, w2, off, dout = layer_inputs(counts, cols, wide, torch.bfloat16, 5)
    n = w1[0].numel()
    dy = torch.zeros(x.shape[0], wide, dtype=torch.bfloat16, device="cuda")
    bucket, flat = torch.zeros(2 * 4 * n, device="cuda"), torch.zeros(n, device="cuda")

    def both(bucket, flat):
        return (*layer(tlc, x, w1, w2, off, dout, bucket, ckpt8_ref.E4M3),
                *step8(tlc, x, w1[0], dy, off, w1, flat))

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        both(bucket, flat)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(bucket, flat)
    for r in range(4):
        g = gen(90 + r)
        x.copy_(randn(g, *x.shape, dtype=torch.bfloat16))
        dout.copy_(randn(g, *dout.shape, dtype=torch.bfloat16))
        dy.copy_(randn(g, *dy.shape, dtype=torch.bfloat16))
        ends = torch.sort(torch.randint(0, 301, (3,), generator=g)).values.tolist()
        off.copy_(torch.tensor([0, *ends, 300]))  # other shares of the rows in the same graph
        start = randn(g, n).cuda()
        flat.copy_(start)
        bucket.fill_(math.nan)
        for o in outs:
            o.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (*outs, bucket, flat)]
        eager = torch.zeros_like(bucket)
        want = both(eager, start)
        for i, (a, b) in enumerate(zip(got, (*want, eager, start))):
            assert torch.equal(a, b), (r, i)


def test_on_other_streams(tlc):
    """The same calls on streams of their own, two at a time, each with a workspace of its own."""
    counts, cols, wide = [100, 33, 0, 167], 256, 320
    x, w1, w2, off, dout = layer_inputs(counts, cols, wide, torch.bfloat16, 7)
    q, w8 = tlc.q8_pack_rows(x), tlc.q8_pack_columns(w1.view(-1, cols).t().contiguous())
    x8 = tlc.ckpt8_pack(x, ckpt8_ref.INT8)

    def calls(stream):
        return [tlc.expert_product(x, w1, off, stream=stream), tlc.expert_input_grad(dout, w2, off, stream=stream),
                tlc.expert_weight_grad(dout, x8, off, stream=stream), tlc.q8_pack_rows(x, stream=stream).codes,
                tlc.q8_pack_columns(x, stream=stream).codes, tlc.q8_product(q, w8, offsets=off, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [calls(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_refusals(tlc):
    x = torch.zeros(6, 40, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(6, 24, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 24, 40, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 6], device="cuda")
    q, w8 = tlc.q8_pack_rows(x), tlc.q8_pack_rows(w.view(48, 40))
    x8 = tlc.ckpt8_pack(x, ckpt8_ref.INT8)
    f32 = torch.float32
    refused = [
        lambda: tlc.q8_pack_rows(x.double()),
        lambda: tlc.q8_pack_rows(x.cpu()),
        lambda: tlc.q8_pack_rows(x[0]),
        lambda: tlc.q8_pack_rows(x, out=tlc.q8_pack_rows(x[:3])),
        lambda: tlc.q8_pack_rows(torch.zeros(1, 131073, dtype=torch.bfloat16, device="cuda")),
        lambda: tlc.q8_pack_columns(x, out=q),
        lambda: tlc.q8_pack_columns(x[:0]),
        lambda: tlc.q8_pack_columns(torch.zeros(131073, 1, dtype=torch.bfloat16, device="cuda")),
        lambda: tlc.q8_pack_columns(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: tlc.q8_product(q, w8, torch.float64),
        lambda: tlc.q8_product(q, w8, offsets=off[:1]),
        lambda: tlc.q8_product(q, w8, offsets=off.int()),
        lambda: tlc.q8_product(q, w8, offsets=off.cpu()),
        lambda: tlc.q8_product(q, w8, offsets=torch.zeros(6, dtype=torch.int64, device="cuda")),
        lambda: tlc.q8_product(q, tlc.Rows8(w8.codes, w8.scales, 41)),
        lambda: tlc.q8_product(q, tlc.Rows8(w8.codes, w8.scales[:5], 40)),
        lambda: tlc.q8_product(q, tlc.Rows8(w8.codes[:, :40], w8.scales, 40)),
        lambda: tlc.q8_product(tlc.Rows8(q.codes.view(torch.uint8), q.scales, 40), w8),
        lambda: tlc.q8_product(q, w8, y=torch.zeros(6, 24, device="cuda")),
        lambda: tlc.q8_product(q, w8, accumulate=True),
        lambda: tlc.q8_product(q, w8, torch.bfloat16, y=torch.zeros(6, 48, dtype=torch.bfloat16, device="cuda"),
                               accumulate=True),
        lambda: tlc.q8_product(q, w8, f32, y=torch.zeros(6, 48, device="cuda").t()),
        lambda: tlc.expert_product(x, w),
        lambda: tlc.expert_product(x, w[0]),
        lambda: tlc.expert_product(x, w.float(), off),
        lambda: tlc.expert_product(x, w[:, :, :39], off),
        lambda: tlc.expert_product(x, w.transpose(1, 2), off),
        lambda: tlc.expert_product(x, w, off[:2]),
        lambda: tlc.expert_product(x, w, off.view(1, 3)),
        lambda: tlc.expert_product(x, w, off, y=torch.zeros(6, 24, device="cuda")),
        lambda: tlc.expert_product(x, w[:0], off[:1]),
        lambda: tlc.expert_product(x.t(), w, off),
        lambda: tlc.expert_input_grad(x, w, off),
        lambda: tlc.expert_input_grad(dy, w, None),
        lambda: tlc.expert_input_grad(dy, w, off, dx=dy),
        lambda: tlc.expert_weight_grad(dy[:3], x8, off),
        lambda: tlc.expert_weight_grad(dy, x8, off[:1]),
        lambda: tlc.expert_weight_grad(dy, x8, off, dw=torch.zeros(24, 40, device="cuda")),
        lambda: tlc.expert_weight_grad(dy, x8, off, dw=torch.zeros(1, 24, 40, device="cuda").expand(2, 24, 40)),
        lambda: tlc.expert_weight_grad(dy, x8, off, accumulate=True),
        lambda: tlc.expert_weight_grad(dy, x8, off, col_scale=torch.zeros(39, device="cuda")),
        lambda: tlc.expert_weight_grad(dy, x8, off, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for k, call in enumerate(refused):
        with pytest.raises((ValueError, tlc.TLCError)):
            call()
            raise AssertionError(f"call {k} was taken")
    torch.cuda.synchronize()
