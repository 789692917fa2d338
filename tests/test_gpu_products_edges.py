"""8-bit integer products and products grouped by expert on the GPU, where the
chip is full and the sizes are awkward: many blocks of the kernel for few rows,
sums in slices that are added to, scales at the ends of the range in every
kernel, the larger tile without offsets, thousands of experts, calls at once."""
import math
import threading
import weakref

import pytest
import torch

import ckpt8_ref
import products_ref as ref
from gpu_util import say
from test_gpu_products import (DTYPES, LEAST, U, assert_close, gen, offsets_of, randn, random_codes, rows8, strided,
                               whole)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlc():
    from gradient_compression_distributed_lc_amd import tlc
    return tlc


def uneven(g, rows, experts):
    """Rows of each expert, some of them many, some none."""
    share = torch.rand(experts, generator=g).log().neg()
    share[::7] *= 4
    share[3::11] = 0
    counts = (share / share.sum() * rows).long()
    counts[experts // 2] += rows - int(counts.sum())
    return counts.tolist()


# ---- few rows, many blocks ---------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [27, 121, 123, 124, 244, 1051])
def test_few_rows_on_a_full_chip(tlc, k, dtype):
    """Many more blocks than compute units, so that wavefronts share a SIMD, and rows that end inside a turn of 128
    bytes, in its second half too: whole numbers, so exact."""
    say(f"few rows, full chip k={k} {dtype}")
    rows, n = 16, 16384
    g = gen(k)
    x, w = whole(g, rows, k, dtype=dtype), whole(g, 1, n, k, dtype=dtype)
    want = (x.double() @ w[0].double().t()).to(dtype)
    xd, wd = x.cuda(), w.cuda()
    for _ in range(4):
        y = torch.full((rows, n), math.nan, dtype=dtype, device="cuda")
        tlc.expert_product(xd, wd, y=y)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("seed", [1, 2, 3])
@pytest.mark.parametrize("k,n", [(123, 515), (244, 183), (121, 952)])
@pytest.mark.parametrize("experts", [16, 48, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_step_of_many_uneven_experts(tlc, dtype, experts, k, n, seed):
    """Output, input gradient and weight gradients one after the other, rows up to those of the kernel for few rows and
    one more, several experts of more than 16: every output against 64 bits after the last call."""
    most = 32 * experts if dtype == torch.float32 else 8 * experts + 16
    for rows in (most // 3, most, most + 1):
        say(f"step of many experts {experts} {rows} {k} {n} {dtype} {seed}")
        g = gen(rows * 31 + seed)
        counts = uneven(g, rows, experts)
        assert sum(counts) == rows and (rows < most or max(counts) > 16)
        x, dy = randn(g, rows, k, dtype=dtype), randn(g, rows, n, dtype=dtype, scale=0.1)
        w = randn(g, experts, n, k, dtype=dtype, scale=k ** -0.5)
        codes, scales = ckpt8_ref.encode(x.float(), ckpt8_ref.INT8)
        values = ckpt8_ref.decode(codes, scales, ckpt8_ref.INT8, k)
        offsets = offsets_of(counts)
        off, wd, xd, dyd = offsets.cuda(), strided(w, 3, 1), strided(x, 5, 1), strided(dy, 3)
        x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), k, ckpt8_ref.INT8)
        y = torch.full((rows, n), math.nan, dtype=dtype, device="cuda")
        dx = torch.full((rows, k), math.nan, dtype=dtype, device="cuda")
        dw = torch.full((experts, n, k), math.nan, device="cuda")
        tlc.expert_product(xd, wd, off, y=y)
        tlc.expert_input_grad(dyd, wd, off, dx=dx)
        tlc.expert_weight_grad(dyd, x8, off, dw=dw)
        torch.cuda.synchronize()
        for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
            we, dye = w[e].double(), dy[b:t].double()
            for name, got, left, right, terms, out in (("y", y[b:t], x[b:t].double(), we.t(), k, dtype),
                                                       ("dx", dx[b:t], dye, we, n, dtype),
                                                       ("dw", dw[e], dye.t(), values[b:t], 3 * (t - b), torch.float32)):
                want, size = left @ right, left.abs() @ right.abs()
                # each of `terms` additions in fp32, and in fp32 each product, rounds by 2^-24 of at most `size`; dy is
                # up to three numbers in the last, whose products are exact
                bound = 2 * terms * 2.0 ** -24 * size + U[out] * want.abs() * 1.01 + LEAST[out]
                assert_close(got, want, bound, (name, e, rows))


# ---- workspaces --------------------------------------------------------------


def test_workspace_lives_until_the_call_is_launched(tlc, monkeypatch):
    """A call's own workspace is not given back before its kernels are launched: another thread's call on the same stream
    could be given it in between, and its results be written over."""
    rows, k, n = 128, 4096, 256
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, n, k, dtype=torch.bfloat16, device="cuda")
    a8, w8 = tlc.q8_pack_rows(x), tlc.q8_pack_rows(w[0])
    assert tlc.expert_product_workspace_size(rows, k, n, 1, x.dtype) and tlc.q8_product_workspace_size(rows, n, k)
    assert tlc.expert_input_grad_workspace_size(rows, k, n, 1, x.dtype)
    real, made, seen = tlc.lib(), [], []
    make = tlc._ckpt8_workspace

    def made_and_watched(nbytes, device, workspace):
        t = make(nbytes, device, workspace)
        made.append(weakref.ref(t))
        return t

    class Watch:
        def __getattr__(self, name):
            f = getattr(real, name)

            def call(*args):
                if not name.endswith("_size"):
                    seen.append((name, made[-1]() is not None))
                return f(*args)
            return call

    monkeypatch.setattr(tlc, "_ckpt8_workspace", made_and_watched)
    monkeypatch.setattr(tlc, "lib", lambda: Watch())
    tlc.expert_product(x, w)
    tlc.expert_input_grad(x, w.transpose(1, 2).contiguous())
    tlc.q8_product(a8, w8)
    torch.cuda.synchronize()
    assert seen == [("tlc_expert_product", True), ("tlc_expert_input_grad", True), ("tlc_q8_product", True)]


# ---- sums in slices ----------------------------------------------------------


@pytest.mark.parametrize("rows,n,k", [(140, 77, 8191), (768, 768, 4096), (43, 1000, 20000)])
@pytest.mark.parametrize("experts", [0, 3])
def test_product8_in_slices_added_to_a_bucket(tlc, experts, rows, n, k):
    """Reductions cut into slices, whose sums are added to a strided place of whole numbers."""
    say(f"product8 in slices, added {rows}x{n}x{k} {experts}")
    many = max(experts, 1)
    assert tlc.q8_product_workspace_size(rows, n, k, many) > 0
    g = gen(rows + k)
    (a, _), (w, _) = random_codes(g, rows, k), random_codes(g, many * n, k)
    sa, sw = torch.ones(rows), torch.ones(many * n)
    offsets = offsets_of([rows - rows // 3, 0, rows // 3 - 2], 1) if experts else torch.tensor([0, rows])
    start = whole(g, rows, n, most=1000)
    want = start.double()
    for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
        sums = a[b:t].float().cuda() @ w[e * n:(e + 1) * n].float().cuda().t()  # below 2^24: exact
        assert sums.numel() == 0 or sums.abs().max() < 2 ** 23
        want[b:t] += sums.cpu().double()
    bucket = strided(start, 3, 2)
    off = offsets.cuda() if experts else None
    y = tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32, offsets=off, y=bucket,
                       accumulate=True)
    assert y is bucket and torch.equal(y.cpu().double(), want)
    assert torch.isnan(torch.as_strided(bucket, (rows, 3), (n + 3, 1), bucket.storage_offset() + n)).all()


def test_a_smaller_batch_may_need_a_larger_workspace(tlc):
    """A workspace that holds for many rows can be too small for fewer, whose reduction is cut: the call is refused, and
    the size for just these rows is taken."""
    k = n = 4096
    sizes = {r: tlc.expert_product_workspace_size(r, k, n, 1, torch.bfloat16) for r in (1024, 4096)}
    assert sizes[1024] > sizes[4096] == 0
    x = whole(gen(2), 1024, k, dtype=torch.bfloat16, most=1).cuda()
    w = whole(gen(3), 1, n, k, dtype=torch.bfloat16, most=1).cuda()
    off = offsets_of([1024]).cuda()
    with pytest.raises(tlc.TLCError):
        tlc.expert_product(x, w, off, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    y = tlc.expert_product(x, w, off, workspace=torch.empty(sizes[1024], dtype=torch.uint8, device="cuda"))
    assert torch.equal(y, (x.float() @ w[0].float().t()).bfloat16())


@pytest.mark.parametrize("counts", [[70, 0, 130, 9], [2, 0, 5, 1]])
def test_input_gradient_by_expert_from_columns_packed_one_by_one(tlc, counts):
    """8 bits by expert: each expert's columns packed into its part of the codes, then one product of dy's rows."""
    g = gen(16)
    k, n, experts, rows = 300, 200, len(counts), sum(counts)
    w, dy = randn(g, experts, n, k, scale=k ** -0.5).cuda(), randn(g, rows, n).cuda()
    back = tlc.Rows8(torch.empty(experts * k, 256, dtype=torch.int8, device="cuda"),
                     torch.empty(experts * k, device="cuda"), n)
    for e in range(experts):
        part = slice(e * k, (e + 1) * k)
        tlc.q8_pack_columns(w[e], out=tlc.Rows8(back.codes[part], back.scales[part], n))
    off = offsets_of(counts)
    dx = tlc.q8_product(tlc.q8_pack_rows(dy), back, torch.float32, offsets=off.cuda())
    for e, (b, t) in enumerate(ref.spans(off.tolist(), rows)):
        (a, sa), (c, sc) = ref.pack_rows(dy[b:t].cpu()) if t > b else (None, None), ref.pack_columns(w[e].cpu())
        if t > b:
            want, _ = ref.product8(a, sa, c, sc)
            # sums below 2^24 are exact, the products with the scales round
            assert_close(dx[b:t], want, 3.01 * 2.0 ** -24 * want.abs(), e)


# ---- codes and scales --------------------------------------------------------


@pytest.mark.parametrize("rows", [3, 200])
def test_product8_of_codes_of_the_least_value(tlc, rows):
    """-128 by -128 over 131071: 2^31 less 2^14, the largest sum there is, exact before it is rounded to fp32."""
    k = 131071
    a, w = torch.full((rows, 131072), -128, dtype=torch.int8), torch.full((40, 131072), -128, dtype=torch.int8)
    a[:, k:], w[:, k:] = 0, 0
    a[1], w[7, ::3] = 127, 126
    a[1, k:] = 0
    w[7, k:] = 0
    one = torch.ones
    want = a.double() @ w.double().t()
    assert want.max() == 2 ** 31 - 2 ** 14
    y = tlc.q8_product(rows8(tlc, a, one(rows), k), rows8(tlc, w, one(40), k), torch.float32)
    assert torch.equal(y.cpu(), want.float())



@pytest.mark.parametrize("rows,n,k", [(7, 203, 64), (200, 203, 64), (140, 77, 8191), (700, 520, 300)])
def test_product8_scales_of_every_size_side_by_side(tlc, rows, n, k):
    """Scales from 2^-126 to 2^121 and NaN next to each other in a wavefront's rows and columns, in the kernels for few
    rows, for tiles with a ragged end and for slices.  Scales are powers of two and sums below 2^24, so one rounding at
    most, to a subnormal value, is what the result differs by from the exact one."""
    say(f"product8 scales {rows}x{n}x{k}")
    g = gen(rows + n)
    a, w = torch.zeros(rows, -(-k // 128) * 128, dtype=torch.int8), torch.zeros(n, -(-k // 128) * 128, dtype=torch.int8)
    a[:, :k], w[:, :k] = whole(g, rows, k).to(torch.int8), whole(g, n, k).to(torch.int8)
    exponents = torch.tensor([-126, -100, -20, 0, 5, 60, 96, 97, 120, 121])
    sa = torch.ldexp(torch.ones(rows), exponents[torch.randint(0, 10, (rows,), generator=g)])
    sw = torch.ldexp(torch.ones(n), exponents[torch.randint(0, 10, (n,), generator=g)])
    sa[3], sw[n - 2], sw[5] = math.nan, math.nan, math.nan
    want, sums = ref.product8(a, sa, w, sw)
    assert sums.abs().max() < 2 ** 24
    want = want.float()
    assert torch.isinf(want).any() and (want.abs() < 2.0 ** -126).any() and torch.isfinite(want).any()
    for add in (False, True):
        start = whole(g, rows, n, most=1000)
        y = strided(start, 1, 1)
        tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32, y=y, accumulate=add)
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.5, posinf=8.5, neginf=9.5),
                           torch.nan_to_num(want + start if add else want, nan=7.5, posinf=8.5, neginf=9.5)), add


# ---- the larger tile without offsets -----------------------------------------


@pytest.mark.parametrize("rows", [4008, 4264])
@pytest.mark.parametrize("k", [1096, 1027])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_large_dense_products_of_whole_numbers_are_exact(tlc, dtype, k, rows):
    """256 large tiles in one round, and 272, whose last 16 smaller ones compute, the host deciding."""
    say(f"large dense products {rows} {k} {dtype}")
    n = 4091
    g = gen(k + rows)
    x, w = whole(g, rows, k, dtype=dtype).cuda(), whole(g, 1, n, k, dtype=dtype).cuda()
    want = (x.float() @ w[0].float().t()).to(dtype)  # whole numbers below 2^24
    assert torch.equal(tlc.expert_product(x, w), want)
    assert torch.equal(tlc.expert_input_grad(x, w.transpose(1, 2).contiguous()), want)
    z = strided(torch.full((rows, n), math.nan, dtype=dtype), 3, 1)
    tlc.expert_product(strided(x.cpu(), 5, 1), strided(w.cpu(), 3), y=z)
    assert torch.equal(z, want)


@pytest.mark.parametrize("rows", [4008, 4264])
def test_large_dense_product8_is_exact(tlc, rows):
    n, k = 4091, 2055
    g = gen(rows)
    a, w = torch.zeros(rows, 2176, dtype=torch.int8), torch.zeros(n, 2176, dtype=torch.int8)
    a[:, :k] = torch.randint(-80, 81, (rows, k), generator=g).to(torch.int8)
    w[:, :k] = torch.randint(-80, 81, (n, k), generator=g).to(torch.int8)
    sa = torch.ldexp(torch.ones(rows), torch.randint(-3, 4, (rows,), generator=g))
    sa[70::128] = 2.0 ** 97  # with a scale that reverses the order of the products
    sw = torch.ldexp(torch.ones(n), torch.randint(-3, 4, (n,), generator=g))
    want = (a.cuda().float() @ w.cuda().float().t()) * sa.cuda()[:, None] * sw.cuda()  # 2055 * 80 * 80 is below 2^24
    assert torch.equal(tlc.q8_product(rows8(tlc, a, sa, k), rows8(tlc, w, sw, k), torch.float32), want)


# ---- thousands of experts ----------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", [1000, 65536])
@pytest.mark.parametrize("k,n,rows", [(40, 24, 3000), (3, 8, 300), (136, 8, 20000)])
def test_thousands_of_experts(tlc, k, n, rows, experts, dtype):
    """Up to as many experts as the calls take: whole numbers, so exact."""
    say(f"thousands of experts {experts} {k} {n} {rows} {dtype}")
    g = gen(experts + k)
    who = torch.sort(torch.randint(0, experts, (rows,), generator=g)).values
    who[: rows // 3] = who[rows // 3]  # a long one, the first with rows
    offsets = torch.searchsorted(who, torch.arange(experts + 1)).cuda()
    who = who.cuda()
    x, dy = whole(g, rows, k, dtype=dtype).cuda(), whole(g, rows, n, dtype=dtype).cuda()
    w = torch.randint(-3, 4, (experts, n, k), device="cuda").to(dtype)
    y, dx = tlc.expert_product(x, w, offsets), tlc.expert_input_grad(dy, w, offsets)
    x8 = tlc.ckpt8_pack(x, ckpt8_ref.INT8)
    dw = tlc.expert_weight_grad(dy, x8, offsets)
    q = tlc.q8_pack_rows(x), tlc.q8_pack_rows(w.view(experts * n, k))
    y8 = tlc.q8_product(*q, torch.float32, offsets=offsets)
    for b in range(0, rows, 1000):
        some = slice(b, b + 1000)
        we, xs, ds = w[who[some]].float(), x[some].float(), dy[some].float()
        assert torch.equal(y[some], (we * xs[:, None, :]).sum(2).to(dtype))
        assert torch.equal(dx[some], (we * ds[:, :, None]).sum(1).to(dtype))
        codes = q[1].codes.view(experts, n, -1)[who[some]].float() * q[0].codes[some].float()[:, None, :]
        scales = q[0].scales[some][:, None] * q[1].scales.view(experts, n)[who[some]]
        # the sum's conversion is exact here, the two products with the scales round, in either order
        assert ((y8[some] - codes.sum(2) * scales).abs() <= 4 * 2.0 ** -24 * (codes.sum(2) * scales).abs()).all()
    ends = offsets.tolist()
    some = sorted({0, 1, experts - 1, int(who[0]), *who[:: max(1, rows // 50)].tolist()})
    for e in some:
        b, t = ends[e], ends[e + 1]
        assert torch.equal(dw[e], dy[b:t].float().t() @ x[b:t].float()), e
    empty = offsets[1:] == offsets[:-1]
    assert not dw[empty].any()


# ---- weight gradients --------------------------------------------------------


@pytest.mark.parametrize("fmt", [ckpt8_ref.INT8, ckpt8_ref.E4M3])
@pytest.mark.parametrize("dtype", DTYPES)
def test_expert_weight_gradient_in_slices_added_to_a_bucket(tlc, dtype, fmt):
    """Small weights over many rows, whose sums over slices of the rows are added to a strided place."""
    counts, n, cols = [5000, 0, 9001], 130, 77
    assert tlc.expert_weight_grad_workspace_size(sum(counts) + 3, n, cols, 3) > 256
    g = gen(12)
    offsets, rows = offsets_of(counts, 1), sum(counts) + 3
    dy, x = whole(g, rows, n, dtype=dtype, most=2), whole(g, rows, cols, most=2)
    codes, scales = ckpt8_ref.encode(x, fmt)
    x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, fmt)
    start = whole(g, 3, n, cols, most=50)
    bucket = strided(start, 3, 2)
    tlc.expert_weight_grad(strided(dy, 1, 1), x8, offsets.cuda(), dw=bucket, accumulate=True)
    for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
        assert torch.equal(bucket[e].cpu(), start[e] + dy[b:t].float().t() @ x[b:t]), e  # below 2^24: exact
    gaps = torch.as_strided(bucket, (3 * n, 3), (cols + 3, 1), bucket.storage_offset() + cols)
    assert torch.isnan(gaps).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_expert_weight_gradient_of_values_that_are_not_finite(tlc, dtype):
    """An infinity or NaN of a row reaches its own expert's gradient only, in the row of dw or the column that it is in;
    rows of no expert are not read."""
    n, cols, counts = 70, 100, [40, 0, 65, 31]
    g = gen(13)
    offsets, rows = offsets_of(counts, 2), sum(counts) + 5
    dy, x = whole(g, rows, n, dtype=dtype), whole(g, rows, cols)
    dy[0], dy[1], dy[-3:], x[0], x[-2:] = math.nan, math.inf, math.nan, math.nan, math.inf
    dy[2 + 39, 7], dy[2 + 40, 8], x[2 + 39, 70] = math.inf, math.nan, math.nan  # the first's last row, the third's first
    codes, scales = ckpt8_ref.encode(x, ckpt8_ref.INT8)
    x8 = tlc.Checkpoint8(codes.cuda(), scales.cuda(), cols, ckpt8_ref.INT8)
    dw = tlc.expert_weight_grad(dy.cuda(), x8, offsets.cuda()).cpu()
    bad = torch.zeros(4, n, cols, dtype=torch.bool)
    bad[0, 7], bad[2, 8] = True, True
    bad[0, :, 64:96] = True  # the group of 32 columns that has no scale
    assert not torch.isfinite(dw[bad]).any() and torch.isfinite(dw[~bad]).all()
    for e, (b, t) in enumerate(ref.spans(offsets.tolist(), rows)):
        want = dy[b:t].float().t() @ x[b:t]
        assert torch.equal(dw[e][~bad[e]], want[~bad[e]]), e


@pytest.mark.parametrize("rows,n,cols", [(333, 1000, 515), (5000, 128, 96)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_one_expert_without_offsets_is_the_dense_gradient(tlc, dtype, rows, n, cols):
    g = gen(14)
    dy, x = randn(g, rows, n, dtype=dtype).cuda(), randn(g, rows, cols, dtype=dtype).cuda()
    x8 = tlc.ckpt8_pack(x, ckpt8_ref.E4M3)
    dense = tlc.ckpt8_weight_grad(dy, x8)
    assert torch.equal(tlc.expert_weight_grad(dy, x8)[0], dense)
    # with offsets the rows are cut alike, at places that the device finds
    assert torch.equal(tlc.expert_weight_grad(dy, x8, offsets_of([rows]).cuda())[0], dense)


# ---- calls at once -----------------------------------------------------------


def test_calls_of_two_threads_at_once(tlc):
    """Two host threads, on one stream and on one of their own each: every result is that of a call alone."""
    g = gen(15)
    counts, k, n = [100, 0, 50, 6], 2048, 264
    off, w = offsets_of(counts).cuda(), randn(g, 4, n, k, dtype=torch.bfloat16, scale=k ** -0.5).cuda()
    assert tlc.expert_product_workspace_size(156, k, n, 4, w.dtype) > 0
    xs = [randn(g, 156, k, dtype=torch.bfloat16).cuda() for _ in range(2)]
    ds = [randn(g, 156, n, dtype=torch.bfloat16).cuda() for _ in range(2)]

    def calls(i, stream):
        return [tlc.expert_product(xs[i], w, off, stream=stream), tlc.expert_input_grad(ds[i], w, off, stream=stream),
                tlc.expert_weight_grad(ds[i], tlc.ckpt8_pack(xs[i], ckpt8_ref.INT8, stream=stream), off, stream=stream),
                tlc.q8_product(tlc.q8_pack_rows(xs[i], stream=stream), tlc.q8_pack_rows(xs[1 - i], stream=stream),
                               stream=stream)]

    want = [calls(i, None) for i in range(2)]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    for streams in ((one, one), (torch.cuda.Stream(), torch.cuda.Stream())):
        got = [[], []]

        def work(i):
            for _ in range(30):
                got[i].append(calls(i, streams[i]))

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for i in range(2):
            assert len(got[i]) == 30
            for r in got[i]:
                assert all(torch.equal(a, b) for a, b in zip(r, want[i]))
