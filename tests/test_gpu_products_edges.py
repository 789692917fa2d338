"""8-bit integer products and products grouped by expert on the GPU, where the
chip is full and the sizes are awkward: many blocks of the kernel for few rows,
sums in slices that are added to, scales at the ends of the range in every
kernel, the larger tile without offsets, thousands of experts, calls at once."""
import math
import weakref

import pytest
import torch

import ckpt8_ref
import products_ref as ref
from gpu_util import say
from test_gpu_products import DTYPES, LEAST, U, assert_close, gen, offsets_of, randn, strided, whole

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
