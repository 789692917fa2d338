"""The 8-bit checkpoint calls on the host: layout sizes, workspace sizes and
every refusal that is made before a launch.  No GPU needed: pointers are never
followed."""
import ctypes

import pytest
import torch

from gradient_compression_distributed_lc_amd import tlc

import ckpt8_ref as ref

V = ctypes.c_void_p
P = V(0x10000)     # 256-byte aligned
ODD = V(0x10001)
TWO = V(0x10002)
FOUR = V(0x10004)
BIG = 1 << 31
BAD = tlc.ERR_INVALID_ARG


def L():
    return tlc.lib()


def test_strides():
    for cols, codes, scales in [(1, 32, 4), (32, 32, 4), (33, 64, 4), (128, 128, 4), (129, 160, 8), (4096, 4096, 128)]:
        assert tlc.ckpt8_code_stride(cols) == codes
        assert tlc.ckpt8_scale_stride(cols) == scales
    for cols in (0, BIG):
        assert tlc.ckpt8_code_stride(cols) == 0 and tlc.ckpt8_scale_stride(cols) == 0


def test_workspace_sizes():
    assert tlc.ckpt8_norm_grad_workspace_size(10, 0) == 0
    assert tlc.ckpt8_norm_grad_workspace_size(10, 16385) == 0
    assert tlc.ckpt8_norm_grad_workspace_size(BIG, 64) == 0
    assert tlc.ckpt8_weight_grad_workspace_size(10, 0, 64) == 0
    assert tlc.ckpt8_weight_grad_workspace_size(10, 64, 0) == 0
    assert tlc.ckpt8_weight_grad_workspace_size(BIG, 64, 64) == 0
    for rows in (0, 1, 100, 1 << 20):
        for cols in (1, 33, 1024, 16384):
            v = tlc.ckpt8_norm_grad_workspace_size(rows, cols)
            assert v >= 256 and v % 256 == 0
            # a row of fp32 sums per wavefront at most, of a bounded number of blocks
            assert v <= 256 + 4 * cols * min(rows + 3, 4 * 2048)
            w = tlc.ckpt8_weight_grad_workspace_size(rows, 512, cols)
            assert w >= 256 and w % 256 == 0


def test_pack_and_unpack_refusals():
    f = L().tlc_ckpt8_pack
    good = [P, 64, 2, 4, 40, 1, P, P, None]
    for at, v in [(0, None), (0, ODD), (1, 39), (1, BIG), (2, 3), (2, -1), (3, BIG), (4, 0), (4, BIG), (5, 0), (5, 3),
                  (6, None), (6, FOUR), (7, None), (7, TWO)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)
    a = list(good)
    a[0], a[2] = TWO, 0  # fp32 at an address that is not a multiple of 4
    assert f(*a) == BAD
    f = L().tlc_ckpt8_unpack
    good = [P, P, 1, 4, 40, P, 64, 2, None]
    for at, v in [(0, None), (0, FOUR), (1, None), (2, 0), (2, 3), (3, BIG), (4, 0), (5, None), (5, ODD), (6, 39),
                  (7, 3)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)


def test_act_refusals():
    f = L().tlc_ckpt8_act
    #       act a  as  b  bs  dt r  c   y  ys  fmt ac as bc bs
    good = [1, P, 64, P, 64, 2, 4, 40, P, 64, 1, P, P, P, P, None]
    for at, v in [(0, 0), (0, 4), (1, None), (1, ODD), (2, 39), (3, ODD), (4, 39), (5, 3), (6, BIG), (7, 0), (8, None),
                  (9, 39), (10, 0), (11, None), (11, FOUR), (12, None), (13, None), (14, None), (3, None)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)
    f = L().tlc_ckpt8_act_grad
    #       act ac as bc bs fmt dy ds dt r  c   da das db dbs yc ys
    good = [1, P, P, P, P, 1, P, 64, 2, 4, 40, P, 64, P, 64, P, P, None]
    for at, v in [(0, 0), (1, None), (2, None), (3, None), (4, None), (5, 3), (6, None), (6, ODD), (7, 39), (8, 3),
                  (9, BIG), (10, 0), (11, None), (12, 39), (13, None), (14, 39), (15, None), (15, FOUR), (16, None)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)


def test_norm_refusals():
    f = L().tlc_ckpt8_norm
    #       x  xs  r  rs  dt r  c   w  wd eps  wtd s  ss  y  ys  fmt c  s  rstd
    good = [P, 64, P, 64, 2, 4, 40, P, 2, 1e-5, 0, P, 64, P, 64, 1, P, P, P, None]
    nan, inf = float("nan"), float("inf")
    for at, v in [(0, None), (0, ODD), (1, 39), (2, ODD), (3, 39), (4, 3), (5, BIG), (6, 0), (6, 16385), (7, ODD),
                  (8, 3), (8, 1), (9, 0.0), (9, -1.0), (9, nan), (9, inf), (11, ODD), (12, 39), (13, ODD), (14, 39), (15, 0),
                  (16, None), (16, FOUR), (17, None), (18, TWO), (2, None)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)
    a = list(good)
    a[7], a[10] = None, 1  # weighted without a weight
    assert f(*a) == BAD
    a = list(good)
    a[13] = a[16] = a[17] = None  # nothing asked for
    assert f(*a) == BAD
    f = L().tlc_ckpt8_norm_grad
    #       dy ds  dt  dts dtype r c  sum ss fmt c  s  rstd w  wd dx dxs dw acc ws  nws
    good = [P, 64, P, 64, 2, 4, 40, None, 0, 1, P, P, P, P, 2, P, 64, P, 0, P, 1 << 20, None]
    for at, v in [(0, None), (1, 39), (2, ODD), (3, 39), (4, 3), (5, BIG), (6, 0), (6, 16385), (7, P), (9, 0),
                  (10, None), (11, None), (12, None), (12, TWO), (13, ODD), (14, 3), (14, 1), (15, None), (16, 39), (17, TWO)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)
    a = list(good)
    a[10] = a[11] = None  # neither a checkpoint nor the sum
    assert f(*a) == BAD
    for at, v in [(19, None), (19, FOUR), (20, 255)]:
        a = list(good)
        a[at] = v
        assert f(*a) == tlc.ERR_WORKSPACE, (at, v)


def test_weight_grad_refusals():
    f = L().tlc_ckpt8_weight_grad
    #       dy ds dt r  n   fmt c  s  cols cs cd dw ds acc ws nws
    good = [P, 64, 2, 4, 50, 1, P, P, 40, P, 2, P, 64, 0, P, 1 << 20, None]
    for at, v in [(0, None), (0, ODD), (1, 49), (2, 3), (3, BIG), (4, 0), (4, BIG), (5, 0), (6, None), (6, FOUR),
                  (7, None), (8, 0), (8, BIG), (9, ODD), (10, 3), (10, 1), (11, None), (11, TWO), (12, 39), (12, BIG)]:
        a = list(good)
        a[at] = v
        assert f(*a) == BAD, (at, v)
    for at, v in [(14, None), (14, FOUR), (15, 255)]:
        a = list(good)
        a[at] = v
        assert f(*a) == tlc.ERR_WORKSPACE, (at, v)


def test_tensors_that_are_not_on_a_gpu_are_refused():
    x = torch.zeros(4, 40)
    c = tlc.Checkpoint8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 40, 1)
    for call in (lambda: tlc.ckpt8_pack(x, 1), lambda: tlc.ckpt8_unpack(c), lambda: tlc.ckpt8_act(x, 1, 1),
                 lambda: tlc.ckpt8_act_grad(x, 1, c), lambda: tlc.ckpt8_norm(x, None, 1e-5, 1),
                 lambda: tlc.ckpt8_norm_grad(x, c, x[:, 0]), lambda: tlc.ckpt8_weight_grad(x, c)):
        with pytest.raises(ValueError, match="GPU|must be on"):
            call()


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_reference_of_the_format(fmt):
    """The 64-bit reference itself: nearest codes by search over all of them, and the worked scale borders."""
    vals = ref.code_values(torch.arange(256, dtype=torch.uint8), fmt)
    keep = vals.isfinite() & (vals.abs() <= ref.LARGEST[fmt])
    table = torch.unique(vals[keep])
    x = torch.randn(50, 32, generator=torch.Generator().manual_seed(1)).double() * 5
    codes, scales = ref.encode(x, fmt)
    s = torch.exp2(scales[:, :1].double() - 127)
    amax = x.abs().amax(1, keepdim=True)
    assert (amax <= ref.LARGEST[fmt] * s).all() and (amax > ref.LARGEST[fmt] * s / 2).all()
    q = x / s
    nearest = (q.unsqueeze(2) - table).abs().amin(2)
    assert torch.equal((ref.code_values(codes, fmt) - q).abs(), nearest)
    one = torch.zeros(1, 32, dtype=torch.float64)
    for amax, e in [(ref.LARGEST[fmt], 0), (ref.LARGEST[fmt] * 1.0001, 1), (ref.LARGEST[fmt] / 2, -1)]:
        one[0, 5] = -amax
        assert int(ref.encode(one, fmt)[1][0, 0]) == 127 + e
