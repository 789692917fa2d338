"""The 8-bit integer and grouped products on the host: layout and workspace
sizes and every refusal that is made before a launch.  No GPU needed: pointers
are never followed."""
import ctypes

import pytest
import torch

from gradient_compression_distributed_lc_amd import tlc

V = ctypes.c_void_p
P = V(0x10000)  # 256-byte aligned
ODD, TWO, FOUR = V(0x10001), V(0x10002), V(0x10004)
BIG = 1 << 31
BAD = tlc.ERR_INVALID_ARG


def L():
    return tlc.lib()


def refuses(f, good, changes, code=BAD):
    for change in changes:
        a = list(good)
        for at, v in change.items():
            a[at] = v
        assert f(*a) == code, change


def test_code_stride():
    for cols, stride in [(1, 128), (128, 128), (129, 256), (4096, 4096), (131072, 131072)]:
        assert tlc.q8_code_stride(cols) == stride
    for cols in (0, 131073, BIG):
        assert tlc.q8_code_stride(cols) == 0


def test_workspace_sizes():
    for rows, cols in [(0, 4), (4, 0), (131073, 4), (4, BIG)]:
        assert tlc.q8_pack_columns_workspace_size(rows, cols) == 0
    for rows in (1, 100, 131072):
        for cols in (1, 33, 1024, 100000):
            v = tlc.q8_pack_columns_workspace_size(rows, cols)
            assert v >= 256 and v % 256 == 0 and v <= 32 * 4 * (cols + 255)
    for experts in (0, 65537):
        assert tlc.expert_weight_grad_workspace_size(10, 64, 64, experts) == 0
    assert tlc.expert_weight_grad_workspace_size(BIG, 64, 64, 2) == 0
    for rows in (0, 1, 1000, 1 << 20):
        for experts in (1, 7, 64):
            v = tlc.expert_weight_grad_workspace_size(rows, 512, 96, experts)
            assert v >= 256 and v % 256 == 0
            assert v <= 256 + 32 * experts * 512 * 512 * 4
    # one expert with every row is the dense gradient
    for rows, n, cols in [(4096, 1024, 4096), (333, 1000, 515), (100000, 128, 128)]:
        assert tlc.expert_weight_grad_workspace_size(rows, n, cols, 1) == \
            tlc.ckpt8_weight_grad_workspace_size(rows, n, cols)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        for args in [(BIG, 8, 8, 1), (8, 0, 8, 1), (8, 8, 0, 1), (8, 8, 8, 0), (8, 8, 8, 65537)]:
            assert tlc.expert_product_workspace_size(*args, dt) == 0
            assert tlc.expert_input_grad_workspace_size(*args, dt) == 0
        for args in [(1, 8192, 8192, 1), (100, 64, 64, 8), (16384, 4096, 4096, 8)]:
            assert tlc.expert_product_workspace_size(*args, dt) % 256 == 0
            assert tlc.expert_input_grad_workspace_size(*args, dt) % 256 == 0


def test_pack_refusals():
    #       x  xs  dt r  c   codes scales st
    good = [P, 64, 2, 4, 40, P, P, None]
    refuses(L().tlc_q8_pack_rows, good,
            [{0: None}, {0: ODD}, {1: 39}, {1: BIG}, {2: 3}, {2: -1}, {3: BIG}, {4: 0}, {4: 131073, 1: 131073},
             {5: None}, {5: FOUR}, {6: None}, {6: TWO}, {0: TWO, 2: 0}])
    good = [P, 64, 2, 4, 40, P, P, P, 1 << 20, None]
    refuses(L().tlc_q8_pack_columns, good,
            [{0: None}, {0: ODD}, {1: 39}, {1: BIG}, {2: 3}, {3: 0}, {3: 131073}, {4: 0}, {4: BIG}, {5: None},
             {5: FOUR}, {6: None}, {6: TWO}])
    refuses(L().tlc_q8_pack_columns, good, [{7: None}, {7: FOUR}, {8: 16}], tlc.ERR_WORKSPACE)


def test_product8_refusals():
    #       a  sa rows w  sw n  k   off ex y  ys  dt acc ws bytes st
    good = [P, P, 4, P, P, 24, 40, P, 2, P, 24, 0, 0, P, 1 << 30, None]
    refuses(L().tlc_q8_product, good,
            [{0: None}, {0: FOUR}, {1: None}, {1: TWO}, {2: BIG}, {3: None}, {3: FOUR}, {4: None}, {4: TWO}, {5: 0},
             {5: BIG}, {6: 0}, {6: 131073}, {7: None}, {7: FOUR}, {8: 0}, {8: 65537}, {9: None}, {9: TWO}, {10: 23},
             {10: BIG}, {11: 3}, {11: 2, 12: 1}])
    # more than 2^24 tiles of 128 x 128
    refuses(L().tlc_q8_product, good, [{2: 1 << 24, 5: 1 << 24, 10: 1 << 24}])


@pytest.mark.parametrize("name", ["tlc_expert_product", "tlc_expert_input_grad"])
def test_expert_refusals(name):
    #       x  xs  dt r  k   w  ws  we   n   off ex y  ys  ws bytes st
    good = [P, 64, 2, 4, 40, P, 64, 960, 40, P, 2, P, 40, P, 1 << 30, None]
    refuses(getattr(L(), name), good,
            [{0: None}, {0: ODD}, {1: 39}, {1: BIG}, {2: 3}, {3: BIG}, {4: 0}, {4: BIG}, {5: None}, {5: ODD}, {6: 39},
             {6: BIG}, {7: 1 << 48}, {8: 0}, {8: BIG}, {9: None}, {9: FOUR}, {10: 0}, {10: 65537}, {11: None},
             {11: ODD}, {12: 39}, {12: BIG}, {0: TWO, 2: 0}, {5: TWO, 2: 0}, {11: TWO, 2: 0},
             {3: 1 << 24, 8: 1 << 24, 12: 1 << 24, 6: 1 << 24}])


def test_expert_weight_grad_refusals():
    #       dy ds  dt r  n   fmt c  s  cols off ex cs cdt dw st  est  acc ws bytes st
    good = [P, 64, 2, 4, 24, 1, P, P, 40, P, 2, None, 0, P, 40, 960, 0, P, 1 << 30, None]
    refuses(L().tlc_expert_weight_grad, good,
            [{0: None}, {0: ODD}, {1: 23}, {1: BIG}, {2: 3}, {3: BIG}, {4: 0}, {4: BIG}, {5: 0}, {5: 3}, {6: None},
             {6: FOUR}, {7: None}, {7: TWO}, {8: 0}, {9: None}, {9: FOUR}, {10: 0}, {10: 65537}, {11: ODD},
             {11: P, 12: 1}, {13: None}, {13: TWO}, {14: 39}, {15: 959}, {15: 1 << 48},
             {4: 1 << 20, 1: 1 << 20, 8: 1 << 20, 14: 1 << 20, 15: 1 << 41}])
    refuses(L().tlc_expert_weight_grad, good, [{17: None}, {17: FOUR}, {18: 16}], tlc.ERR_WORKSPACE)


def test_binding_refuses_tensors_on_the_host():
    x = torch.zeros(4, 40)
    q = tlc.Rows8(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4), 40)
    c = tlc.Checkpoint8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 40, 1)
    w = torch.zeros(1, 24, 40)
    for call in (lambda: tlc.q8_pack_rows(x), lambda: tlc.q8_pack_columns(x), lambda: tlc.q8_product(q, q),
                 lambda: tlc.expert_product(x, w), lambda: tlc.expert_input_grad(x[:, :24], w),
                 lambda: tlc.expert_weight_grad(x, c)):
        with pytest.raises(ValueError):
            call()
