"""The 8-bit integer products and the products grouped by expert in 64 bits, on the CPU."""
import torch

LEAST = 2.0 ** -126


def pack_rows(x):
    """(codes int8[rows, 128*ceil(cols/128)], scales float32[rows])."""
    rows, cols = x.shape
    codes = torch.zeros(rows, -(-cols // 128) * 128, dtype=torch.int8)
    amax = x.float().abs().amax(1)
    finite = torch.isfinite(amax)
    small = amax < 127 * LEAST
    most = torch.full_like(amax, 127.0)
    scale = torch.where(small, torch.full_like(amax, LEAST), amax / most)
    inverse = torch.where(small, torch.full_like(amax, 1 / LEAST), most / amax)
    ok = finite.unsqueeze(1)
    # x has 24 significant bits and the inverse too: the product in 64 bits is exact
    wide = torch.where(ok, x.double(), 0.0) * torch.where(finite, inverse, 0.0).double().unsqueeze(1)
    codes[:, :cols] = torch.round(wide).to(torch.int8)
    return codes, torch.where(finite, scale, torch.full_like(scale, float("nan")))


def pack_columns(x):
    return pack_rows(x.t().contiguous())


def spans(offsets, rows):
    """Rows of each expert, whatever the offsets hold."""
    held, most = [], 0
    for v in offsets:
        v = rows if v < 0 or v > rows else v  # read as unsigned
        most = max(most, v)
        held.append(most)
    return list(zip(held, held[1:]))


def product8(a, sa, w, sw):
    """The values in 64 bits, and the exact sums."""
    sums = a.double() @ w.double().t()
    return sums * (sa.double().unsqueeze(1) * sw.double()), sums
