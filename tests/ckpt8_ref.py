"""The 8-bit checkpoint operators from their definitions, in 64 bits on the
CPU, for the tests.  Shares no code with the package."""
from __future__ import annotations

import math

import torch

INT8, E4M3 = 1, 2
GELU, GELU_TANH, SILU = 1, 2, 3
LARGEST = {INT8: 127.0, E4M3: 448.0}
LOW = {INT8: -126, E4M3: -117}
HIGH = {INT8: 121, E4M3: 119}


def e4m3_values() -> torch.Tensor:
    """The number each of the 256 bytes stands for (the two NaN patterns as NaN)."""
    out = []
    for c in range(256):
        ex, fr = (c >> 3) & 15, c & 7
        v = fr * 2.0 ** -9 if ex == 0 else (8 + fr) * 2.0 ** (ex - 10)
        if c & 127 == 127:
            v = math.nan
        out.append(-v if c > 127 else v)
    return torch.tensor(out, dtype=torch.float64)


def code_values(codes: torch.Tensor, fmt: int) -> torch.Tensor:
    if fmt == INT8:
        return codes.view(torch.int8).double()
    return e4m3_values()[codes.long()]


def decode(codes, scales, fmt, cols):
    groups = -(-cols // 32)
    s = torch.where(scales[:, :groups] == 255, torch.tensor(math.nan, dtype=torch.float64),
                    torch.exp2(scales[:, :groups].double() - 127))
    return (code_values(codes, fmt) * s.repeat_interleave(32, 1))[:, :cols]


def _round_code(q: torch.Tensor, fmt: int) -> torch.Tensor:
    """Bytes of the nearest codes to q (|q| at most the largest), ties to even."""
    if fmt == INT8:
        return q.round().to(torch.int8).view(torch.uint8)
    a = q.abs()
    binade = torch.floor(torch.log2(torch.where(a == 0, 1.0, a))).clamp(-6, 8)
    binade = torch.where(a < torch.exp2(binade), binade - 1, binade)  # in case the logarithm rounded up
    binade = torch.where(a >= torch.exp2(binade + 1), binade + 1, binade).clamp(-6, 8)
    steps = (a / torch.exp2(binade - 3)).round()  # 8..16 of them in a normal binade, 0..8 below
    v = steps * torch.exp2(binade - 3)
    ex = torch.floor(torch.log2(torch.where(v == 0, 1.0, v))).clamp(-6, 8)
    normal = v >= 2.0 ** -6
    byte = torch.where(normal, (ex + 7) * 8 + v / torch.exp2(ex - 3) - 8, v * 512)
    return (byte + torch.where(torch.signbit(q), 128, 0)).to(torch.uint8)


def encode(x: torch.Tensor, fmt: int):
    """(codes, scales) of x[rows, cols] in float64, pads included."""
    rows, cols = x.shape
    groups = -(-cols // 32)
    v = torch.zeros(rows, groups * 32, dtype=torch.float64)
    v[:, :cols] = x
    v = v.view(rows, groups, 32)
    fine = torch.isfinite(v).all(2)
    v = torch.where(fine.unsqueeze(2), v, 0.0)
    amax = v.abs().amax(2)
    e = torch.full_like(amax, float(LOW[fmt]))
    for k in range(LOW[fmt], HIGH[fmt]):
        e = torch.where(amax > LARGEST[fmt] * 2.0 ** k, float(k + 1), e)
    q = (v / torch.exp2(e).unsqueeze(2)).clamp(-LARGEST[fmt], LARGEST[fmt])
    codes = torch.where(fine.unsqueeze(2), _round_code(q, fmt), 0).to(torch.uint8)
    scales = torch.zeros(rows, -(-groups // 4) * 4, dtype=torch.uint8)
    scales[:, :groups] = torch.where(fine, torch.where(amax > 0, e + 127, 0.0), 255.0).to(torch.uint8)
    return codes.view(rows, groups * 32), scales


def act(kind: int, x: torch.Tensor):
    """f(x) and f'(x) in 64 bits."""
    if kind == GELU:
        p = 0.5 * torch.special.erfc(-x / math.sqrt(2))
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x ** 3))
        return x * (1 + t) / 2, (1 + t) / 2 + x / 2 * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)
    p = 1 / (1 + torch.exp(-x))
    return x * p, p * (1 + x * (1 - p))


def norm(total: torch.Tensor, eps: float):
    """(rstd, normalised rows) of a sum in float64."""
    rstd = 1 / torch.sqrt((total * total).mean(1) + eps)
    return rstd, total * rstd.unsqueeze(1)


def norm_grad(dy, n, rstd, w, dtotal=None):
    g = dy * w
    dx = rstd.unsqueeze(1) * (g - n * (g * n).mean(1, keepdim=True))
    return dx if dtotal is None else dx + dtotal, (dy * n).sum(0)
