"""Measured cases of the 8-bit integer products and the products grouped by
expert, with their plain forms.

A matrix kept in 8-bit integers has one fp32 scale per row: per token where it
holds activations, per output channel where it holds a weight.  The products of
a layer (forward, input gradient, weight gradient) are each one such product,
from the rows or the columns of its operands.  Products grouped by expert take
rows that lie expert by expert, as many for each as the offsets say, and each
expert's own weight.

``run`` computes a case with elementary torch operations, or, where ``own`` is
set, with the package's kernels.  ``exact`` states the same results in 64 bits
on its own.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new token's activations on their way to an 8-bit product: call latency counts
        {"name": "rows8_token", "op": "rows8", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # the input of a wide layer for a full batch
        {"name": "rows8_batch_bf16", "op": "rows8", "rows": 16384, "cols": 8192, "dtype": "bf16"},
        # an activation of a small fp32 model, transposed for its weight gradient, odd sizes
        {"name": "columns8_odd_fp32", "op": "columns8", "rows": 1000, "cols": 1031, "dtype": "fp32"},
        # the output gradient of a layer for a full batch, transposed for its weight gradient
        {"name": "columns8_batch_bf16", "op": "columns8", "rows": 16384, "cols": 4096, "dtype": "bf16"},
        # serving: one token through a layer whose weight is kept in 8 bits
        {"name": "linear8_token", "op": "linear8", "rows": 1, "cols": 4096, "n": 8192, "dtype": "bf16", "experts": 0},
        # a wide layer's forward pass for a full batch
        {"name": "linear8_wide", "op": "linear8", "rows": 16384, "cols": 8192, "n": 8192, "dtype": "bf16",
         "experts": 0},
        # BERT-large's feed-forward layer, 8 sequences of 512: output, input gradient and weight gradient, all in 8 bits
        {"name": "step8_bert", "op": "step8", "rows": 4096, "cols": 1024, "n": 4096, "dtype": "bf16"},
        # a layer of many small experts in 8 bits, a ragged share of the rows each
        {"name": "linear8_experts", "op": "linear8", "rows": 4096, "cols": 2048, "n": 1024, "dtype": "fp16",
         "experts": 32},
        # serving: a few tokens spread over experts
        {"name": "expert_tokens", "op": "expert", "rows": 8, "cols": 4096, "n": 2048, "dtype": "bf16", "experts": 16},
        # training: a layer of experts for a full batch, forward and input gradient
        {"name": "expert_batch_bf16", "op": "expert_grad", "rows": 16384, "cols": 4096, "n": 4096, "dtype": "bf16",
         "experts": 8},
        # its weight gradients from the 8-bit checkpoint of its input
        {"name": "expert_weight_grad_batch", "op": "expert_weight_grad", "rows": 16384, "cols": 4096, "n": 4096,
         "dtype": "bf16", "experts": 8, "format": "e4m3"},
        # a small fp32 layer of odd sizes: output, input gradient and weight gradients
        {"name": "expert_step_odd_fp32", "op": "expert_step", "rows": 777, "cols": 515, "n": 1000, "dtype": "fp32",
         "experts": 5, "format": "int8"},
    ]


def _size(rng, low, high):
    """A size between low and high, even over its logarithm; mostly odd in the last places."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.4 and v >= 256:
        v -= v % 128
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(("rows8", "columns8", "linear8", "linear8", "step8", "expert", "expert_grad",
                     "expert_weight_grad", "expert_step"))
    case = {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 33, 8192),
            "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if op in ("rows8", "columns8"):
        return case
    case["n"] = _size(rng, 33, 8192)
    if op == "linear8":
        case["experts"] = rng.choice((0, _size(rng, 1, 64)))
    elif op != "step8":
        case["experts"] = _size(rng, 1, 64)
    if op in ("expert_weight_grad", "expert_step"):
        case["format"] = rng.choice(("int8", "e4m3"))
    weight = max(case.get("experts", 0), 1) * case["cols"]
    case["n"] = max(33, min(case["n"], 2 ** 27 // weight))
    most = {"linear8": 2 ** 40, "step8": 2 ** 37, "expert_step": 2 ** 36}.get(op, 2 ** 38)
    case["rows"] = max(1, min(case["rows"], most // (case["n"] * case["cols"])))
    return case


def work(case):
    r, c, s, op = case["rows"], case["cols"], SIZE[case["dtype"]], case["op"]
    if op in ("rows8", "columns8"):  # values in, codes and scales out
        return {"bytes": s * r * c + r * c + 4 * (r if op == "rows8" else c), "flops": 3 * r * c}
    n = case["n"]
    if op == "step8":  # x, w and dy in; y, dx and dw out; three products
        return {"bytes": s * (r * c + n * c + r * n) + s * (r * n + r * c) + 4 * n * c, "flops": 6 * r * n * c}
    used = min(max(case["experts"], 1), r)  # experts that can have rows
    if op == "linear8":  # x and the weight's codes and scales in, y out
        return {"bytes": s * r * (c + n) + used * n * (c + 4), "flops": 2 * r * n * c}
    w, x8, dw = s * used * n * c, r * c + r * -(-c // 32), 4 * case["experts"] * n * c
    if op == "expert":
        return {"bytes": s * r * (c + n) + w, "flops": 2 * r * n * c}
    if op == "expert_grad":  # x, dy and w in; y and dx out
        return {"bytes": 2 * s * r * (c + n) + w, "flops": 4 * r * n * c}
    if op == "expert_weight_grad":
        return {"bytes": s * r * n + x8 + dw, "flops": 2 * r * n * c}
    return {"bytes": 2 * s * r * (c + n) + w + x8 + dw, "flops": 6 * r * n * c}


# ----------------------------------------------------------------------------
# the plain form

_LEAST = 2.0 ** -126  # the least scale


def _quantise(x):
    """(codes, scales) of the rows of x: a scale of a 127th of the row's largest magnitude."""
    amax = x.abs().amax(1).float()
    most = torch.full_like(amax, 127.0)
    small = amax < 127 * _LEAST
    scale = torch.where(small, torch.full_like(amax, _LEAST), amax / most)
    inverse = torch.where(small, torch.full_like(amax, 1 / _LEAST), most / amax)
    # next to a border between two codes: 64 bits
    codes = (x.double() * inverse.double().unsqueeze(1)).round().to(torch.int8)
    return codes, scale


def _product8(a, w, dt):
    """a and w: (codes, scales)."""
    sums = a[0].float() @ w[0].float().t()
    return (sums * a[1].unsqueeze(1) * w[1]).to(dt)


def _values(codes, scales):
    return codes.float() * scales.unsqueeze(1)


def _rows_of(counts):
    at = 0
    for e, k in enumerate(counts):
        yield e, slice(at, at + k)
        at += k


def _checkpoint_values(codes, scales, fmt, cols):
    """The values of an 8-bit checkpoint in 32 bits, exactly."""
    rows, padded = codes.shape
    v = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().view(rows, padded // 32, 32)
    factor = torch.ldexp(torch.ones((), device=codes.device), scales[:, :padded // 32].to(torch.int32) - 127)
    return (v * factor.unsqueeze(2)).view(rows, padded)[:, :cols]


def _checkpoint(v, fmt):
    """(codes, scale bytes) of v[rows, cols]: groups of 32 columns, a power of two each, pads zero."""
    rows, cols = v.shape
    groups = -(-cols // 32)
    top, shift, low, high = {"int8": (127 / 128, 7, -126, 121), "e4m3": (448 / 512, 9, -117, 119)}[fmt]
    full = torch.nn.functional.pad(v, (0, groups * 32 - cols)).view(rows, groups, 32)
    amax = full.abs().amax(2)
    m, e = torch.frexp(amax)
    e = (e - shift + (m > top)).clamp(low, high)
    scaled = torch.ldexp(full, -e.unsqueeze(2))
    if fmt == "int8":
        codes = torch.round(scaled).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    else:
        codes = scaled.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.zeros(rows, -(-groups // 4) * 4, dtype=torch.uint8, device=v.device)
    scales[:, :groups] = torch.where(amax > 0, e + 127, torch.zeros_like(e)).to(torch.uint8)
    return codes.reshape(rows, groups * 32), scales


# ----------------------------------------------------------------------------
# inputs


def _counts(rows, experts, seed):
    """Rows of each expert: uneven, as a router's choices are, some of them often none."""
    rng = random.Random(seed)
    weights = [rng.expovariate(1.0) for _ in range(experts)]
    counts = [int(rows * w / sum(weights)) for w in weights]
    for _ in range(rows - sum(counts)):
        counts[rng.randrange(experts)] += 1
    return counts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt, op = "cuda", DTYPES[case["dtype"]], case["op"]
    rows, cols, n, experts = case["rows"], case["cols"], case.get("n"), case.get("experts", 0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    # activations: some columns run a few times larger than the rest, as trained models' do
    spread = torch.exp(torch.randn(cols, generator=g, device=dev) * 0.5)
    st = {"case": case, "x": normal(rows, cols, scale=spread)}
    if op in ("rows8", "columns8"):
        return st
    if experts:
        st["counts"] = _counts(rows, experts, seed)
        ends = [0]
        for k in st["counts"]:
            ends.append(ends[-1] + k)
        st["offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
    if op == "linear8":  # the weight is kept in 8 bits, rows 128 bytes or a multiple apart
        many = max(experts, 1)
        st["w"] = torch.zeros(many * n, -(-cols // 128) * 128, dtype=torch.int8, device=dev)
        st["w_scales"] = torch.empty(many * n, dtype=torch.float32, device=dev)
        for e in range(many):
            part = slice(e * n, (e + 1) * n)
            st["w"][part, :cols], st["w_scales"][part] = _quantise(normal(n, cols, scale=cols ** -0.5))
        return st
    if op == "step8":
        st["w"] = normal(n, cols, scale=cols ** -0.5)
    elif op != "expert_weight_grad":
        st["w"] = torch.empty(experts, n, cols, dtype=dt, device=dev)
        for e in range(experts):
            st["w"][e] = normal(n, cols, scale=cols ** -0.5)
    if op != "expert":
        st["dy"] = normal(rows, n, scale=1e-3)
    if "format" in case:
        st["x8"] = _checkpoint(st["x"].float(), case["format"])
    return st


# ----------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(st):
    case = st["case"]
    op, cols, dt = case["op"], case["cols"], DTYPES[case["dtype"]]
    if op == "rows8":
        return _values(*_quantise(st["x"]))
    if op == "columns8":
        return _values(*_quantise(st["x"].t()))
    if op == "linear8":
        x, w = _quantise(st["x"]), (st["w"][:, :cols], st["w_scales"])
        if not case["experts"]:
            return _product8(x, w, dt)
        n = case["n"]
        y = torch.empty(case["rows"], n, dtype=dt, device=st["x"].device)
        for e, rows in _rows_of(st["counts"]):
            part = slice(e * n, (e + 1) * n)
            y[rows] = _product8((x[0][rows], x[1][rows]), (w[0][part], w[1][part]), dt)
        return y
    if op == "step8":
        x, w, dy = st["x"], st["w"], st["dy"]
        return {"y": _product8(_quantise(x), _quantise(w), dt),
                "dx": _product8(_quantise(dy), _quantise(w.t()), dt),
                "dw": _product8(_quantise(dy.t()), _quantise(x.t()), torch.float32)}
    out = {}
    if op != "expert_weight_grad":
        out["y"] = torch.empty(case["rows"], case["n"], dtype=dt, device=st["x"].device)
        for e, rows in _rows_of(st["counts"]):
            out["y"][rows] = (st["x"][rows].float() @ st["w"][e].float().t()).to(dt)
    if op in ("expert_grad", "expert_step"):
        out["dx"] = torch.empty(case["rows"], cols, dtype=dt, device=st["x"].device)
        for e, rows in _rows_of(st["counts"]):
            out["dx"][rows] = (st["dy"][rows].float() @ st["w"][e].float()).to(dt)
    if op in ("expert_weight_grad", "expert_step"):
        x = _checkpoint_values(*st["x8"], case["format"], cols)
        out["dw"] = torch.empty(case["experts"], case["n"], cols, dtype=torch.float32, device=x.device)
        for e, rows in _rows_of(st["counts"]):
            out["dw"][e] = st["dy"][rows].float().t() @ x[rows]
    return out


def _run_own(st):
    from gradient_compression_distributed_lc_amd import tlc
    case = st["case"]
    op, cols, dt = case["op"], case["cols"], DTYPES[case["dtype"]]
    if op == "rows8":
        c = tlc.q8_pack_rows(st["x"])
        return _values(c.codes[:, :c.cols], c.scales)
    if op == "columns8":
        c = tlc.q8_pack_columns(st["x"])
        return _values(c.codes[:, :c.cols], c.scales)
    if op == "linear8":
        w = tlc.Rows8(st["w"], st["w_scales"], cols)
        return tlc.q8_product(tlc.q8_pack_rows(st["x"]), w, dt, offsets=st.get("offsets"))
    if op == "step8":
        x, w, dy = st["x"], st["w"], st["dy"]
        return {"y": tlc.q8_product(tlc.q8_pack_rows(x), tlc.q8_pack_rows(w), dt),
                "dx": tlc.q8_product(tlc.q8_pack_rows(dy), tlc.q8_pack_columns(w), dt),
                "dw": tlc.q8_product(tlc.q8_pack_columns(dy), tlc.q8_pack_columns(x), torch.float32)}
    out = {}
    if op != "expert_weight_grad":
        out["y"] = tlc.expert_product(st["x"], st["w"], st["offsets"])
    if op in ("expert_grad", "expert_step"):
        out["dx"] = tlc.expert_input_grad(st["dy"], st["w"], st["offsets"])
    if op in ("expert_weight_grad", "expert_step"):
        fmt = tlc.CKPT8_INT8 if case["format"] == "int8" else tlc.CKPT8_E4M3
        out["dw"] = tlc.expert_weight_grad(st["dy"], tlc.Checkpoint8(*st["x8"], cols, fmt), st["offsets"])
    return out


# ----------------------------------------------------------------------------
# the definition in 64 bits


def _exact_rows(x):
    """(integers, scales) of the rows of x in 64 bits.  The scale and its inverse are fp32 numbers by definition."""
    wide = x.double()
    amax = wide.abs().max(dim=1).values
    scale = (amax / 127).float().double().clamp(min=2.0 ** -126)
    inverse = torch.where(amax < 127 * 2.0 ** -126, 2.0 ** 126, (127 / amax).float().double())
    t = wide * inverse[:, None]
    low = torch.floor(t)
    part = t - low
    odd = torch.remainder(low, 2) == 1
    return low + ((part > 0.5) | ((part == 0.5) & odd)).double(), scale


def _exact_product8(a, w):
    return torch.matmul(a[0], w[0].t()) * (a[1][:, None] * w[1][None, :])


def _exact_checkpoint(codes, scales, fmt, cols):
    """Values of a checkpoint, from the bits of its bytes."""
    u = codes.to(torch.int64)
    if fmt == "int8":
        v = torch.where(u > 127, u - 256, u).double()
    else:  # sign, 4 exponent bits of bias 7, 3 fraction bits
        ex, fr = (u >> 3) & 15, (u & 7).double()
        v = torch.where(ex == 0, fr * 2.0 ** -9, (8 + fr) * torch.exp2(ex.double() - 10))
        v = torch.where(u > 127, -v, v)
    per_column = scales.to(torch.int64).repeat_interleave(32, 1)[:, :codes.shape[1]]
    return (v * torch.exp2(per_column.double() - 127))[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op, cols, n = case["op"], case["cols"], case.get("n")
    if op in ("rows8", "columns8"):
        q, s = _exact_rows(st["x"] if op == "rows8" else st["x"].t())
        return q * s[:, None]
    if op == "step8":
        x, w, dy = st["x"], st["w"], st["dy"]
        return {"y": _exact_product8(_exact_rows(x), _exact_rows(w)),
                "dx": _exact_product8(_exact_rows(dy), _exact_rows(w.t())),
                "dw": _exact_product8(_exact_rows(dy.t()), _exact_rows(x.t()))}
    bounds = st["offsets"].tolist() if "offsets" in st else [0, case["rows"]]
    pairs = list(zip(bounds, bounds[1:]))
    if op == "linear8":
        q, s = _exact_rows(st["x"])
        w, sw = st["w"][:, :cols], st["w_scales"].double()
        return torch.cat([_exact_product8((q[a:b], s[a:b]), (w[e * n:(e + 1) * n].double(), sw[e * n:(e + 1) * n]))
                          for e, (a, b) in enumerate(pairs)])
    out = {}
    if op != "expert_weight_grad":
        out["y"] = torch.cat([torch.matmul(st["x"][a:b].double(), st["w"][e].double().t())
                              for e, (a, b) in enumerate(pairs)])
    if op in ("expert_grad", "expert_step"):
        out["dx"] = torch.cat([torch.matmul(st["dy"][a:b].double(), st["w"][e].double())
                               for e, (a, b) in enumerate(pairs)])
    if op in ("expert_weight_grad", "expert_step"):
        x = _exact_checkpoint(*st["x8"], case["format"], cols)
        out["dw"] = torch.stack([torch.matmul(st["dy"][a:b].double().t(), x[a:b]) for a, b in pairs])
    return out
