"""Measured cases of the 8-bit checkpoint operators, with their plain forms.

An activation that the backward pass needs is kept as 8-bit codes with one
power-of-two scale per 32 columns of a row, and the backward pass works from
the codes: ``pack`` and ``unpack``, the activation functions and their
gradients, the root-mean-square norm and its gradient, and the weight gradient
whose fp32 result is what the gradient codec compresses.

``run`` computes a case with elementary torch operations, or, where ``own`` is
set, with the package's kernels.  ``exact`` states the same results in 64 bits
on its own.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-6


# ----------------------------------------------------------------------------
# cases


def listed():
    return [
        # the activations of one short odd sequence through a checkpoint and back: call latency counts
        {"name": "pack_short_fp32", "op": "pack", "rows": 77, "cols": 1000, "dtype": "fp32", "format": "int8"},
        # a layer's input for a full batch of long sequences, kept for the backward pass and read again there
        {"name": "pack_batch_bf16", "op": "pack", "rows": 32768, "cols": 4096, "dtype": "bf16", "format": "e4m3"},
        # BERT-large's feed-forward activation, 8 sequences of 512: forward, checkpoint, gradient
        {"name": "gelu_step_bert", "op": "act", "rows": 4096, "cols": 4096, "dtype": "bf16", "format": "int8",
         "act": "gelu", "gated": False},
        # a gated activation of a small fp32 model, both halves in one fused projection of odd width
        {"name": "geglu_step_odd_fp32", "op": "act", "rows": 333, "cols": 1031, "dtype": "fp32", "format": "int8",
         "act": "gelu_tanh", "gated": True},
        # a gated activation's backward at a large batch, with the product rebuilt in 8 bits for the next weight gradient
        {"name": "silu_gated_grad", "op": "act_grad", "rows": 16384, "cols": 8192, "dtype": "bf16", "format": "e4m3",
         "act": "silu", "gated": True},
        # serving: one new token's norm with the residual, 8-bit output for the projection that follows
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "format": "e4m3",
         "weighted": True},
        # training: the norm before a block at a full batch, its normalised values kept in 8 bits
        {"name": "norm_batch_bf16", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16", "format": "int8",
         "weighted": False},
        # its backward from the 8-bit checkpoint
        {"name": "norm_grad_batch_bf16", "op": "norm_grad", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "format": "int8", "saved": "checkpoint"},
        # a norm's backward from the sum kept in full, odd sizes
        {"name": "norm_grad_odd_fp32", "op": "norm_grad", "rows": 1000, "cols": 1023, "dtype": "fp32",
         "format": "int8", "saved": "sum"},
        # BERT-large's feed-forward weight gradient, 8 sequences of 512
        {"name": "weight_grad_bert", "op": "weight_grad", "rows": 4096, "n": 4096, "cols": 1024, "dtype": "bf16",
         "format": "int8", "scaled": False},
        # a wide layer's weight gradient at a full batch, the norm's weight folded in
        {"name": "weight_grad_wide", "op": "weight_grad", "rows": 16384, "n": 8192, "cols": 8192, "dtype": "bf16",
         "format": "e4m3", "scaled": True},
        # an fp16 layer of odd sizes and a short batch
        {"name": "weight_grad_odd_fp16", "op": "weight_grad", "rows": 333, "n": 1000, "cols": 515, "dtype": "fp16",
         "format": "int8", "scaled": False},
    ]


def _size(rng, low, high):
    """A size between low and high, even over its logarithm; mostly odd in the last places."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.4 and v >= 256:
        v -= v % 128
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(("pack", "act", "act_grad", "norm", "norm_grad", "weight_grad"))
    case = {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 33, 8192),
            "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32")), "format": rng.choice(("int8", "e4m3"))}
    if op in ("act", "act_grad"):
        case["act"] = rng.choice(("gelu", "gelu_tanh", "silu"))
        case["gated"] = rng.random() < 0.5
    elif op == "norm":
        case["weighted"] = rng.random() < 0.3
    elif op == "norm_grad":
        case["saved"] = rng.choice(("checkpoint", "sum"))
    if op == "weight_grad":
        case["n"] = _size(rng, 33, 8192)
        case["scaled"] = rng.random() < 0.5
    else:
        case["rows"] = min(case["rows"], 2 ** 26 // case["cols"])
    return case


def work(case):
    r, c, s = case["rows"], case["cols"], SIZE[case["dtype"]]
    n, ck = r * c, r * c + r * -(-c // 32)  # values; bytes of a checkpoint
    op = case["op"]
    if op == "pack":  # x in, checkpoint out; checkpoint in, y out
        return {"bytes": 2 * (s * n + ck), "flops": 4 * n}
    if op == "act":  # forward: a (b) in, y and checkpoints out; gradient: dy and checkpoints in, da (db) out
        k = 2 if case["gated"] else 1
        return {"bytes": (k + 1) * s * n + k * ck + (k + 1) * s * n + k * ck, "flops": 40 * n}
    if op == "act_grad":  # dy and checkpoints in; da (db) and the product's checkpoint out, read once more
        k = 2 if case["gated"] else 1
        return {"bytes": (k + 1) * s * n + k * ck + 2 * ck + 2 * n, "flops": 40 * n}
    if op == "norm":  # x and residual in; sum, y, checkpoint and rstd out; the checkpoint read and decoded
        return {"bytes": 4 * s * n + ck + 4 * r + 4 * c + ck + 2 * n, "flops": 10 * n}
    if op == "norm_grad":  # dy, the sum's gradient and the saved values in; dx and dw out
        return {"bytes": 3 * s * n + (ck if case["saved"] == "checkpoint" else s * n) + 4 * r + 8 * c,
                "flops": 12 * n}
    m = case["n"]
    return {"bytes": s * r * m + ck + 4 * m * c, "flops": 2 * r * m * c}


# ----------------------------------------------------------------------------
# the plain form


_LIMIT = {"int8": (127 / 128, 7, -126, 121), "e4m3": (448 / 512, 9, -117, 119)}


def _encode(v, fmt):
    """(codes, scale bytes) of v[rows, cols]: groups of 32 columns, pads zero."""
    rows, cols = v.shape
    groups = -(-cols // 32)
    full = torch.zeros(rows, groups * 32, dtype=v.dtype, device=v.device)
    full[:, :cols] = v
    full = full.view(rows, groups, 32)
    amax = full.abs().amax(2)
    top, shift, low, high = _LIMIT[fmt]
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


def _decode(codes, scales, fmt, cols):
    """The values in 32 bits, exactly."""
    rows, padded = codes.shape
    v = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().view(rows, padded // 32, 32)
    factor = torch.ldexp(torch.ones((), device=codes.device), scales[:, :padded // 32].to(torch.int32) - 127)
    return (v * factor.unsqueeze(2)).view(rows, padded)[:, :cols]


def _act(act, a):
    if act == "gelu":
        return a * (0.5 + 0.5 * torch.erf(a * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return a * (0.5 + 0.5 * torch.tanh((2 / math.pi) ** 0.5 * (a + 0.044715 * a * a * a)))
    return a / (1 + torch.exp(-a))


def _act_slope(act, a):
    if act == "gelu":
        return (0.5 + 0.5 * torch.erf(a * 0.5 ** 0.5)) + a * torch.exp(-0.5 * a * a) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        t = torch.tanh((2 / math.pi) ** 0.5 * (a + 0.044715 * a * a * a))
        return 0.5 + 0.5 * t + 0.5 * a * (1 - t * t) * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * a * a)
    p = 1 / (1 + torch.exp(-a))
    return p * (1 + a * (1 - p))


def _plain_act_grad(act, dy, a, b):
    dy = dy.float()
    if b is None:
        return dy * _act_slope(act, a), None
    return dy * b * _act_slope(act, a), dy * _act(act, a)


# ----------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt, fmt = "cuda", DTYPES[case["dtype"]], case["format"]
    rows, cols, op = case["rows"], case["cols"], case["op"]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    # activations: some columns run a few times larger than the rest, as trained models' do
    spread = torch.exp(torch.randn(cols, generator=g, device=dev) * 0.5)
    st = {"case": case}
    if op == "pack":
        st["x"] = normal(rows, cols, scale=spread)
    elif op in ("act", "act_grad"):
        fused = normal(rows, 2 * cols if case["gated"] else cols, scale=2.0)  # one projection gives both halves
        a, b = fused[:, :cols], fused[:, cols:] if case["gated"] else None
        st["dy"] = normal(rows, cols, scale=1e-3)
        if op == "act":
            st["a"], st["b"] = a, b
        else:
            st["a"] = _encode(a.float(), fmt)
            st["b"] = _encode(b.float(), fmt) if b is not None else None
    elif op == "norm":
        st["x"], st["residual"] = normal(rows, cols), normal(rows, cols, scale=3 * spread)
        st["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=dev)).to(dt)
    elif op == "norm_grad":
        total = normal(rows, cols, scale=3 * spread)
        st["dy"], st["dtotal"] = normal(rows, cols, scale=1e-3), normal(rows, cols, scale=1e-3)
        st["weight"] = (1 + 0.2 * torch.randn(cols, generator=g, device=dev)).to(dt)
        rstd = (total.double().square().mean(1) + EPS).rsqrt()
        st["rstd"] = rstd.float()
        if case["saved"] == "checkpoint":
            st["saved"] = _encode((total.double() * rstd.unsqueeze(1)).float(), fmt)
        else:
            st["saved"] = total
    else:
        st["dy"] = normal(rows, case["n"], scale=1e-3)
        st["x"] = _encode(normal(rows, cols, scale=spread).float(), fmt)
        st["col_scale"] = 1 + 0.2 * torch.randn(cols, generator=g, device=dev) if case["scaled"] else None
    return st


# ----------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(st):
    case = st["case"]
    op, fmt, cols, dt = case["op"], case["format"], case["cols"], DTYPES[case["dtype"]]
    if op == "pack":
        return _decode(*_encode(st["x"].float(), fmt), fmt, cols).to(dt)
    if op == "act":
        a, b = st["a"].float(), st["b"].float() if case["gated"] else None
        y = _act(case["act"], a) if b is None else _act(case["act"], a) * b
        a = _decode(*_encode(a, fmt), fmt, cols)
        b = None if b is None else _decode(*_encode(b, fmt), fmt, cols)
        da, db = _plain_act_grad(case["act"], st["dy"], a, b)
        return {"y": y.to(dt), "da": da.to(dt), "db": None if db is None else db.to(dt)}
    if op == "act_grad":
        a = _decode(*st["a"], fmt, cols)
        b = _decode(*st["b"], fmt, cols) if case["gated"] else None
        da, db = _plain_act_grad(case["act"], st["dy"], a, b)
        y = _act(case["act"], a) if b is None else _act(case["act"], a) * b
        y8 = _decode(*_encode(y, fmt), fmt, cols)
        return {"da": da.to(dt), "db": None if db is None else db.to(dt), "y8": y8.to(torch.bfloat16)}
    if op == "norm":
        total = (st["x"].float() + st["residual"].float()).to(dt)
        t = total.double()  # the codes lie next to borders: 64 bits up to them
        rstd = (t.square().mean(1, keepdim=True) + EPS).rsqrt()
        n = t * rstd
        y = n.float() * st["weight"].float()
        coded = n * st["weight"].double() if case["weighted"] else n
        n8 = _decode(*_encode(coded, fmt), fmt, cols)
        return {"total": total, "y": y.to(dt), "n8": n8.to(torch.bfloat16), "rstd": rstd.float().flatten()}
    if op == "norm_grad":
        rstd = st["rstd"].unsqueeze(1)
        if case["saved"] == "checkpoint":
            n = _decode(*st["saved"], fmt, cols)
        else:
            n = st["saved"].float() * rstd
        dy = st["dy"].float()
        gw = dy * st["weight"].float()
        dx = st["dtotal"].float() + rstd * (gw - n * (gw * n).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dw": (dy * n).sum(0)}
    x = _decode(*st["x"], fmt, cols)
    dw = st["dy"].float().t() @ x
    return dw * st["col_scale"] if case["scaled"] else dw


def _run_own(st):
    from gradient_compression_distributed_lc_amd import tlc
    case = st["case"]
    op, cols = case["op"], case["cols"]
    fmt = tlc.CKPT8_INT8 if case["format"] == "int8" else tlc.CKPT8_E4M3

    def kept(c):
        return tlc.Checkpoint8(c[0], c[1], cols, fmt)

    if op == "pack":
        return tlc.ckpt8_unpack(tlc.ckpt8_pack(st["x"], fmt), st["x"].dtype)
    if op in ("act", "act_grad"):
        act = {"gelu": tlc.ACT_GELU, "gelu_tanh": tlc.ACT_GELU_TANH, "silu": tlc.ACT_SILU}[case["act"]]
    if op == "act":
        y, a8, b8 = tlc.ckpt8_act(st["a"], act, fmt, b=st["b"])
        da, db, _ = tlc.ckpt8_act_grad(st["dy"], act, a8, b8)
        return {"y": y, "da": da, "db": db}
    if op == "act_grad":
        da, db, y8 = tlc.ckpt8_act_grad(st["dy"], act, kept(st["a"]), kept(st["b"]) if case["gated"] else None,
                                        want_y=True)
        return {"da": da, "db": db, "y8": tlc.ckpt8_unpack(y8, torch.bfloat16)}
    if op == "norm":
        total, y, n8, rstd = tlc.ckpt8_norm(st["x"], st["weight"], EPS, fmt, residual=st["residual"],
                                            weighted=case["weighted"])
        return {"total": total, "y": y, "n8": tlc.ckpt8_unpack(n8, torch.bfloat16), "rstd": rstd}
    if op == "norm_grad":
        saved = kept(st["saved"]) if case["saved"] == "checkpoint" else st["saved"]
        dx, dw = tlc.ckpt8_norm_grad(st["dy"], saved, st["rstd"], st["weight"], dtotal=st["dtotal"])
        return {"dx": dx, "dw": dw}
    return tlc.ckpt8_weight_grad(st["dy"], kept(st["x"]), col_scale=st["col_scale"])


# ----------------------------------------------------------------------------
# the definition in 64 bits


def _exact_values(codes, scales, fmt, cols):
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


def _exact_quantised(v, fmt):
    """What a checkpoint of v stands for: each value at the nearest step of its group."""
    rows, cols = v.shape
    pad = -cols % 32
    w = torch.nn.functional.pad(v, (0, pad)).view(rows, -1, 32)
    largest, least, most = (127.0, -126, 121) if fmt == "int8" else (448.0, -117, 119)
    e = torch.full(w.shape[:2], float(least), dtype=torch.float64, device=v.device)
    amax = w.abs().amax(2)
    guess = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0) / largest))
    for step in (guess - 1, guess, guess + 1, guess + 2):  # the least of these that holds the largest value
        e = torch.where((amax > 0) & (amax > largest * torch.exp2(e)), step.clamp(least, most), e)
    scale = torch.exp2(e).unsqueeze(2)
    q = w / scale
    if fmt == "int8":
        q = q.round()
    else:  # steps of 2^-3 of the value's binade, and of 2^-9 below 2^-6
        binade = torch.floor(torch.log2(torch.where(q == 0, 1.0, q.abs()))).clamp(-6, 8)
        unit = torch.exp2(binade - 3)
        q = (q / unit).round() * unit
    return (q.clamp(-largest, largest) * scale).view(rows, -1)[:, :cols]


def _exact_act(act, a):
    """f(a) and f'(a)."""
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-a / math.sqrt(2))
        return a * phi, phi + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        p = torch.sigmoid(2 * k * (a + 0.044715 * a ** 3))
        return a * p, p + a * p * (1 - p) * 2 * k * (1 + 0.134145 * a ** 2)
    p = torch.sigmoid(a)
    return a * p, p + a * p * (1 - p)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt, cols = case["op"], case["format"], case["cols"]
    if op == "pack":
        return _exact_quantised(st["x"].double(), fmt)
    if op in ("act", "act_grad"):
        gated, dy = case["gated"], st["dy"].double()
        out = {}
        if op == "act":
            a, b = st["a"].double(), st["b"].double() if gated else 1.0
            out["y"] = _exact_act(case["act"], a)[0] * b
            a, b = _exact_quantised(a, fmt), _exact_quantised(b, fmt) if gated else 1.0
        else:
            a = _exact_values(*st["a"], fmt, cols)
            b = _exact_values(*st["b"], fmt, cols) if gated else 1.0
        f, slope = _exact_act(case["act"], a)
        out["da"], out["db"] = dy * slope * b, dy * f if gated else None
        if op == "act_grad":
            out["y8"] = _exact_quantised(f * b, fmt)
        return out
    if op == "norm":
        # the sum is rounded to its type before the norm reads it; the rounding of an exact sum
        total = (st["x"].double() + st["residual"].double()).to(DTYPES[case["dtype"]]).double()
        rstd = 1 / torch.sqrt((total * total).sum(1) / cols + EPS)
        n = total * rstd.unsqueeze(1)
        y = n * st["weight"].double()
        return {"total": total, "y": y, "n8": _exact_quantised(y if case["weighted"] else n, fmt), "rstd": rstd}
    if op == "norm_grad":
        rstd = st["rstd"].double().unsqueeze(1)
        if case["saved"] == "checkpoint":
            n = _exact_values(*st["saved"], fmt, cols)
        else:
            n = st["saved"].double() * rstd
        dy, w = st["dy"].double(), st["weight"].double()
        dot = ((dy * w) * n).sum(1, keepdim=True) / cols
        return {"dx": st["dtotal"].double() + rstd * (dy * w - n * dot), "dw": (dy * n).sum(0)}
    x = _exact_values(*st["x"], fmt, cols)
    dw = torch.matmul(st["dy"].double().t(), x)
    return dw * st["col_scale"].double() if case["scaled"] else dw
