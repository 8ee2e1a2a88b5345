"""The block-scaled (MX) operators measured as a user calls them.

A matrix in an MX format holds its rows in blocks of 32 elements.  A block
has one power-of-two scale 2^e, stored as the byte e + 127, and 4- or 8-bit
elements: mxfp4 (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6), mxfp8 (E4M3) or mxint8
(an 8-bit integer, in 64ths).  e = floor(log2(largest magnitude)) - emax with
emax = 2, 8 and 0, at least -127; elements are x / 2^e rounded to nearest
even and saturated.  Rows are padded with zeros to whole groups of 256
elements: the elements sit at q[row, bytes] (two 4-bit elements to a byte,
the even one in the low half) and the scale of block b of row r at
s[b // 8, r, b % 8].

Operators:
  quantize  rounding a matrix (or its transpose) to MX and back
  product   act(X W^T + bias), X rounded to MX in the pass, W kept in mxfp4
  backward  op(dY) times a matrix kept in MX: dX = dY W, dW = dY^T X
  save      an activation's forward, with its input kept in 8 bits
  grad      the activation's backward from that input, with the bias gradient
"""
import math

import torch

own = False

BLOCK, GROUP = 32, 256
EMAX = {"mxfp4": 2, "mxfp8": 8, "mxint8": 0}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # a projection's weights (d_model 2048, FFN 5632) brought to 4 bits and read back, as when a model is loaded
        {"name": "weights to 4 bits", "op": "quantize", "rows": 5632, "cols": 2048, "type": "bf16", "format": "mxfp4", "trans": False, "pad": 0},
        # a ragged fp32 matrix stored the other way round, rows at an odd distance
        {"name": "ragged transposed to 8 bits", "op": "quantize", "rows": 4095, "cols": 1031, "type": "f32", "format": "mxfp8", "trans": True, "pad": 3},
        # one new token through a 4-bit projection: latency counts
        {"name": "one token", "op": "product", "M": 1, "N": 5632, "K": 2048, "type": "bf16", "format": "mxfp8", "act": "none", "bias": False, "pad": 0},
        # a few sequences' tokens, odd sizes, with bias and gelu
        {"name": "ragged batch", "op": "product", "M": 37, "N": 4097, "K": 1031, "type": "f16", "format": "mxfp8", "act": "gelu", "bias": True, "pad": 1},
        # a long prompt through a large layer, both sides in 4 bits
        {"name": "large prompt", "op": "product", "M": 8192, "N": 8192, "K": 8192, "type": "bf16", "format": "mxfp4", "act": "none", "bias": False, "pad": 0},
        # the gradient of a step's 512 tokens through a frozen 4-bit up projection
        {"name": "dX through 4-bit weights", "op": "backward", "M": 512, "N": 2048, "K": 5632, "type": "bf16", "out": "bf16", "format": "mxfp4", "trans": False, "pad": 0},
        # the rank-32 adapter's weight gradient from a saved 8-bit input
        {"name": "adapter dW", "op": "backward", "M": 32, "N": 2048, "K": 4096, "type": "f16", "out": "f32", "format": "mxfp8", "trans": True, "pad": 0},
        # a full layer's weight gradient over many tokens from a saved 8-bit input
        {"name": "layer dW", "op": "backward", "M": 5632, "N": 2048, "K": 16384, "type": "bf16", "out": "f32", "format": "mxint8", "trans": True, "pad": 0},
        # the hidden layer of one 512-token step, and of a large batch of tokens
        {"name": "save a step", "op": "save", "rows": 512, "cols": 5632, "type": "f16", "format": "mxint8", "act": "gelu", "pad": 0},
        {"name": "save a large batch", "op": "save", "rows": 32768, "cols": 5632, "type": "bf16", "format": "mxfp8", "act": "gelu", "pad": 0},
        # their backward passes; the first with an odd number of rows and columns
        {"name": "grad of a ragged step", "op": "grad", "rows": 511, "cols": 5631, "type": "f16", "format": "mxfp8", "act": "relu", "pad": 1},
        {"name": "grad of a large batch", "op": "grad", "rows": 32768, "cols": 5632, "type": "bf16", "format": "mxint8", "act": "gelu", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "backward", "backward", "save", "grad"])
    pad = rng.choice([0, 0, 1, 8])
    t16 = rng.choice(["f16", "bf16"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "cols": _log_int(rng, 1, 8192), "type": rng.choice(["f32", "f16", "bf16"]),
                "format": rng.choice(["mxfp4", "mxfp8", "mxint8"]), "trans": rng.random() < 0.5, "pad": pad}
    if op == "product":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 16, 8192), "K": _log_int(rng, 16, 8192), "type": t16,
                "format": rng.choice(["mxfp4", "mxfp8"]), "act": rng.choice(["none", "relu", "gelu"]), "bias": rng.random() < 0.5, "pad": pad}
    if op == "backward":
        trans = rng.random() < 0.5
        return {"op": op, "M": _log_int(rng, 1, 6144), "N": _log_int(rng, 16, 6144), "K": _log_int(rng, 16, 8192), "type": t16,
                "out": rng.choice([t16, "f32"]), "format": rng.choice(["mxfp8", "mxint8"]) if trans else "mxfp4", "trans": trans, "pad": pad}
    return {"op": op, "rows": _log_int(rng, 1, 32768), "cols": _log_int(rng, 32, 5632), "type": t16,
            "format": rng.choice(["mxfp8", "mxint8"]), "act": rng.choice(["relu", "gelu"]), "pad": pad}


# ---- MX matrices in elementary torch operations, 32 bits ---------------------------
def _row_bytes(fmt, cols):
    return -(-cols // GROUP) * (GROUP // 2 if fmt == "mxfp4" else GROUP)


def _scale(byte):
    """2^(byte - 127) in fp32, from its bits (byte 0: the subnormal 2^-127)."""
    b = byte.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _round_mx(x, fmt):
    """(element values, scale bytes) of an fp32 [rows, cols], padded to whole groups."""
    rows, cols = x.shape
    p = torch.zeros(rows, -(-cols // GROUP) * GROUP, dtype=torch.float32, device=x.device)
    p[:, :cols] = x
    b = p.view(rows, -1, BLOCK)
    _, e = torch.frexp(b.abs().amax(-1))
    byte = (e - 1 + 127 - EMAX[fmt]).clamp(min=0)
    byte = torch.where(b.abs().amax(-1) == 0, torch.zeros_like(byte), byte)
    v = b / _scale(byte)[..., None]
    if fmt == "mxint8":
        v = torch.round(v * 64).clamp(-127, 127) / 64
    elif fmt == "mxfp8":
        v = v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    else:
        # steps of 0.5 below 2, of 1 below 4, of 2 above; halves to even
        m = v.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        v = torch.copysign((torch.round(m / step) * step).clamp(max=6), v)
    return v.view(rows, -1), byte.to(torch.uint8)


def _pack(v, byte, fmt):
    """The stored form (q, s) of element values and scale bytes."""
    rows = v.shape[0]
    s = byte.view(rows, -1, GROUP // BLOCK).transpose(0, 1).contiguous()
    if fmt == "mxfp8":
        return v.to(torch.float8_e4m3fn).view(torch.uint8), s
    if fmt == "mxint8":
        return (v * 64).to(torch.int8).view(torch.uint8), s
    m = v.abs()
    code = (torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4))).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def _elements(q, fmt, dtype=torch.float32):
    if fmt == "mxfp8":
        return q.view(torch.float8_e4m3fn).to(dtype)
    if fmt == "mxint8":
        return q.view(torch.int8).to(dtype) / 64
    t = torch.tensor(FP4, dtype=dtype, device=q.device)
    return torch.stack([t[(q & 15).int()], t[(q >> 4).int()]], -1).flatten(1)


def _unpack(q, s, fmt, cols):
    """The fp32 values a stored MX matrix stands for."""
    v = _elements(q, fmt)
    sc = _scale(s.transpose(0, 1).reshape(q.shape[0], -1))
    return (v.view(q.shape[0], -1, BLOCK) * sc[..., None]).view(q.shape[0], -1)[:, :cols]


def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x * 0.70710678118654752)
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    return 0.5 * torch.erfc(-x * 0.70710678118654752) + x * torch.exp(-0.5 * x * x) * 0.3989422804014327


# ---- inputs ----------------------------------------------------------------------------
def _matrix(g, rows, cols, std, dtype, pad):
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").mul_(std).to(dtype)
    return x[:, :cols]


def _activations(g, rows, cols, dtype, pad):
    """Activations as a norm leaves them: unit variance, a few columns far larger."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols + pad, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return x.to(dtype)[:, :cols]


def _mx(x, fmt):
    v, byte = _round_mx(x.float(), fmt)
    q, s = _pack(v, byte, fmt)
    return {"format": fmt, "rows": x.shape[0], "cols": x.shape[1], "q": q, "s": s}


def _empty_mx(fmt, rows, cols):
    return {"format": fmt, "rows": rows, "cols": cols, "q": torch.empty(rows, _row_bytes(fmt, cols), dtype=torch.uint8, device="cuda"),
            "s": torch.empty(-(-cols // GROUP), rows, 8, dtype=torch.uint8, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, pad, fmt, dt = case["op"], case["pad"], case["format"], TYPES[case["type"]]
    st = {"case": case}
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        st["X"] = _matrix(g, *((c, r) if case["trans"] else (r, c)), 0.02, dt, pad)
        st["M"] = _empty_mx(fmt, r, c)
        st["Y"] = torch.empty(r, c, dtype=dt, device="cuda")
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        st["X"] = _activations(g, M, K, dt, pad)
        st["W"] = _mx(_matrix(g, N, K, 0.02, dt, 0), "mxfp4")
        st["bias"] = _matrix(g, 1, N, 0.5, dt, 0)[0] if case["bias"] else None
        st["A"] = _empty_mx(fmt, M, K)
        st["C"] = torch.empty(M, N, dtype=dt, device="cuda")
    elif op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        st["A"] = _matrix(g, *((K, M) if case["trans"] else (M, K)), 0.01, dt, pad)
        b = _activations(g, K, N, dt, 0) if case["trans"] else _matrix(g, K, N, 0.02, dt, 0)
        st["B"] = _mx(b, fmt)
        st["C"] = torch.empty(M, N, dtype=TYPES[case["out"]], device="cuda")
    else:
        r, c = case["rows"], case["cols"]
        z = _activations(g, r, c, dt, pad)
        if op == "save":
            st["Z"] = z
            st["H"] = torch.empty(r, c, dtype=dt, device="cuda")
            st["M"] = _empty_mx(fmt, r, c)
        else:
            st["M"] = _mx(z, fmt)
            st["dH"] = _matrix(g, r, c, 0.01, dt, pad)
            st["dZ"] = torch.empty(r, c, dtype=dt, device="cuda")
            st["dbias"] = torch.empty(c, dtype=torch.float32, device="cuda")
    return st


def _saved(m):
    """What a saved 8-bit matrix holds: its elements and its scales, as values."""
    q = m["q"][:, :m["cols"]]
    return {"q": q.view(torch.float8_e4m3fn if m["format"] == "mxfp8" else torch.int8), "s": m["s"].view(torch.float8_e8m0fnu)}


def _run_own(st):
    import dense_gemm_amd as dg

    c = st["case"]
    op = c["op"]
    mx = lambda m: dg.MxMatrix(m["format"], m["rows"], m["cols"], m["q"], m["s"])  # noqa: E731
    if op == "quantize":
        m = dg.quantize_mx(st["X"], trans=c["trans"], out=mx(st["M"]))
        return dg.dequantize_mx(m, out=st["Y"])
    if op == "product":
        a = dg.quantize_mx(st["X"], out=mx(st["A"]))
        return dg.gemm_mx(a, mx(st["W"]), C=st["C"], bias=st["bias"], activation=c["act"])
    if op == "backward":
        return dg.gemm_dq(st["A"], mx(st["B"]), C=st["C"], transA=c["trans"])
    if op == "save":
        h, _ = dg.act_checkpoint(st["Z"], c["act"], H=st["H"], out=mx(st["M"]))
        return {"h": h, **_saved(st["M"])}
    dz = dg.act_backward(st["dH"], mx(st["M"]), c["act"], dZ=st["dZ"], dbias=st["dbias"])
    return {"dz": dz, "dbias": st["dbias"]}


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op, fmt = c["op"], c["format"]
    if op == "quantize":
        x = st["X"].t() if c["trans"] else st["X"]
        q, s = _pack(*_round_mx(x.float(), fmt), fmt)
        return _unpack(q, s, fmt, c["cols"]).to(st["Y"].dtype)
    if op == "product":
        q, s = _pack(*_round_mx(st["X"].float(), fmt), fmt)
        w = st["W"]
        y = _unpack(q, s, fmt, c["K"]) @ _unpack(w["q"], w["s"], "mxfp4", c["K"]).t()
        if c["bias"]:
            y = y + st["bias"].float()
        return _act(y, c["act"]).to(st["C"].dtype)
    if op == "backward":
        a = st["A"].float()
        b = st["B"]
        return ((a.t() if c["trans"] else a) @ _unpack(b["q"], b["s"], fmt, c["N"])).to(st["C"].dtype)
    if op == "save":
        z = st["Z"].float()
        q, s = _pack(*_round_mx(z, fmt), fmt)
        return {"h": _act(z, c["act"]).to(st["H"].dtype), **_saved({"format": fmt, "cols": c["cols"], "q": q, "s": s})}
    m = st["M"]
    dz = st["dH"].float() * _act_slope(_unpack(m["q"], m["s"], fmt, c["cols"]), c["act"])
    return {"dz": dz.to(st["dZ"].dtype), "dbias": dz.sum(0)}


def work(case):
    op = case["op"]
    es = 4 if case["type"] == "f32" else 2
    mxb = lambda r, c, f: r * c * (0.5 if f == "mxfp4" else 1.0) + r * -(-c // BLOCK)  # noqa: E731
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * es + 2 * mxb(case["rows"], case["cols"], case["format"]), "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * 2 + 2 * mxb(M, K, case["format"]) + mxb(N, K, "mxfp4") + M * N * 2 + (N * 2 if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "backward":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * 2 + mxb(K, N, case["format"]) + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    r, c = case["rows"], case["cols"]
    return {"bytes": r * c * 2 * 2 + mxb(r, c, case["format"]) + (c * 4 if op == "grad" else 0), "flops": 20 * r * c}


# ---- the definition in 64 bits -------------------------------------------------------
def _pow2(e):
    """2^e in fp64 for whole e between -1022 and 1023, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(x, fmt):
    """What x (fp64 [rows, cols]) stands for after rounding: elements and scales by
    value, blocks of 32 along the columns, the last one short."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    full = torch.cat([x, x.new_zeros(rows, nb * 32 - cols)], 1).reshape(rows, nb, 32)
    top = full.abs().max(-1, keepdim=True).values
    lg = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
    lg = torch.where(_pow2(lg) > top, lg - 1, lg)
    lg = torch.where(_pow2(lg + 1) <= top, lg + 1, lg)
    scale = _pow2((lg - {"mxfp4": 2, "mxfp8": 8, "mxint8": 0}[fmt]).clamp(min=-127))
    u = full / scale
    if fmt == "mxint8":
        el = torch.round(u * 64).clamp(-127, 127)
        return el.reshape(rows, -1)[:, :cols], scale[..., 0], (el / 64 * scale).reshape(rows, -1)[:, :cols]
    # a float of `bits` fraction bits and least exponent `low`: a step of 2^(exponent - bits)
    bits, low, most = (1, 0, 6.0) if fmt == "mxfp4" else (3, -6, 448.0)
    ex = torch.frexp(u.abs().clamp(min=2.0 ** low))[1].to(torch.float64) - 1
    step = _pow2(ex - bits)
    el = (torch.round(u / step) * step).clamp(-most, most)
    return el.reshape(rows, -1)[:, :cols], scale[..., 0], (el * scale).reshape(rows, -1)[:, :cols]


def _exact_value(m):
    """A stored matrix's values: each code by its fields."""
    q, fmt = m["q"].to(torch.int64), m["format"]
    if fmt == "mxint8":
        el = torch.where(q > 127, q - 256, q).to(torch.float64) / 64
    else:
        if fmt == "mxfp4":
            q = torch.stack([q % 16, q // 16], 2).reshape(q.shape[0], -1)
            sign, ex, fr, bias, bits = q // 8, (q // 2) % 4, q % 2, 1, 1
        else:
            sign, ex, fr, bias, bits = q // 128, (q // 8) % 16, q % 8, 7, 3
        mant = torch.where(ex > 0, 2 ** bits + fr, fr).to(torch.float64)
        el = mant * _pow2(ex.clamp(min=1) - bias - bits) * (1 - 2 * sign)
    sc = _pow2(m["s"].permute(1, 0, 2).reshape(q.shape[0], -1).to(torch.int64) - 127)
    return (el * sc.repeat_interleave(32, 1))[:, :m["cols"]]


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case["format"]
    root2 = math.sqrt(2.0)
    if op == "quantize":
        x = st["X"].to(torch.float64)
        return _exact_round(x.transpose(0, 1) if case["trans"] else x, fmt)[2]
    if op == "product":
        a = _exact_round(st["X"].to(torch.float64), fmt)[2]
        y = torch.mm(a, _exact_value(st["W"]).transpose(0, 1).contiguous())
        if case["bias"]:
            y += st["bias"].to(torch.float64)
        if case["act"] == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif case["act"] == "gelu":
            y = y * torch.special.erfc(-y / root2) / 2
        return y
    if op == "backward":
        a = st["A"].to(torch.float64)
        a = a.transpose(0, 1).contiguous() if case["trans"] else a
        return torch.mm(a, _exact_value(st["B"]))
    if op == "save":
        z = st["Z"].to(torch.float64)
        el, sc, _ = _exact_round(z, fmt)
        h = torch.maximum(z, torch.zeros_like(z)) if case["act"] == "relu" else z * torch.special.erfc(-z / root2) / 2
        s = z.new_full((z.shape[0], -(-case["cols"] // 256) * 8), 2.0 ** -127)
        s[:, :sc.shape[1]] = sc
        return {"h": h, "q": el if fmt == "mxfp8" else None, "s": s.reshape(z.shape[0], -1, 8).permute(1, 0, 2)}
    z = _exact_value(st["M"])
    dh = st["dH"].to(torch.float64)
    if case["act"] == "relu":
        dz = torch.where(z > 0, dh, torch.zeros_like(dh))
    else:
        dz = dh * (torch.special.erfc(-z / root2) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return {"dz": dz, "dbias": dz.sum(0)}
