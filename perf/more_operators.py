"""A layer's products with their whole epilogue, dense and grouped by expert,
measured as a user calls them.

Rows of X are tokens.  W is one matrix, or one per expert; then the tokens lie
sorted by expert, expert g's rows being offsets[g] .. offsets[g + 1] - 1 of X and
of every other matrix of rows (a count may be zero).

Operators:
  fused     Z = X W + bias,  Y = act(Z) + R, with Z kept or not (one W)
  grouped   the same with a W and a bias for each expert
  act_grad  dH = dY W + R,  dZ = dH * act'(Z): what a layer's backward pass hands
            to the layer below it (one W, or one for each expert)
  dw        dW = dY^T X and dbias = the column sums of dY, over all rows or for
            each expert over its own rows
W is stored [K, N], or [N, K] where "trans" is true.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token through an up projection with gelu: latency, and one pass over the weights
        {"name": "one token", "op": "fused", "groups": 0, "M": 1, "N": 5632, "K": 2048, "type": "bf16", "out": "bf16", "trans": True, "act": "gelu", "bias": True, "res": False, "keep": False, "pad": 0},
        # a decoding batch through the down projection, onto the residual stream
        {"name": "decoding batch", "op": "fused", "groups": 0, "M": 24, "N": 2048, "K": 5632, "type": "f16", "out": "f16", "trans": True, "act": "none", "bias": True, "res": True, "keep": False, "pad": 0},
        # full precision at odd sizes, rows at an odd distance, everything at once
        {"name": "ragged fp32", "op": "fused", "groups": 0, "M": 511, "N": 1031, "K": 2047, "type": "f32", "out": "f32", "trans": False, "act": "gelu", "bias": True, "res": True, "keep": True, "pad": 3},
        # the up projection of a large training batch, its input to gelu kept
        {"name": "large batch", "op": "fused", "groups": 0, "M": 16384, "N": 5632, "K": 2048, "type": "bf16", "out": "bf16", "trans": True, "act": "gelu", "bias": True, "res": False, "keep": True, "pad": 0},
        # decoding with experts: a few tokens to each, some to none
        {"name": "experts, decoding", "op": "grouped", "groups": 16, "M": 64, "N": 5632, "K": 2048, "type": "bf16", "out": "bf16", "trans": True, "act": "gelu", "bias": False, "res": False, "keep": False, "pad": 0},
        # many small experts over a ragged batch, weights stored [K, N], odd row strides
        {"name": "many small experts", "op": "grouped", "groups": 64, "M": 4095, "N": 1032, "K": 2040, "type": "f16", "out": "f32", "trans": False, "act": "relu", "bias": True, "res": True, "keep": False, "pad": 1},
        # a training batch routed to 8 experts
        {"name": "experts, large batch", "op": "grouped", "groups": 8, "M": 16384, "N": 5632, "K": 2048, "type": "bf16", "out": "bf16", "trans": True, "act": "gelu", "bias": True, "res": False, "keep": True, "pad": 0},
        # backward of a 512-token step through the down projection and gelu
        {"name": "dZ of a step", "op": "act_grad", "groups": 0, "M": 512, "N": 5632, "K": 2048, "type": "f16", "out": "f16", "trans": False, "act": "gelu", "res": False, "keep": False, "pad": 0},
        # the same for a large batch and its 8 experts
        {"name": "dZ of experts", "op": "act_grad", "groups": 8, "M": 16384, "N": 5632, "K": 2048, "type": "bf16", "out": "bf16", "trans": False, "act": "gelu", "res": False, "keep": False, "pad": 0},
        # a rank-32 adapter's weight gradient with its bias's
        {"name": "adapter dW", "op": "dw", "groups": 0, "rows": 4096, "M": 2048, "N": 32, "type": "f16", "out": "f32", "bias": True, "pad": 0},
        # weight gradients of many small experts, odd sizes
        {"name": "dW of many experts", "op": "dw", "groups": 32, "rows": 4095, "M": 1031, "N": 517, "type": "bf16", "out": "bf16", "bias": False, "pad": 1},
        # weight gradients of a large batch's 8 experts, kept in fp32
        {"name": "dW of experts", "op": "dw", "groups": 8, "rows": 16384, "M": 5632, "N": 2048, "type": "bf16", "out": "f32", "bias": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["fused", "fused", "grouped", "grouped", "act_grad", "dw"])
    typ = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    out = rng.choice([typ, "f32"])
    pad = rng.choice([0, 0, 1, 8])
    act = rng.choice(["none", "relu", "gelu"])
    groups = 0 if op == "fused" or (op != "grouped" and rng.random() < 0.5) else _log_int(rng, 1, 64)
    rows, n, k = _log_int(rng, 1, 16384), _log_int(rng, 16, 5632), _log_int(rng, 16, 5632)
    # no more work than the largest listed case (fp32 matrix cores: a sixteenth of the rate)
    most = 16384 * 5632 * 2048 // (16 if typ == "f32" else 1)
    while rows * n * k > most:
        rows = (rows + 1) // 2
    if op == "dw":
        return {"op": op, "groups": groups, "rows": rows, "M": n, "N": k, "type": typ, "out": out, "bias": rng.random() < 0.5, "pad": pad}
    case = {"op": op, "groups": groups, "M": rows, "N": n, "K": k, "type": typ, "out": out, "trans": rng.random() < 0.5, "act": act,
            "res": rng.random() < 0.4, "keep": rng.random() < 0.4, "pad": pad}
    if op == "act_grad":
        case["act"] = "relu" if act == "none" else act
    else:
        case["bias"] = rng.random() < 0.7
    return case


# ---- inputs -----------------------------------------------------------------------
def _matrix(g, rows, cols, std, dtype, pad):
    """[rows, cols] normal values, rows `pad` elements further apart than they are long."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").mul_(std).to(dtype)
    return x[:, :cols]


def _activations(g, rows, cols, dtype, pad):
    """Activations as a norm leaves them: unit variance, a few columns far larger."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols + pad, generator=g, device="cuda") < 0.01, 4.0, 1.0)
    return x.to(dtype)[:, :cols]


def _counts(seed, groups, rows):
    """Tokens per expert as a router leaves them: uneven, a few experts with none."""
    g = torch.Generator()
    g.manual_seed(seed + 1)
    w = torch.softmax(0.5 * torch.randn(groups, generator=g), 0)
    if groups > 4:
        w[torch.randperm(groups, generator=g)[:groups // 8]] = 0
    n = torch.multinomial(w, rows, replacement=True, generator=g)
    return torch.bincount(n, minlength=groups).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, pad, G, dt, odt = case["op"], case["pad"], case["groups"], TYPES[case["type"]], TYPES[case["out"]]
    rows = case["rows"] if op == "dw" else case["M"]
    st = {"case": case, "sizes": _counts(seed, G, rows) if G else [rows]}
    if G:
        st["offsets"] = torch.tensor([0] + st["sizes"], dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    if op == "dw":
        M, N = case["M"], case["N"]
        st["dY"] = _matrix(g, rows, M, 0.01, dt, pad)
        st["X"] = _activations(g, rows, N, dt, pad)
        st["dW"] = torch.empty((G, M, N) if G else (M, N), dtype=odt, device="cuda")
        st["dbias"] = torch.empty((G, M) if G else (M,), dtype=torch.float32, device="cuda") if case["bias"] else None
        return st
    M, N, K = case["M"], case["N"], case["K"]
    wr, wc = (N, K) if case["trans"] else (K, N)
    w = _matrix(g, max(G, 1) * wr, wc, 1 / math.sqrt(K), dt, 0)
    st["W"] = w.view(G, wr, wc) if G else w
    st["R"] = _matrix(g, M, N, 1.0 if op != "act_grad" else 0.01, odt, pad) if case["res"] else None
    st["Y"] = torch.empty(M, N, dtype=odt, device="cuda")
    st["keep"] = torch.empty(M, N, dtype=odt, device="cuda") if case["keep"] else None
    if op == "act_grad":
        st["X"] = _matrix(g, M, K, 0.01, dt, pad)
        st["Z"] = _activations(g, M, N, odt, pad)
    else:
        st["X"] = _activations(g, M, K, dt, pad)
        b = _matrix(g, max(G, 1), N, 0.5, odt, 0)
        st["bias"] = (b if G else b[0]) if case["bias"] else None
    return st


# ---- the plain form: elementary operations in 32 bits ---------------------------------
def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x * 0.70710678118654752)
    return x


def _slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    return 0.5 * torch.erfc(-x * 0.70710678118654752) + x * torch.exp(-0.5 * x * x) * 0.3989422804014327


def _products(x, w, sizes, trans):
    """Each group's rows of x times its own matrix of w."""
    parts, at = [], 0
    for g, n in enumerate(sizes):
        if n:
            m = w[g].float() if w.dim() == 3 else w.float()
            parts.append(x[at:at + n].float() @ (m.t() if trans else m))
        at += n
    return torch.cat(parts)


def _run_own(st):
    import dense_gemm_amd as dg

    c = st["case"]
    op, G = c["op"], c["groups"]
    if op == "dw":
        dw = dg.gemm_dw(st["dY"], st["X"], st["dW"], offsets=st.get("offsets"), dbias=st["dbias"])
        return {"dw": dw, "dbias": st["dbias"]} if c["bias"] else dw
    if op == "act_grad":
        grad = dict(transB=c["trans"], activation=c["act"], R=st["R"], H=st["keep"])
        if G:
            y = dg.gemm_grouped_act_grad(st["X"], st["W"], st["offsets"], st["Z"], st["Y"], **grad)
        else:
            y = dg.gemm_act_grad(st["X"], st["W"], st["Z"], st["Y"], **grad)
    else:
        layer = dict(transB=c["trans"], bias=st["bias"], activation=c["act"], R=st["R"], Z=st["keep"])
        if G:
            y = dg.gemm_grouped(st["X"], st["W"], st["offsets"], st["Y"], **layer)
        else:
            y = dg.gemm_fused(st["X"], st["W"], st["Y"], **layer)
    return {"y": y, "keep": st["keep"]} if c["keep"] else y


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op, G, sizes = c["op"], c["groups"], st["sizes"]
    odt = TYPES[c["out"]]
    if op == "dw":
        dw, db, at = [], [], 0
        for n in sizes:
            dy, x = st["dY"][at:at + n].float(), st["X"][at:at + n].float()
            dw.append((dy.t() @ x).to(odt))
            db.append(dy.sum(0))
            at += n
        dw = torch.stack(dw) if G else dw[0]
        return {"dw": dw, "dbias": torch.stack(db) if G else db[0]} if c["bias"] else dw
    x = _products(st["X"], st["W"], sizes, c["trans"])
    if op == "act_grad":
        if c["res"]:
            x = x + st["R"].float()
        y, keep = x * _slope(st["Z"].float(), c["act"]), x
    else:
        if c["bias"]:
            b = st["bias"].float()
            x = x + (torch.cat([b[g].expand(n, -1) for g, n in enumerate(sizes)]) if G else b)
        y, keep = _act(x, c["act"]), x
        if c["res"]:
            y = y + st["R"].float()
    return {"y": y.to(odt), "keep": keep.to(odt)} if c["keep"] else y.to(odt)


def work(case):
    op, G = case["op"], case["groups"]
    e, o = (4 if case["type"] == "f32" else 2), (4 if case["out"] == "f32" else 2)
    if op == "dw":
        R, M, N = case["rows"], case["M"], case["N"]
        return {"bytes": R * (M + N) * e + max(G, 1) * M * N * o + (max(G, 1) * M * 4 if case["bias"] else 0), "flops": 2 * R * M * N}
    M, N, K = case["M"], case["N"], case["K"]
    # the matrices of experts that have a token: an eighth has none by design, and no more than there are tokens
    used = min(M, G - (G // 8 if G > 4 else 0)) if G else 1
    mats = 1 + case["res"] + case["keep"] + (op == "act_grad")
    bias = used * N * o if op != "act_grad" and case["bias"] else 0
    return {"bytes": M * K * e + used * N * K * e + bias + mats * M * N * o, "flops": 2 * M * N * K}


# ---- the definition in 64 bits ----------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    ends = [sum(st["sizes"][:i + 1]) for i in range(len(st["sizes"]))]
    spans = [(e - n, e) for e, n in zip(ends, st["sizes"])]
    if case["op"] == "dw":
        M, N = case["M"], case["N"]
        dw = torch.zeros(len(spans), M, N, dtype=f64, device="cuda")
        db = torch.zeros(len(spans), M, dtype=f64, device="cuda")
        for g, (a, b) in enumerate(spans):
            if a < b:
                dy = st["dY"][a:b].to(f64)
                torch.mm(dy.transpose(0, 1).contiguous(), st["X"][a:b].to(f64), out=dw[g])
                db[g] = dy.sum(0)
        if not case["groups"]:
            dw, db = dw[0], db[0]
        return {"dw": dw, "dbias": db} if case["bias"] else dw
    M, N = case["M"], case["N"]
    y = torch.empty(M, N, dtype=f64, device="cuda")
    keep = torch.empty(M, N, dtype=f64, device="cuda") if case["keep"] else None
    root2 = math.sqrt(2.0)
    for g, (a, b) in enumerate(spans):
        if a == b:
            continue
        w = (st["W"][g] if case["groups"] else st["W"]).to(f64)
        z = torch.mm(st["X"][a:b].to(f64), w.transpose(0, 1).contiguous() if case["trans"] else w)
        if case["op"] == "act_grad":
            if case["res"]:
                z += st["R"][a:b].to(f64)
            t = st["Z"][a:b].to(f64)
            if case["act"] == "relu":
                v = torch.where(t > 0, z, torch.zeros_like(z))
            else:
                v = z * (torch.special.erfc(-t / root2) / 2 + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi))
        else:
            if case["bias"]:
                z += (st["bias"][g] if case["groups"] else st["bias"]).to(f64)
            if case["act"] == "relu":
                v = torch.maximum(z, torch.zeros_like(z))
            elif case["act"] == "gelu":
                v = z * torch.special.erfc(-z / root2) / 2
            else:
                v = z.clone()
            if case["res"]:
                v = v + st["R"][a:b].to(f64)
        y[a:b] = v
        if keep is not None:
            keep[a:b] = z
    return {"y": y, "keep": keep} if case["keep"] else y
