"""A layer's products in 64 bits, from their formulas, with bounds on how far an
fp32-accumulated result rounded once may lie from them.

The bounds.  Let u = 2^-24 (half an fp32 step).  K products summed in fp32 in any
order are off by at most (K + 1) u sum |a b| to first order, and the epilogue's
few operations by a few u of what they handle: `err` below carries an absolute
bound beside every value.  Phi's relative error on its smaller tail is at most
PHI(x): 16-bit outputs 6e-6 for the polynomial and (4 + 3 x^2) 2^-23 for exp(-x^2 / 2)
by the hardware's exp2 of an argument rounded to fp32; fp32 outputs 16 u for
erfcf and 4 x^2 u for its rounded argument.  A rounding to the output's type adds half a
step, eps / 2 of the value, and half the least subnormal."""
import math

import numpy as np
import torch
from scipy.special import erfc

U = 2.0 ** -24
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def np64(t):
    return t.detach().double().cpu().numpy()


def phi_rel(x, out):
    return (16 + 4 * x * x) * U if out == torch.float32 else 6e-6 + (4 + 3 * x * x) * 2.0 ** -23


def tail(x):
    """Phi(-|x|)."""
    return 0.5 * erfc(np.abs(x) / math.sqrt(2))


def act(x, name):
    if name == "relu":
        return np.where(x < 0, 0, x)
    if name == "gelu":
        return x * 0.5 * erfc(-x / math.sqrt(2))
    return x


def slope(x, name):
    if name == "relu":
        return np.where(x > 0, 1.0, np.where(x <= 0, 0.0, x))
    pdf = np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    with np.errstate(invalid="ignore"):
        s = 0.5 * erfc(-x / math.sqrt(2)) + np.where(np.abs(x) < 40, x * pdf, 0)
    return np.where(np.isnan(x), x, s)


def rounding(ref, out):
    f = torch.finfo(out)
    return np.abs(ref) * f.eps / 2 + f.smallest_normal * f.eps / 2


def spans(offsets, rows):
    """The rows of each group, or all rows as one."""
    return [(0, rows)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def product(A, B, offsets, transB, alpha):
    """(alpha A op(B_g) by rows, bound): rows of no group stay NaN."""
    M = A.shape[0]
    N = B.shape[-2] if transB else B.shape[-1]
    z, err = np.full((M, N), np.nan), np.full((M, N), np.nan)
    for g, (a, b) in enumerate(spans(offsets, M)):
        w = B if offsets is None else B[g]
        w = w.T if transB else w
        z[a:b] = alpha * (A[a:b] @ w)
        err[a:b] = abs(alpha) * (np.abs(A[a:b]) @ np.abs(w)) * (A.shape[1] + 4) * U
    return z, err


def forward(A, B, offsets=None, transB=False, alpha=1.0, bias=None, activation="none", R=None, beta=1.0, out=torch.float32):
    """{name: (value, bound)} of C and Z."""
    z, err = product(A, B, offsets, transB, alpha)
    if bias is not None:
        for g, (a, b) in enumerate(spans(offsets, A.shape[0])):
            z[a:b] += bias if offsets is None else bias[g]
    err = err + 2 * U * np.abs(z)
    c = act(z, activation)
    cerr = err * (1.13 if activation == "gelu" else 1)
    if activation == "gelu":
        cerr = cerr + phi_rel(z, out) * np.abs(z) * tail(z) + 4 * U * np.abs(c)
    if R is not None:
        c = c + beta * R
        cerr = cerr + 2 * U * (np.abs(c) + np.abs(beta * R))
    return {"C": (c, cerr + rounding(c, out)), "Z": (z, err + rounding(z, out))}


def act_grad(A, B, Z, offsets=None, transB=False, alpha=1.0, activation="gelu", R=None, beta=1.0, out=torch.float32):
    """{name: (value, bound)} of C and H."""
    h, err = product(A, B, offsets, transB, alpha)
    if R is not None:
        h = h + beta * R
        err = err + 2 * U * (np.abs(h) + np.abs(beta * R))
    err = err + 2 * U * np.abs(h)
    s = slope(Z, activation)
    with np.errstate(invalid="ignore"):
        c = np.where(s == 0, 0, h * s) if activation == "relu" else h * s
        serr = 0
        if activation == "gelu":
            zphi = np.abs(Z) * np.exp(-Z * Z / 2) / math.sqrt(2 * math.pi)
            # exp's and Phi's relative errors, and those of four fp32 operations
            serr = phi_rel(Z, out) * (tail(Z) + zphi) + 4 * U * (1 + zphi)
        cerr = err * np.abs(s) + np.abs(h) * serr + 2 * U * np.abs(c)
    return {"C": (c, cerr + rounding(c, out)), "H": (h, err + rounding(h, out))}


def dw(A, B, offsets=None, alpha=1.0, beta=0.0, C=None, dbias=None, out=torch.float32):
    """{name: (value, bound)} of C and dbias."""
    cs, ce, ds, de = [], [], [], []
    for g, (a, b) in enumerate(spans(offsets, A.shape[0])):
        x, y = A[a:b], B[a:b]
        c = alpha * (x.T @ y)
        e = abs(alpha) * (np.abs(x).T @ np.abs(y)) * (b - a + 4) * U
        d, f = x.sum(0), np.abs(x).sum(0) * (b - a + 2) * U
        if beta:
            c0 = C if offsets is None else C[g]
            c, e = c + beta * c0, e + 2 * U * np.abs(beta * c0)
            if dbias is not None:
                d0 = dbias if offsets is None else dbias[g]
                d, f = d + beta * d0, f + 2 * U * np.abs(beta * d0)
        cs.append(c), ce.append(e + 2 * U * np.abs(c) + rounding(c, out))
        ds.append(d), de.append(f + 2 * U * np.abs(d))
    if offsets is None:
        return {"C": (cs[0], ce[0]), "dbias": (ds[0], de[0])}
    N, M = B.shape[1], A.shape[1]
    return {"C": (np.array(cs).reshape(-1, M, N), np.array(ce).reshape(-1, M, N)),
            "dbias": (np.array(ds).reshape(-1, M), np.array(de).reshape(-1, M))}


def check(got, want, what=""):
    """Every element within its bound; NaN where the reference is NaN, equal infinities."""
    ref, bound = want
    x = np64(got)
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    if x.size == 0:
        return
    nan, inf = np.isnan(ref), np.isinf(ref)
    assert (np.isnan(x) == nan).all(), f"{what}: NaN in other places"
    assert (x[inf] == ref[inf]).all(), f"{what}: infinities differ"
    ok = ~(nan | inf)
    over = np.abs(x[ok] - ref[ok]) - bound[ok]
    if over.size and over.max() > 0:
        i = np.argmax(over)
        r = np.abs(x[ok] - ref[ok]) / bound[ok]
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.size} elements past their bound, worst "
                             f"{r.max():.3g} times it; got {x[ok][i]!r}, want {ref[ok][i]!r}")
