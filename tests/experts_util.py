"""Plain 64-bit references and derived tolerances for the expert products and
the router.

Tolerances count roundings.  u(t) = finfo(t).eps / 2 is half a step of the
output's type.  A float32 sum of n products is off by at most n 2^-24 times
the sum of their absolute values, in whatever order it is taken (the
first-order bound); the matrix instructions sum 32 products at a time to
3.6e-8 = 2^-24.7 of their absolute sum (measured), within that bound."""

from __future__ import annotations

import torch

DEV = "cuda:0"
U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(y, dtype):
    """One rounding of y to dtype; the second term is half the smallest
    subnormal."""
    f = torch.finfo(dtype)
    return y.abs() * half_step(dtype) + f.tiny * f.eps / 2


def segments(counts, align=1, extra=0):
    """Offsets [E + 1], sizes [E, 3] and capacity for these row counts."""
    c = torch.tensor(counts, dtype=torch.int64)
    off = torch.zeros(len(counts) + 1, dtype=torch.int64)
    off[1:] = torch.cumsum((c + align - 1) // align * align, 0)
    sizes = torch.stack((c, torch.full_like(c, 11), torch.full_like(c, 13)), 1)
    return {"offsets": off.to(torch.int32).to(DEV), "sizes": sizes.to(torch.int32).to(DEV),
            "rows": int(off[-1]) + extra,
            "spans": [(int(off[e]), int(c[e])) for e in range(len(counts))]}


def live(seg):
    m = torch.zeros(seg["rows"], dtype=torch.bool)
    for b, c in seg["spans"]:
        m[b:b + c] = True
    return m


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def rows_with_nan(seg, width, dtype, seed, scale=1.0):
    """Rows of the segments from N(0, scale^2), NaN everywhere else."""
    x = normal((seg["rows"], width), dtype, seed, scale)
    x[~live(seg)] = float("nan")
    return x


def products(seg, x, w):
    """y[r] = w[e] @ x[r] and the sum of absolute products, float64 on the CPU
    (zeros outside the segments)."""
    y = torch.zeros(seg["rows"], w.shape[1], dtype=torch.float64)
    s = torch.zeros_like(y)
    for e, (b, c) in enumerate(seg["spans"]):
        a, m = x[b:b + c].double(), w[e].double()
        y[b:b + c] = a @ m.T
        s[b:b + c] = a.abs() @ m.abs().T
    return y, s


def gated(y, err):
    """silu(g) u of y = (g, u) with errors err, and its error: silu' <= 1.1,
    |silu(g)| <= |g|, and 8 more float32 roundings (the exponential, with an
    argument of |g| roundings, the sum, the division and the product)."""
    n = y.shape[1] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu + h.abs() * (8 + g.abs()) * U32


def check(got, want, err, dtype, what=""):
    """|got - want| <= err + one rounding of what may lie err away."""
    got = got.detach().cpu().double()
    tol = err + rounding(want.abs() + err, dtype)
    off = (got - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got "
                             f"{float(got[i])}, want {float(want[i])} +- {float(tol[i])}")
