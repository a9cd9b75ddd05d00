"""The 64-bit form of adapter_matmul and of its gradients, from the formulas of
include/hkv.h, with a bound for each output.

Sums are float32 sums in tensor cores, which cut what they add up: a unit in the
last place, 2^-23, of the sum of magnitudes for each addition of a chain, one for
each 16 terms (six where float32 matrices are taken in three parts), and 128 more
where the parts of warps and blocks are joined.  A float32 matrix goes in as three
parts; what is left of the products is below 2^-22 of a term.  The hidden numbers
go on in two parts of 8 bits where matrices have 16 (the rest is below 2^-15), in
three where they have 32.  A result is then rounded once, by half a unit of its type."""
import torch

from tests.operators_plain import U

TINY = {torch.float32: 2.0 ** -148, torch.bfloat16: 2.0 ** -132, torch.float16: 2.0 ** -24}


def _product(a, b, e_a, rest, wide):
    """a b^T, and its bound: a is off by e_a, and `rest` of each term is left out."""
    size = a.abs() @ b.abs().t()
    chain = (6 if wide else 1) * a.shape[1] / 16 + 128
    e = size * (chain * 2.0 ** -23 + rest)
    return a @ b.t(), e if e_a is None else e + e_a @ b.abs().t()


def adapter_matmul(x, down, up, offsets, which, scales=None, base=None, dy=None, dx_base=None):
    """{name: (value, bound)} of out, and of dx, ddown and dup where dy is given."""
    kind = x.dtype
    wide = kind == torch.float32
    first = 2.0 ** -22 if wide else 0.0
    then = 2.0 ** -22 if wide else 2.0 ** -15
    tokens, k = x.shape
    count, rank = down.shape[:2]
    n = up.shape[1]
    dev = x.device
    zero = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    u = 2.0 ** -24

    def rounded(v, e):
        return v, e * (1 + U[kind]) + (v.abs() * U[kind]).nan_to_num(0, 0, 0) + TINY[kind]

    y = zero(tokens, n) if base is None else base.double().clone()
    e_y = zero(tokens, n)
    if dy is not None:
        dx = zero(tokens, k) if dx_base is None else dx_base.double().clone()
        e_dx = zero(tokens, k)
        dd, e_dd, du, e_du = zero(count, rank, k), zero(count, rank, k), zero(count, n, rank), zero(count, n, rank)
    ends = offsets.tolist()
    for a, b, w in zip(ends, ends[1:], which.tolist()):
        if not 0 <= w < count or b <= a:
            continue
        c = 1.0 if scales is None else float(scales[w])
        d, v, xs = down[w].double(), up[w].double(), x[a:b].double()
        h, e_h = _product(xs, d, None, first, wide)
        p, e_p = _product(h, v, e_h, then + 4 * u, wide)
        y[a:b] += c * p
        e_y[a:b] = abs(c) * e_p + 2 * u * y[a:b].abs()
        if dy is None:
            continue
        g = dy[a:b].double()
        dh, e_dh = _product(g, v.t(), None, first, wide)
        dh, e_dh = c * dh, abs(c) * e_dh + 2 * u * (c * dh).abs()
        p, e_p = _product(dh, d.t(), e_dh, then, wide)
        dx[a:b] += p
        e_dx[a:b] = e_p + 2 * u * dx[a:b].abs()
        p, e_p = _product(dh.t(), xs.t(), e_dh.t(), then, wide)
        dd[w] += p
        e_dd[w] += e_p + 2.0 ** -20 * (dh.abs().t() @ xs.abs())  # (further requests lengthen the chain)
        p, e_p = _product(g.t(), (c * h).t(), None, then + 4 * u, wide)
        du[w] += p
        e_du[w] += e_p + abs(c) * (g.abs().t() @ e_h) + 2.0 ** -20 * abs(c) * (g.abs().t() @ h.abs())
    out = {"out": rounded(y, e_y)}
    if dy is not None:
        out |= {"dx": rounded(dx, e_dx), "ddown": rounded(dd, e_dd), "dup": rounded(du, e_du)}
    return out
