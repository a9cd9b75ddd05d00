"""The 64-bit form of token_logps and of its gradient, from the formulas of
include/hkv.h, with a bound for each output.

u is half a unit in the last place of a float32, 2^-24.  Let near be the largest
magnitude among the entries that count (within 120 of the row's maximum m; below
that exp is under 2^-173 and 0 in float32), at most 16384 + 120: past 16384 the
kernels subtract the maximum before they scale.  An exponential is then off by
2^-21 of itself (CUDA's fast one near zero) and by what its argument is rounded
by, 8 near u; a float32 sum of V terms by V / 32 + 64 roundings (the longest chain
of one thread, and the joins).  Together: rel = 2^-20 + 8 near u + (V / 32 + 64) u.
 - log sum exp: rel for the sum, 4 u of itself; log p: as much.
 - entropy = log s - w / s with w / s = sum p (x - m): each term is off by rel, and
   by 2 rel again through s, and x - m by 4 near u.
 - p itself is a multiple of 2^-149 where it is below 2^-126 (the spacing of float32's
   subnormals): its rounding and the exponential's last place are up to 2^-148 there,
   no longer relative, and the gradient has them times its bracket.
 - gradient p (-g - h (log p + H)) + g [label]: p is off by what log p is off by and by
   2^-20 + 8 |log p| u, the bracket by log p's and H's errors and 8 u of itself;
   the label's entry by 4 u g; then half a unit of the output's type."""
import torch

from tests.operators_plain import U

u = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -148, torch.bfloat16: 2.0 ** -132, torch.float16: 2.0 ** -24}


def token_logps(logits, labels, top, g=None, h=None):
    """{name: (value, bound)}, and top_ids as they have to be."""
    x = logits.double()
    rows, vocab = x.shape
    counted = torch.ones(rows, dtype=torch.bool, device=x.device)
    if labels is not None:
        counted = (labels >= 0) & (labels < vocab)
    # a counted row without a sum has NaNs
    bad = counted & (x.isnan().any(1) | (x == torch.inf).any(1) | (x == -torch.inf).all(1))
    fine = (counted & ~bad)[:, None]
    x = torch.where(fine, x, 0.0)
    m = x.amax(1, keepdim=True)
    d = x - m
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    finite = torch.where(d > -120, lp, 0.0)  # p of the others is below 2^-173
    ent = -(p * finite).sum(1)
    near = (torch.where(d > -120, x, m).abs().amax(1)).clamp_max(16384.0) + 120
    rel = 2.0 ** -20 + 8 * near * u + (vocab / 32 + 64) * u
    lse = torch.logsumexp(x, 1)
    e_lp = rel + 4 * u * (lse - m[:, 0]).abs() + 2 * u
    e_ent = 3 * rel * (1 + (p * torch.where(d > -120, d, 0.0).abs()).sum(1)) + 4 * near * u + 8 * u * (1 + ent)

    def rowwise(v, none, e):
        v = torch.where(counted, torch.where(bad, torch.nan, v), none)
        return v, torch.where(fine[:, 0], e, 0.0)

    out = {"entropy": rowwise(ent, 0.0, e_ent)}
    at = torch.arange(rows, device=x.device)
    label = None
    if labels is not None:
        label = torch.where(counted, labels, 0)
        v = lp[at, label]
        out["logps"] = rowwise(v, 0.0, e_lp + 4 * u * v.nan_to_num(0, 0, 0).abs())
    if top:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        v = lp.gather(1, order)
        e = e_lp[:, None] + 4 * u * v.nan_to_num(0, 0, 0).abs()
        v = torch.where(counted[:, None], torch.where(bad[:, None], torch.nan, v), -torch.inf)
        out["top_logps"] = v, torch.where(fine, e, 0.0)
        out["top_ids"] = torch.where(fine, order, -1)
    if g is not None or h is not None:
        g = torch.zeros(rows, dtype=torch.float64, device=x.device) if g is None else g.double()
        h = torch.zeros_like(g) if h is None else h.double()
        g, h = g[:, None], h[:, None]
        e_lp_v = e_lp[:, None] + 4 * u * finite.abs()
        bracket = -g - h * (finite + ent[:, None])
        size = g.abs() + h.abs() * (finite.abs() + ent[:, None])
        grad = p * bracket
        e = p * (e_lp_v + 2.0 ** -20 + 8 * u * finite.abs()) * size
        e = e + 2.0 ** -148 * size
        e = e + p * (h.abs() * (e_lp_v + e_ent[:, None]) + 8 * u * size)
        if label is not None:
            grad[at, label] += g[:, 0]
            e[at, label] += 4 * u * g[:, 0].abs()
        kind = U[logits.dtype]
        e = e * (1 + kind) + grad.abs() * kind + TINY[logits.dtype]
        grad = torch.where(fine, grad, torch.where(bad[:, None], torch.nan, 0.0))
        out["grad"] = grad, torch.where(fine, e, 0.0)
    return out
