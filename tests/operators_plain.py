"""Plain 64-bit forms of the operators on looked-up rows, from the formulas of
include/hkv.h, and the error bounds the tests hold the kernels to.

Bounds.  u(type) is half a unit in the last place, relative: 2^-24, 2^-8,
2^-11 for float32, bfloat16, float16.  An exponential or logarithm of CUDA's
fast single-precision functions is taken as right to 2^-21 for arguments near
zero, and an argument's own rounding moves exp by the argument's error."""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def quantize(x):
    """(codes [rows, blocks, 32], scale bytes [rows, blocks]) of a matrix, on the
    CPU and element by element: the nearest level, ties to the even code."""
    x = x.detach().cpu().double()
    rows, cols = x.shape
    blocks = -(-cols // 32)
    b = torch.zeros((rows, blocks * 32), dtype=torch.float64)
    b[:, :cols] = x
    b = b.view(rows, blocks, 32)
    top = b.abs().amax(2)
    finite = top.isfinite()
    _, e = torch.frexp(torch.where(finite, top, 1.0))  # top = f * 2^e, f in [.5, 1)
    biased = torch.where(top < 2.0 ** -126, 0, e.long() - 1 + 127)
    byte = torch.where(finite, (biased - 2).clamp_min(0), 255)
    scale = torch.tensor(2.0, dtype=torch.float64) ** (byte.double() - 127)
    v = torch.where(finite[..., None], b / scale[..., None], 0.0)
    a = v.abs().clamp_max(6.0)
    levels = torch.tensor(LEVELS, dtype=torch.float64)
    gap = (a[..., None] - levels).abs()
    best = gap.amin(-1, keepdim=True)
    # of two levels equally near, the even code
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[(gap[..., order] == best).to(torch.uint8).argmax(-1)]
    code = code + 8 * (torch.signbit(b) & finite[..., None])
    return code, byte


def values(code, byte, cols):
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64)
    scale = torch.tensor(2.0, dtype=torch.float64) ** (byte.double() - 127)
    scale = torch.where(byte == 255, torch.nan, scale)
    return (levels[code.long()] * scale[..., None]).flatten(1)[:, :cols]


def layout(code, byte):
    """The bytes of include/hkv.h for codes and scale bytes."""
    rows, blocks = byte.shape
    code = code.reshape(rows, blocks * 32)
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    groups = -(-blocks // 4)
    scales = torch.zeros((-(-rows // 128), groups, 512), dtype=torch.uint8)
    r = torch.arange(rows)[:, None]
    k = torch.arange(blocks)[None]
    scales[r // 128, k // 4, (r % 32) * 16 + r // 32 % 4 * 4 + k % 4] = byte.to(torch.uint8)
    return codes, scales


def matmul(a, b):
    """a b^T of 64-bit values and the bound of a float32 sum in any order whose
    longest chain is one addition for each 64 columns and 64 more."""
    y = a @ b.t()
    size = a.abs() @ b.abs().t()
    return y, size * ((a.shape[1] / 64 + 64) * 2.0 ** -23)


def preference(logits, labels, offsets, ref, beta, smoothing, average, dlosses=None):
    """Losses, ratios, token log probabilities, the gradient, and a bound for each."""
    x = logits.double()
    rows, vocab = x.shape
    ends = offsets.tolist()
    pairs = len(ends) // 2
    counted = (labels >= 0) & (labels < vocab)
    at = torch.arange(rows, device=x.device)
    label = torch.where(counted, labels, 0)
    lse = torch.logsumexp(x, 1)
    lp = torch.where(counted, x[at, label] - lse, 0.0)
    delta = torch.where(counted, lp - (ref.double() if ref is not None else 0.0), 0.0)
    u = 2.0 ** -24
    top = x.masked_fill(~x.isfinite(), 0).abs().amax(1)
    # sum of exponentials: a relative error of each (2^-21 and its argument's
    # rounding, up to 2 max|x| u) and of the additions (vocab / 32 in one
    # thread at most, 64 to join); then the logarithm and two subtractions
    e_lp = torch.where(counted, 2.0 ** -20 + 8 * top * u + (vocab / 32 + 64) * u
                       + 4 * u * lse.nan_to_num(0, 0, 0).abs(), 0.0)
    r, e_r, n = [], [], []
    for a, b in zip(ends, ends[1:]):
        k = int(counted[a:b].sum())
        d = delta[a:b]
        s, e = d.sum(), e_lp[a:b].sum() + (b - a + 2) * u * d.nan_to_num(0, 0, 0).abs().sum()
        n.append(1.0 / k if average and k else 0.0 if average else 1.0)
        r.append(s * n[-1])
        e_r.append(e * n[-1] + 4 * u * (s * n[-1]).nan_to_num(0, 0, 0).abs())
    r, e_r = torch.stack(r), torch.stack(e_r)
    h = beta * (r[:pairs] - r[pairs:])
    e_h = abs(beta) * (e_r[:pairs] + e_r[pairs:]) + 4 * u * abs(beta) * (
        r[:pairs].abs() + r[pairs:].abs()).nan_to_num(0, 0, 0)
    ls = torch.nn.functional.logsigmoid
    loss = torch.zeros_like(h)
    if smoothing < 1:
        loss = loss - (1 - smoothing) * ls(h)
    if smoothing > 0:
        loss = loss - smoothing * ls(-h)
    e_loss = e_h + 2.0 ** -21 * (1 + loss.nan_to_num(0, 0, 0).abs())
    slope = beta * (torch.sigmoid(h) - (1 - smoothing))
    e_slope = abs(beta) * (e_h / 4 + 2.0 ** -21)
    up = dlosses.double() if dlosses is not None else torch.ones_like(h)
    grad, e_grad = torch.zeros_like(x), torch.zeros_like(x)
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        p, sign = i % pairs, 1 if i < pairs else -1
        g = sign * slope[p] * up[p] * n[i]
        e_g = (e_slope[p] * up[p].abs() + 4 * u * g.abs()) * n[i]
        soft = torch.softmax(x[a:b], 1)
        hot = torch.zeros_like(soft)
        hot[at[:b - a], label[a:b]] = 1
        keep = counted[a:b, None]
        grad[a:b] = torch.where(keep, g * (hot - soft), 0.0)
        e_soft = soft * (e_lp[a:b, None] + 2.0 ** -20 + 8 * u * (x[a:b] - lse[a:b, None]).nan_to_num(0, 0, 0).abs())
        e_grad[a:b] = torch.where(keep, e_g * (hot - soft).abs() + g.abs() * (e_soft + 2 * u), 0.0)
    kind = U[logits.dtype]
    tiny = {torch.float32: 2.0 ** -148, torch.bfloat16: 2.0 ** -132, torch.float16: 2.0 ** -24}[logits.dtype]
    e_grad = e_grad * (1 + kind) + grad.abs() * kind + tiny
    return {"losses": (loss, e_loss), "ratios": (r, e_r), "logps": (lp, e_lp), "grad": (grad, e_grad)}


def near(got, want, bound, what=""):
    """Non-finite values agree, finite ones to within the bound."""
    got, want = got.double(), want.to(got.device)
    bound = bound.to(got.device)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaNs differ"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{what}: infinities differ"
    over = (got - want).abs()[fine] - bound[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: {float((got - want).abs()[fine].max()):.3g} off, {float(over.max()):.3g} over the bound"
