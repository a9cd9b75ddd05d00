"""Cases of the operators between a lookup of rows and their write-back: 4-bit
microscaled copies and their product, the preference loss over the logits with
its gradient, and the global gradient norm with clipping.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, through
hash_table_cache_gb300.

The 4-bit format (OCP microscaling, MXFP4): blocks of 32 along a row, a scale
byte s per block standing for 2^(s-127) with s = max(E - 2, 0), E the biased
exponent of the block's largest magnitude as a 32-bit float, and elements of
{0, .5, 1, 1.5, 2, 3, 4, 6} with a sign, nearest to x / scale with ties to the
even code.  A block that holds a NaN or an infinity has s = 255 and stands for
NaN.  Two codes a byte, the lower column in the low half; a row's codes are
padded with zeros to whole blocks; scales are held in groups of 128 rows by 4
blocks, byte (row % 32) * 16 + (row // 32 % 4) * 4 + block % 4 of a group.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the 4-bit copy of a table's rows as a serving process keeps it, read back as bf16
        {"name": "rows to 4 bits", "op": "quantize", "rows": 1000003, "cols": 128, "type": "f32", "both": False},
        # an output gradient, copied along both of its axes for the two products of a backward pass
        {"name": "gradient both ways", "op": "quantize", "rows": 4095, "cols": 8200, "type": "bf16", "both": True},
        # one token through a projection held in 4 bits: latency
        {"name": "one token", "op": "product", "m": 1, "n": 4096, "k": 4096, "type": "bf16"},
        # a batch's logits over candidate rows of 64 floats: the output is what it costs
        {"name": "candidate logits", "op": "product", "m": 2048, "n": 131072, "k": 64, "type": "bf16"},
        # a long prompt through a wide projection
        {"name": "wide projection", "op": "product", "m": 8192, "n": 8192, "k": 8192, "type": "bf16"},
        # a layer's training step: forward, the input's and the weight's gradient, all three products in 4 bits
        {"name": "training step", "op": "step", "m": 4099, "n": 4096, "k": 4096, "type": "bf16"},
        # a few short pairs over a small item vocabulary: latency
        {"name": "a few pairs", "op": "loss", "pairs": 4, "length": 12, "vocab": 1000, "type": "f32", "backward": True},
        # an ordinary training batch
        {"name": "a batch of pairs", "op": "loss", "pairs": 16, "length": 128, "vocab": 32768, "type": "bf16", "backward": True},
        # evaluation over the candidate vocabulary
        {"name": "evaluation", "op": "loss", "pairs": 32, "length": 128, "vocab": 131072, "type": "bf16", "backward": False},
        # a small tower beside the table: latency
        {"name": "a small tower", "op": "clip", "count": 24, "total": 100000, "type": "f32", "out": "f32", "clips": True},
        # a step whose norm stays below the limit: gradients in place, not changed
        {"name": "below the limit", "op": "clip", "count": 300, "total": 100000000, "type": "f32", "out": "in place", "clips": False},
        # many bf16 gradients clipped into the 32-bit buffer that an optimizer reads
        {"name": "clipped into 32 bits", "op": "clip", "count": 400, "total": 1000000000, "type": "bf16", "out": "f32", "clips": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "step", "loss", "clip"])
    t16 = rng.choice(["bf16", "f16"])
    if op == "quantize":
        cols = _log(rng, 8, 16384)
        rows = _log(rng, 1, max(1, min(1000000, 100000000 // cols)))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["f32", "bf16", "f16"]), "both": rng.random() < 0.5}
    if op == "product":
        k = _log(rng, 8, 8192)
        n = _log(rng, 32, 131072)
        m = _log(rng, 1, max(1, min(8192, 250000000 // n, 500000000000 // (n * k))))
        return {"op": op, "m": m, "n": n, "k": k, "type": t16}
    if op == "step":
        n, k = _log(rng, 32, 6000), _log(rng, 32, 6000)
        return {"op": op, "m": _log(rng, 16, 6000), "n": n, "k": k, "type": t16}
    if op == "loss":
        vocab = _log(rng, 50, 131072)
        pairs = _log(rng, 1, 64)
        length = _log(rng, 1, max(1, min(2048, 300000000 // (vocab * pairs))))
        return {"op": op, "pairs": pairs, "length": length, "vocab": vocab, "type": rng.choice(["f32", "bf16", "f16"]),
                "backward": rng.random() < 0.7}
    return {"op": op, "count": _log(rng, 1, 600), "total": _log(rng, 3000, 300000000), "type": rng.choice(["f32", "bf16"]),
            "out": rng.choice(["f32", "in place"]), "clips": False} | ({"out": "f32", "clips": True} if rng.random() < 0.5 else {})


def _sizes(case):
    """Element counts of a clip case's tensors: many small ones, a few that hold most of it."""
    rng = random.Random(case["count"] * 1000003 + case["total"])
    share = [math.exp(rng.gauss(0.0, 1.5)) for _ in range(case["count"])]
    return [max(1, int(case["total"] * s / sum(share))) for s in share]


def _lengths(case):
    """Tokens of each sequence of a loss case: the first half chosen, the second rejected."""
    rng = random.Random(case["pairs"] * 7919 + case["length"])
    return [max(1, int(case["length"] * rng.uniform(0.3, 1.7))) for _ in range(2 * case["pairs"])]


def _starts(sizes, unit):
    """Offsets at multiples of `unit` for consecutive arrays, and the end of the last."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // unit) * unit)
    return at


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
    return x.mul_(scale).to(dtype)


def _hidden(g, m, k, dtype):
    """Hidden states: unit variance with a few columns that are several times larger."""
    x = _normal(g, (m, k), torch.float32)
    x *= 1 + 6 * (torch.rand(k, generator=g, device=DEV) < 0.02)
    return x.to(dtype)


def _pack(x):
    """A matrix in 4 bits, laid out as the format says, for weights that a program lays out once."""
    code, scale, _ = _encode(x.float())
    rows, blocks = scale.shape
    code = code.reshape(rows, blocks * 32).to(torch.uint8)
    up = torch.zeros((-(-rows // 128) * 128, -(-blocks // 4) * 4), dtype=torch.uint8, device=DEV)
    up[:rows, :blocks] = scale.to(torch.uint8)
    up = up.reshape(-1, 4, 32, up.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(up.shape[0] // 128, up.shape[1] // 4, 512)
    return code[:, 0::2] + 16 * code[:, 1::2], up.contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    dtype = TYPES[case["type"]]
    if op == "quantize":
        s["x"] = _normal(g, (case["rows"], case["cols"]), dtype, 0.02)
        # embeddings and gradients alike differ in scale from row to row
        s["x"] *= torch.exp(1.5 * torch.randn((case["rows"], 1), generator=g, device=DEV)).to(dtype)
    elif op == "product":
        s["x"] = _hidden(g, case["m"], case["k"], dtype)
        s["codes"], s["scales"] = _pack(_normal(g, (case["n"], case["k"]), torch.float32, 0.02))
    elif op == "step":
        s["x"] = _hidden(g, case["m"], case["k"], dtype)
        s["w"] = _normal(g, (case["n"], case["k"]), dtype, 0.02)
        s["dy"] = _normal(g, (case["m"], case["n"]), dtype, 0.01)
    elif op == "loss":
        lengths = _lengths(case)
        offsets = _starts(lengths, 1)
        rows, vocab = offsets[-1], case["vocab"]
        logits = _normal(g, (rows, vocab), dtype, 2.0)
        labels = torch.randint(vocab, (rows,), generator=g, device=DEV)
        at = torch.arange(rows, device=DEV)
        logits[at, labels] += (2 + 2 * torch.randn(rows, generator=g, device=DEV)).to(dtype)
        # a prompt's tokens carry no label; a sequence of one token keeps its own
        start = torch.tensor([offsets[i] + lengths[i] // 4 for i in range(len(lengths))], device=DEV)
        s["offsets"] = torch.tensor(offsets, device=DEV)
        seq = torch.bucketize(at, s["offsets"], right=True) - 1
        s["labels"] = torch.where(at < start[seq], -100, labels)
        lp = torch.cat([logits[i:i + 512].float().logsumexp(1) for i in range(0, rows, 512)])
        lp = logits[at, labels].float() - lp
        # the reference model is near the policy
        s["ref"] = lp + 0.3 * torch.randn(rows, generator=g, device=DEV)
        s["logits"] = logits
        s["beta"], s["smoothing"] = 0.1, 0.05
        s["dlosses"] = torch.full((case["pairs"],), 1.0 / case["pairs"], device=DEV)
        if case["backward"]:
            s["dlogits"] = torch.empty_like(logits)
    else:
        sizes = _sizes(case)
        at = _starts(sizes, 64)
        if case["out"] == "in place":
            flat = torch.zeros(at[-1], dtype=dtype, device=DEV)
            s["grads"] = [flat[a:a + n] for a, n in zip(at, sizes)]
            for t in s["grads"]:
                t.copy_(_normal(g, t.shape, dtype, 1e-3))
            s["flat"], s["outs"] = flat, None
        else:
            s["grads"] = [_normal(g, (n,), dtype, 1e-3) for n in sizes]
            s["flat"] = torch.zeros(at[-1], dtype=TYPES[case["out"]], device=DEV)
            s["outs"] = [s["flat"][a:a + n] for a, n in zip(at, sizes)]
        expected = 1e-3 * math.sqrt(sum(sizes))
        s["max_norm"] = expected * (0.25 if case["clips"] else 4.0)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _encode(x):
    """Codes (0..15, [rows, blocks, 32]), scale bytes ([rows, blocks]) and block scales of a 32-bit matrix."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    x = torch.nn.functional.pad(x, (0, blocks * 32 - cols)).reshape(rows, blocks, 32)
    most = x.abs().amax(2)
    e = (most.view(torch.int32) >> 23) & 255
    byte = torch.where(e == 255, 255, (e - 2).clamp_min(0))
    inverse = ((254 - byte.clamp_max(253)) << 23).view(torch.float32)  # 2^(127 - byte)
    a = x * inverse[..., None]
    sign = a.view(torch.int32) < 0
    a = a.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += 8 * sign.to(torch.uint8)
    code = torch.where((byte == 255)[..., None], 0, code)
    return code, byte, _scale(byte)


def _scale(byte):
    """2^(byte - 127), NaN for 255; the smallest is a subnormal."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, 1 << 22, torch.where(b == 255, 0x7FC00000, b << 23))
    return bits.view(torch.float32)


def _decode(code, byte, cols):
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)
    return (level[code.long()] * _scale(byte)[..., None]).flatten(1)[:, :cols]


def _rounded(x):
    """The 32-bit values that a matrix's 4-bit copy stands for."""
    code, byte, _ = _encode(x.float())
    return _decode(code, byte, x.shape[1])


def _unpack(codes, scales, rows, cols):
    blocks = codes.shape[1] // 16
    byte = scales.reshape(scales.shape[0], scales.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = byte.reshape(scales.shape[0] * 128, scales.shape[1] * 4)[:rows, :blocks]
    code = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, blocks, 32)
    return _decode(code, byte, cols)


def _plain_loss(s):
    x = s["logits"].float()
    at = torch.arange(x.shape[0], device=x.device)
    counted = s["labels"] >= 0
    label = s["labels"].clamp_min(0)
    most = x.amax(1)
    lse = most + (x - most[:, None]).exp().sum(1).log()
    logps = torch.where(counted, x[at, label] - lse, 0.0)
    ratio = torch.where(counted, logps - s["ref"], 0.0)
    ends = s["offsets"]
    member = ((at >= ends[:-1, None]) & (at < ends[1:, None])).float()  # [sequences, tokens]
    pairs = s["pairs"]
    r = (member * ratio).sum(1)
    h = s["beta"] * (r[:pairs] - r[pairs:])
    e = s["smoothing"]
    most_h = h.abs()
    tail = (1 + (-most_h).exp()).log()
    losses = (1 - e) * (tail + (-h).clamp_min(0)) + e * (tail + h.clamp_min(0))
    out = {"losses": losses, "ratios": r, "logps": logps}
    if s["backward"]:
        slope = -s["beta"] * ((1 - e) / (1 + h.exp()) - e / (1 + (-h).exp())) * s["dlosses"]
        per_token = (member * torch.cat((slope, -slope))[:, None]).sum(0)
        per_token = torch.where(counted, per_token, 0.0)
        d = -(x - lse[:, None]).exp()
        d[at, label] += 1
        out["dlogits"] = (d * per_token[:, None]).to(s["logits"].dtype)
    return out


def _plain_clip(s):
    outs = s["grads"] if s["outs"] is None else s["outs"]
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    factor = torch.where(norm <= s["max_norm"], 1.0, s["max_norm"] / norm)
    [o.copy_(g.float() * factor) for o, g in zip(outs, s["grads"])]
    return {"norm": norm, "grads": s["flat"]}


def _plain(s):
    op = s["op"]
    if op == "quantize":
        out = [_rounded(s["x"]).to(torch.bfloat16)]
        return out + [_rounded(s["x"].t().contiguous()).to(torch.bfloat16)] if s["both"] else out
    if op == "product":
        return (_rounded(s["x"]) @ _unpack(s["codes"], s["scales"], s["n"], s["k"]).t()).to(s["x"].dtype)
    if op == "step":
        x, w, dy = s["x"], s["w"], s["dy"]
        y = _rounded(x) @ _rounded(w).t()
        dx = _rounded(dy) @ _rounded(w.t().contiguous()).t()
        dw = _rounded(dy.t().contiguous()) @ _rounded(x.t().contiguous()).t()
        return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.to(x.dtype)}
    return _plain_loss(s) if op == "loss" else _plain_clip(s)


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------
def _own(s):
    import hash_table_cache_gb300 as hkv
    op = s["op"]
    if op == "quantize":
        if s["both"]:
            q, qt = hkv.mx_quantize(s["x"], along="both")
            return [q.dequantize(torch.bfloat16), qt.dequantize(torch.bfloat16)]
        return [hkv.mx_quantize(s["x"]).dequantize(torch.bfloat16)]
    if op == "product":
        w = hkv.MXMatrix(s["codes"], s["scales"], s["n"], s["k"])
        return hkv.mx_matmul(hkv.mx_quantize(s["x"]), w, dtype=s["x"].dtype)
    if op == "step":
        dtype = s["x"].dtype
        x, xt = hkv.mx_quantize(s["x"], along="both")
        w, wt = hkv.mx_quantize(s["w"], along="both")
        dy, dyt = hkv.mx_quantize(s["dy"], along="both")
        return {"y": hkv.mx_matmul(x, w, dtype=dtype), "dx": hkv.mx_matmul(dy, wt, dtype=dtype),
                "dw": hkv.mx_matmul(dyt, xt, dtype=dtype)}
    if op == "loss":
        f = hkv.preference_loss(s["logits"], s["labels"], s["offsets"], s["ref"], beta=s["beta"],
                                label_smoothing=s["smoothing"])
        out = {"losses": f.losses, "ratios": f.ratios, "logps": f.logps}
        if s["backward"]:
            out["dlogits"] = hkv.preference_loss_backward(f, s["dlosses"], out=s["dlogits"])
        return out
    norm = hkv.clip_grad_norm(s["grads"], s["max_norm"], outs=s["outs"])
    return {"norm": norm, "grads": s["flat"]}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = 4 if case["type"] == "f32" else 2
    held = lambda r, c: r * (-(-c // 32)) * 17  # noqa: E731  codes and scales of a matrix
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        ways = 2 if case["both"] else 1
        return {"bytes": r * c * (size + 2 * ways), "flops": 2 * r * c * ways}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": size * m * k + held(n, k) + size * m * n, "flops": 2 * m * n * k}
    if op == "step":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * size * (m * k + n * k + m * n), "flops": 6 * m * n * k}
    if op == "loss":
        rows = sum(_lengths(case))
        return {"bytes": rows * (case["vocab"] * size * (2 if case["backward"] else 1) + 16),
                "flops": rows * case["vocab"] * (8 if case["backward"] else 4)}
    total = sum(_sizes(case))
    out = 0 if case["out"] == "in place" else 4
    return {"bytes": total * (size + out), "flops": total * (3 if case["clips"] else 2)}


# --------------------------------------------------------------------------
# 64-bit values
# --------------------------------------------------------------------------
def _two_to(e):
    """2^e in 64 bits, from its bits: a library power may be off in the last place, which would move ties."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rounded(x):
    """4-bit values from the definition in 64 bits: the grid's spacing at each element, rounded half to even."""
    x = x.double()
    r, c = x.shape
    padded = torch.zeros((r, -(-c // 32) * 32), dtype=torch.float64, device=x.device)
    padded[:, :c] = x
    b = padded.view(r, -1, 32)
    top = b.abs().max(2, keepdim=True).values
    e = torch.frexp(torch.where(top.isfinite(), top, 0.0)).exponent - 1
    scale = _two_to(torch.where(top == 0, -127, (e - 2).clamp(min=-127)))
    v = b / scale
    spacing = _two_to((torch.frexp(v).exponent - 1).clamp(min=0) - 1)
    q = (torch.round(v / spacing) * spacing).clamp(-6, 6) * scale
    q = torch.where(top.isfinite(), q, torch.nan)
    return q.view(r, -1)[:, :c]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = [_exact_rounded(s["x"])]
        return out + [_exact_rounded(s["x"].t())] if case["both"] else out
    if op == "product":
        n, k = case["n"], case["k"]
        codes, scales = s["codes"].long(), s["scales"].long()
        column = torch.arange(k, device=DEV)
        row = torch.arange(n, device=DEV)[:, None]
        nibble = (codes[:, column // 2] >> (4 * (column % 2))) & 15
        block = column // 32
        byte = scales[row // 128, block // 4, row % 32 * 16 + row // 32 % 4 * 4 + block % 4]
        level = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)[nibble & 7]
        w = torch.where(nibble > 7, -level, level) * _two_to(byte - 127)
        return _exact_rounded(s["x"]) @ w.t()
    if op == "step":
        x, w, dy = s["x"], s["w"], s["dy"]
        return {"y": _exact_rounded(x) @ _exact_rounded(w).t(), "dx": _exact_rounded(dy) @ _exact_rounded(w.t()).t(),
                "dw": _exact_rounded(dy.t()) @ _exact_rounded(x.t()).t()}
    if op == "loss":
        rows, pairs, ends = s["logits"].shape[0], case["pairs"], s["offsets"].tolist()
        counted = (s["labels"] >= 0).tolist()
        label = s["labels"].tolist()
        lse = torch.cat([torch.logsumexp(s["logits"][i:i + 256].double(), 1) for i in range(0, rows, 256)])
        at = torch.tensor([max(v, 0) for v in label], device=DEV)
        keep = torch.tensor(counted, device=DEV)
        lp = (s["logits"].gather(1, at[:, None])[:, 0].double() - lse) * keep
        delta = (lp - s["ref"].double()) * keep
        r = torch.stack([delta[a:b].sum() for a, b in zip(ends, ends[1:])])
        h = s["beta"] * (r[:pairs] - r[pairs:])
        e = s["smoothing"]
        loss = -(1 - e) * torch.nn.functional.logsigmoid(h) - e * torch.nn.functional.logsigmoid(-h)
        out = {"losses": loss, "ratios": r, "logps": lp}
        if case["backward"]:
            slope = s["beta"] * (torch.sigmoid(h) - (1 - e)) * s["dlosses"].double()
            d = torch.empty(s["logits"].shape, dtype=torch.float64, device=DEV)
            for i, (a, b) in enumerate(zip(ends, ends[1:])):
                c = slope[i] if i < pairs else -slope[i - pairs]
                p = torch.exp(s["logits"][a:b].double() - lse[a:b, None])
                p[torch.arange(b - a, device=DEV), at[a:b]] -= 1
                d[a:b] = p * (-c * keep[a:b, None])
            out["dlogits"] = d
        return out
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]))
    factor = 1.0 if norm <= s["max_norm"] else s["max_norm"] / norm
    sizes = _sizes(case)
    flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device=DEV)
    for t, a, n in zip(s["grads"], _starts(sizes, 64), sizes):
        flat[a:a + n] = t.double() * factor
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": flat}
