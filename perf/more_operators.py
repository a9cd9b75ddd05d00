"""Cases of the operators that answer many users from one model: log
probabilities of given tokens with the entropy and the top alternatives of
their rows of logits, low-rank adapters of many requests beside a shared
projection, and the gradients of both.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, through
hash_table_cache_gb300.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the alternatives to the token just answered, one user: latency
        {"name": "one answer", "op": "logps", "rows": 1, "vocab": 131072, "top": 5, "type": "bf16", "backward": False},
        # a short episode over a small item vocabulary, learned from: latency of both directions
        {"name": "a short episode", "op": "logps", "rows": 24, "vocab": 1000, "top": 0, "type": "f32", "backward": True},
        # one decoding step of a busy server, with twenty alternatives each; rows of odd length
        {"name": "a step of answers", "op": "logps", "rows": 256, "vocab": 50257, "top": 20, "type": "bf16", "backward": False},
        # a policy gradient's batch with an entropy bonus
        {"name": "policy gradient", "op": "logps", "rows": 4096, "vocab": 32768, "top": 0, "type": "bf16", "backward": True},
        # scoring of whole answers over a large candidate vocabulary, the alternatives kept
        {"name": "scored answers", "op": "logps", "rows": 4096, "vocab": 131072, "top": 20, "type": "bf16", "backward": False},
        # one user's next token through an adapter: latency
        {"name": "one token", "op": "adapters", "requests": 1, "length": 1, "k": 4096, "n": 4096, "rank": 16, "adapters": 16, "type": "bf16", "backward": False},
        # one decoding step for many users who share a bank of adapters
        {"name": "a step of requests", "op": "adapters", "requests": 256, "length": 1, "k": 4096, "n": 4096, "rank": 16, "adapters": 64, "type": "bf16", "backward": False},
        # prompts of different lengths, packed
        {"name": "prompts", "op": "adapters", "requests": 24, "length": 341, "k": 4096, "n": 8192, "rank": 32, "adapters": 8, "type": "bf16", "backward": False},
        # adapted logits over candidate rows of 64 floats: the output is what it costs
        {"name": "candidate logits", "op": "adapters", "requests": 16, "length": 128, "k": 64, "n": 131072, "rank": 8, "adapters": 16, "type": "bf16", "backward": False},
        # a training step of a few adapters beside a frozen projection
        {"name": "training step", "op": "adapters", "requests": 32, "length": 257, "k": 4096, "n": 4096, "rank": 64, "adapters": 4, "type": "bf16", "backward": True},
        # every user's adapter a row of the table: short histories, 32 bits, learned online
        {"name": "rows as adapters", "op": "adapters", "requests": 333, "length": 12, "k": 128, "n": 128, "rank": 8, "adapters": 333, "type": "f32", "backward": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["f32", "bf16", "bf16", "f16"])
    size = 4 if kind == "f32" else 2
    backward = rng.random() < 0.5
    if rng.random() < 0.45:
        vocab = _log(rng, 50, 131072)
        rows = _log(rng, 1, min(16384, 2000000000 // (vocab * 2 * size)))
        top = 0 if rng.random() < 0.3 else rng.randint(1, 32)
        return {"op": "logps", "rows": rows, "vocab": vocab, "top": top, "type": kind, "backward": backward}
    k = _log(rng, 16, 8192)
    n = _log(rng, 16, 8192 if backward else 65536)
    rank = _log(rng, 1, 64)
    adapters = _log(rng, 1, min(256, 120000000 // (rank * (k + n))))
    requests = _log(rng, 1, 512)
    most = (60000000 if backward else 200000000) // (k + 2 * n) // requests
    # a decoding step has one token of each, a prompt's or an episode's length varies
    length = 1 if rng.random() < 0.25 else _log(rng, 1, min(2048, most))
    return {"op": "adapters", "requests": requests, "length": length, "k": k, "n": n, "rank": rank, "adapters": adapters,
            "type": kind, "backward": backward}


def _lengths(case):
    """Tokens of each request."""
    if case["length"] == 1:
        return [1] * case["requests"]
    rng = random.Random(case["requests"] * 7919 + case["length"])
    return [max(1, int(case["length"] * rng.uniform(0.3, 1.7))) for _ in range(case["requests"])]


def _which(case):
    """The adapter of each request: a row each where there are as many, else some are asked for more than
    others; a few requests of a large batch have none."""
    r, a = case["requests"], case["adapters"]
    if r == a:
        return list(range(r))
    rng = random.Random(r * 104729 + a)
    return [-1 if r > 8 and rng.random() < 0.06 else int(a * rng.random() ** 1.5) for _ in range(r)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _normal(g, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
    return x.mul_(scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    dtype = TYPES[case["type"]]
    if case["op"] == "logps":
        rows, vocab = case["rows"], case["vocab"]
        logits = _normal(g, (rows, vocab), dtype, 2.0)
        labels = torch.randint(vocab, (rows,), generator=g, device=DEV)
        # what was answered is likelier than most, more or less so from token to token
        logits[torch.arange(rows, device=DEV), labels] += (4 + 3 * torch.randn(rows, generator=g, device=DEV)).to(dtype)
        # a batch's prompts carry no label
        s["labels"] = torch.where(torch.rand(rows, generator=g, device=DEV) < (0.1 if rows > 8 else 0.0), -100, labels)
        s["logits"] = logits
        if case["backward"]:
            s["dlogps"] = torch.randn(rows, generator=g, device=DEV) / rows  # advantages
            s["dentropy"] = torch.full((rows,), -0.01 / rows, device=DEV)
            s["dlogits"] = torch.empty_like(logits)
        return s
    k, n, r, adapters = case["k"], case["n"], case["rank"], case["adapters"]
    lengths = torch.tensor(_lengths(case), device=DEV)
    tokens = sum(_lengths(case))
    s["offsets"] = torch.nn.functional.pad(lengths.cumsum(0), (1, 0))
    s["which"] = torch.tensor(_which(case), device=DEV)
    # where each token stands, and the padded batch that a user without such an operator would build
    at = torch.arange(tokens, device=DEV)
    s["seq"] = torch.bucketize(at, s["offsets"][1:], right=True)
    s["pos"] = at - s["offsets"][s["seq"]]
    place = torch.arange(max(_lengths(case)), device=DEV)
    s["inside"] = place < lengths[:, None]
    s["token"] = torch.where(s["inside"], s["offsets"][:-1, None] + place, 0)
    # hidden states: unit variance with a few columns that are several times larger
    x = _normal(g, (tokens, k), torch.float32)
    x *= 1 + 6 * (torch.rand(k, generator=g, device=DEV) < 0.02)
    s["x"] = x.to(dtype)
    # a row of the bank, as of a table, holds an adapter's two factors one after the other
    bank = torch.empty((adapters, r * (k + n)), dtype=dtype, device=DEV)
    s["down"] = bank[:, :r * k].view(adapters, r, k)
    s["up"] = bank[:, r * k:].view(adapters, n, r)
    s["down"].copy_(_normal(g, (adapters, r, k), dtype, k ** -0.5))
    s["up"].copy_(_normal(g, (adapters, n, r), dtype, 0.3 * r ** -0.5))
    s["scales"] = torch.rand(adapters, generator=g, device=DEV) + 0.5
    s["base"] = _normal(g, (tokens, n), dtype)  # the shared projection's
    s["y"] = torch.empty_like(s["base"])
    if case["backward"]:
        s["dy"] = _normal(g, (tokens, n), dtype, 0.01)
        s["dx_base"] = _normal(g, (tokens, k), dtype, 0.01)
        s["dx"] = torch.empty_like(s["dx_base"])
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_logps(s):
    dtype, top = s["logits"].dtype, s["top"]
    x = s["logits"].float()
    at = torch.arange(x.shape[0], device=x.device)
    counted = s["labels"] >= 0
    label = s["labels"].clamp_min(0)
    most = x.amax(1)
    shifted = x - most[:, None]
    e = shifted.exp()
    total = e.sum(1)
    logs = total.log()
    lse = most + logs
    entropy = logs - (e * shifted).sum(1) / total
    out = {"logps": torch.where(counted, x[at, label] - lse, 0.0), "entropy": torch.where(counted, entropy, 0.0)}
    if top:
        # one whole number for each entry, ordered by the logit and then by the lower index
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        order = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
        ids = 0xFFFFFFFF - (order.topk(top, 1).values & 0xFFFFFFFF)
        out["top_ids"] = torch.where(counted[:, None], ids, -1)
        out["top_logps"] = torch.where(counted[:, None], x.gather(1, ids) - lse[:, None], -torch.inf)
    if s["backward"]:
        lp = x - lse[:, None]
        d = lp.exp() * (-s["dlogps"][:, None] - s["dentropy"][:, None] * (lp + entropy[:, None]))
        d[at, label] += s["dlogps"]
        out["dlogits"] = torch.where(counted[:, None], d, 0.0).to(dtype)
    return out


def _plain_adapters(s):
    dtype = s["x"].dtype
    which = s["which"].clamp_min(0)
    scale = torch.where(s["which"] >= 0, s["scales"][which], 0.0)
    down, up = s["down"].float()[which], s["up"].float()[which]  # [requests, r, k] and [requests, n, r]
    inside = s["inside"][..., None]
    x = torch.where(inside, s["x"].float()[s["token"]], 0.0)  # [requests, longest, k]
    h = x @ down.transpose(1, 2)
    y = (h * scale[:, None, None]) @ up.transpose(1, 2)
    out = {"y": (s["base"].float() + y[s["seq"], s["pos"]]).to(dtype)}
    if s["backward"]:
        dy = torch.where(inside, s["dy"].float()[s["token"]], 0.0) * scale[:, None, None]
        dh = dy @ up
        out["dx"] = (s["dx_base"].float() + (dh @ down)[s["seq"], s["pos"]]).to(dtype)
        # an adapter's gradient is the sum of its requests'
        of = (s["which"] == torch.arange(s["adapters"], device=which.device)[:, None]).float()
        out["ddown"] = (of @ (dh.transpose(1, 2) @ x).flatten(1)).view(s["down"].shape).to(dtype)
        out["dup"] = (of @ (dy.transpose(1, 2) @ h).flatten(1)).view(s["up"].shape).to(dtype)
    return out


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------
def _own(s):
    import hash_table_cache_gb300 as hkv
    if s["op"] == "logps":
        f = hkv.token_logps(s["logits"], s["labels"], top=s["top"])
        out = {"logps": f.logps, "entropy": f.entropy}
        if s["top"]:
            out |= {"top_ids": f.top_ids, "top_logps": f.top_logps}
        if s["backward"]:
            out["dlogits"] = hkv.token_logps_backward(f, s["dlogps"], s["dentropy"], out=s["dlogits"])
        return out
    f = hkv.adapter_matmul(s["x"], s["down"], s["up"], s["offsets"], s["which"], s["scales"], base=s["base"], out=s["y"])
    out = {"y": f.out}
    if s["backward"]:
        out["dx"], out["ddown"], out["dup"] = hkv.adapter_matmul_backward(f, s["dy"], base=s["dx_base"], out=s["dx"])
    return out


def run(state):
    if own:
        return _own(state)
    return _plain_logps(state) if state["op"] == "logps" else _plain_adapters(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "logps":
        rows, vocab = case["rows"], case["vocab"]
        b = case["backward"]
        return {"bytes": rows * (vocab * size * (2 if b else 1) + 16 + 12 * case["top"]), "flops": rows * vocab * (11 if b else 5)}
    k, n, r = case["k"], case["n"], case["rank"]
    tokens = sum(_lengths(case))
    held = r * (k + n)
    used = len({a for a in _which(case) if a >= 0})
    if case["backward"]:
        return {"bytes": size * (3 * tokens * (k + n) + (used + case["adapters"]) * held), "flops": 6 * tokens * held}
    return {"bytes": size * (tokens * (k + 2 * n) + used * held), "flops": 2 * tokens * held}


# --------------------------------------------------------------------------
# 64-bit values
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    out = {}
    if case["op"] == "logps":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        keep = s["labels"] >= 0
        label = torch.where(keep, s["labels"], 0)
        parts = {"logps": [], "entropy": [], "top_ids": [], "top_logps": [], "dlogits": []}
        step = max(1, 1 << 26 >> max(0, (vocab - 1).bit_length()))
        for i in range(0, rows, step):
            lp = torch.log_softmax(s["logits"][i:i + step].double(), 1)
            k, at = keep[i:i + step], label[i:i + step, None]
            p = lp.exp()
            h = -torch.special.xlogy(p, p).sum(1)
            parts["logps"].append(torch.where(k, lp.gather(1, at)[:, 0], 0.0))
            parts["entropy"].append(torch.where(k, h, 0.0))
            if top:
                v, ids = torch.sort(s["logits"][i:i + step].double(), dim=1, descending=True, stable=True)
                ids = ids[:, :top]
                parts["top_ids"].append(torch.where(k[:, None], ids, -1))
                parts["top_logps"].append(torch.where(k[:, None], lp.gather(1, ids), -torch.inf))
                del v
            if case["backward"]:
                g, b = s["dlogps"][i:i + step, None].double(), s["dentropy"][i:i + step, None].double()
                d = -p * (g + b * (lp + h[:, None]))
                d.scatter_add_(1, at, g)
                parts["dlogits"].append(torch.where(k[:, None], d, 0.0))
        return {name: torch.cat(v) for name, v in parts.items() if v}
    x, base = s["x"], s["base"]
    out["y"] = base.double()
    if case["backward"]:
        out["dx"] = s["dx_base"].double()
        out["ddown"] = torch.zeros(s["down"].shape, dtype=torch.float64, device=DEV)
        out["dup"] = torch.zeros(s["up"].shape, dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    for a, b, w in zip(ends, ends[1:], _which(case)):
        if w < 0:
            continue
        c, d, u = float(s["scales"][w]), s["down"][w].double(), s["up"][w].double()
        xs = x[a:b].double()
        h = torch.einsum("tk,rk->tr", xs, d)
        out["y"][a:b] += c * torch.einsum("tr,nr->tn", h, u)
        if case["backward"]:
            dy = c * s["dy"][a:b].double()
            dh = torch.einsum("tn,nr->tr", dy, u)
            out["dx"][a:b] += torch.einsum("tr,rk->tk", dh, d)
            out["ddown"][w] += torch.einsum("tr,tk->rk", dh, xs)
            out["dup"][w] += torch.einsum("tn,tr->nr", dy, h)
    return out
