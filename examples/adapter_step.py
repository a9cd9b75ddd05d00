"""Online learning from rewards, with an adapter for every user in a table.

All users share one projection from hidden states to items' logits, held in 4
bits.  Each user's low-rank adapter of it is a row of a table, found by the user's
key.  A step answers some users, takes the log probabilities of what was answered
(with the likeliest alternatives), learns from the rewards by a policy gradient
with an entropy bonus, and writes the adapters back:

    find -> mx_quantize -> mx_matmul -> adapter_matmul -> token_logps
         -> token_logps_backward -> adapter_matmul_backward -> clip_grad_norm -> assign

    python examples/adapter_step.py --steps 30
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import hash_table_cache_gb300 as hkv  # noqa: E402
import workloads as wl  # noqa: E402


def split(rows, rank, k, n):
    """The two factors of the adapters that rows of a table hold, as views."""
    return rows[:, :rank * k].unflatten(1, (rank, k)), rows[:, rank * k:].unflatten(1, (n, rank))


def step(table, users, x, offsets, labels, advantages, weight, rank, bonus=0.01, max_norm=1.0, lr=0.5, top=3):
    """One step of the requests of `users` (each once: an adapter is written back by its
    request); returns what it has computed."""
    tokens, k = x.shape
    n = weight.rows
    rows, found, _ = table.find(users)
    assert bool(found.all()), "every user is resident"
    down, up = split(rows, rank, k, n)
    which = torch.arange(users.numel(), device=x.device)
    # forward: the shared logits, each user's adapter onto them
    shared = hkv.mx_matmul(hkv.mx_quantize(x), weight, dtype=torch.float32)
    f = hkv.adapter_matmul(x, down, up, offsets, which, base=shared)
    g = hkv.token_logps(f.out, labels, top=top)
    # backward of mean(-advantage * logp - bonus * entropy)
    dlogits = hkv.token_logps_backward(g, -advantages / tokens, torch.full_like(advantages, -bonus / tokens))
    _, ddown, dup = hkv.adapter_matmul_backward(f, dlogits)
    grads = torch.cat((ddown.flatten(1), dup.flatten(1)), 1)
    norm = hkv.clip_grad_norm(grads, max_norm)
    table.assign(users, rows - lr * grads, None)
    return {"rows": rows, "shared": shared, "logits": f.out, "logps": g.logps, "entropy": g.entropy,
            "top_ids": g.top_ids, "dlogits": dlogits, "ddown": ddown, "dup": dup, "norm": norm, "clipped": grads}


def train(steps=30, users=200, items=500, k=64, rank=4, batch=24, length=10, seed=0, device="cuda"):
    """Yields each step's result and its inputs; a user is rewarded for items of a
    kind of its own."""
    dev = torch.device(device, torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    dim = rank * (k + items)
    keys = torch.from_numpy(wl.as_i64(wl.unique_keys(seed + 1, users))).to(dev)
    table = hkv.HashTable(-(-2 * users // 128) * 128, dim, device=dev.index)
    rows = randn(users, dim) / k ** 0.5
    rows[:, rank * k:] = 0  # an adapter starts as none
    table.insert_or_assign(keys, rows, torch.ones_like(keys))
    weight = hkv.mx_quantize(randn(items, k) / k ** 0.5)
    try:
        for _ in range(steps):
            who = torch.randperm(users, generator=g, device=dev)[:batch]
            lengths = torch.randint(1, 2 * length, (batch,), generator=g, device=dev)
            offsets = torch.nn.functional.pad(lengths.cumsum(0), (1, 0))
            tokens = int(offsets[-1])
            x = randn(tokens, k)
            labels = torch.randint(items, (tokens,), generator=g, device=dev)
            liked = labels % 8 == torch.repeat_interleave(who % 8, lengths)
            advantages = torch.where(liked, 1.0, -1.0 / 7)
            yield {"x": x, "offsets": offsets, "labels": labels, "advantages": advantages} | step(
                table, keys[who], x, offsets, labels, advantages, weight, rank)
    finally:
        table.close()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--users", type=int, default=200)
    ap.add_argument("--rank", type=int, default=4)
    a = ap.parse_args()
    for i, s in enumerate(train(a.steps, a.users, rank=a.rank)):
        loss = -(s["advantages"] * s["logps"]).mean()
        print(f"step {i:3d}  loss {float(loss):8.4f}  entropy {float(s['entropy'].mean()):.4f}  "
              f"gradient norm {float(s['norm']):.4f}")
