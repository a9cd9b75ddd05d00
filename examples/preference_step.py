"""Online learning from preferences, on the rows of a table.

A table holds one embedding row per item.  Users prefer one sequence of items
over another; each step looks the candidates' rows up, scores hidden states
against them in 4 bits, takes the preference loss and its gradient, clips the
gradients of the tower's weight and of the rows to one norm, and writes the
rows back:

    find -> mx_quantize -> mx_matmul -> preference_loss -> backward
         -> mx_matmul on the copies along the other axis -> clip_grad_norm -> assign

    python examples/preference_step.py --steps 30
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


def train(steps=30, items=4096, dim=64, inputs=128, pairs=16, length=24, beta=0.2, lr=1.0, max_norm=0.2,
          seed=0, device="cuda"):
    """Returns (losses by step, gradient norms by step, rows before, rows after)."""
    dev = torch.device(device, torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # the items' rows live in the table
    keys = torch.from_numpy(wl.as_i64(wl.unique_keys(seed + 1, items))).to(dev)
    table = hkv.HashTable(-(-2 * items // 128) * 128, dim, device=dev.index)
    table.insert_or_assign(keys, randn(items, dim) / dim ** 0.5, torch.ones_like(keys))
    weight = randn(dim, inputs) / inputs ** 0.5

    # a batch of pairs: token t saw inputs x[t] and was followed by item labels[t]
    tokens = 2 * pairs * length
    offsets = torch.arange(2 * pairs + 1, device=dev) * length
    x = randn(tokens, inputs).to(torch.bfloat16)
    labels = torch.randint(items, (tokens,), generator=g, device=dev)
    ref = None  # the first step's policy is the reference
    losses, norms = [], []
    before = table.find(keys)[0].clone()
    for _ in range(steps):
        rows, found, _ = table.find(keys)
        assert bool(found.all()), "every candidate is resident"
        # forward: hidden states, logits over the candidates
        qx, qxt = hkv.mx_quantize(x, "both")
        hidden = hkv.mx_matmul(qx, hkv.mx_quantize(weight), dtype=torch.bfloat16)
        qh, qht = hkv.mx_quantize(hidden, "both")
        qrows, qrowst = hkv.mx_quantize(rows, "both")
        logits = hkv.mx_matmul(qh, qrows, dtype=torch.bfloat16)
        if ref is None:
            ref = hkv.preference_loss(logits, labels, offsets).logps.clone()
        loss = hkv.preference_loss(logits, labels, offsets, ref, beta=beta)
        losses.append(loss.losses.mean())
        # backward: the logits' gradient takes the logits' place
        share = torch.full((pairs,), 1.0 / pairs, device=dev)
        dlogits = hkv.preference_loss_backward(loss, share, out=logits)
        qd, qdt = hkv.mx_quantize(dlogits, "both")
        drows = hkv.mx_matmul(qdt, qht, dtype=torch.float32)
        dhidden = hkv.mx_matmul(qd, qrowst, dtype=torch.bfloat16)
        dweight = hkv.mx_matmul(hkv.mx_quantize(dhidden, "columns"), qxt, dtype=torch.float32)
        norms.append(hkv.clip_grad_norm([dweight, drows], max_norm))
        # update, and the rows' write-back
        weight -= lr * dweight
        table.assign(keys, rows - lr * drows, None)
    after = table.find(keys)[0].clone()
    table.close()
    return [float(v) for v in losses], [float(v) for v in norms], before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--items", type=int, default=4096)
    ap.add_argument("--dim", type=int, default=64)
    a = ap.parse_args()
    losses, norms, _, _ = train(a.steps, a.items, a.dim)
    for i, (v, n) in enumerate(zip(losses, norms)):
        print(f"step {i:3d}  loss {v:.4f}  gradient norm {n:.4f}")
