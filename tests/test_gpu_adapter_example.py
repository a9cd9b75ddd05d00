"""The example that runs the table, the adapters and the token log probabilities
together: it runs, its gradients are those of the formulas, and the table has what
the last step wrote."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from hash_table_cache_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("adapter_step", os.path.join(ROOT, "examples", "adapter_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("rank,k,items", [(4, 64, 500), (8, 128, 384), (3, 70, 111)])
def test_a_step_s_gradients(example, rank, k, items):
    """Against automatic differentiation in 64 bits from the shared logits on.  The
    logits are off by e1, below (k + rank) / 16 + 256 roundings of 2^-23 of their
    terms' size (at most 8 here with the first product's); log p by as much and 2^-19
    more (tests/token_logps_plain.py, logits below 16); a gradient's sums by the same
    relative to the terms' sizes: 2^-14 of the largest entry holds all of it."""
    for n, s in enumerate(example.train(steps=3, users=40, items=items, k=k, rank=rank, batch=9)):
        rows = s["rows"].double().requires_grad_()
        down, up = example.split(rows, rank, k, items)
        x, ends = s["x"].double(), s["offsets"].tolist()
        logits = s["shared"].double() + torch.cat(
            [x[a:b] @ down[i].t() @ up[i].t() for i, (a, b) in enumerate(zip(ends, ends[1:]))])
        assert s["logits"].double().sub(logits).abs().max() <= 2.0 ** -14 * logits.abs().max()
        lp = torch.log_softmax(logits, 1)
        logps = lp[torch.arange(len(x), device=x.device), s["labels"]]
        entropy = -(lp.exp() * lp).sum(1)
        loss = (-s["advantages"].double() * logps - 0.01 * entropy).mean()
        want, = torch.autograd.grad(loss, rows)
        # (the table's row of a user was read before the step wrote it)
        clipped = s["clipped"].double()
        norm = want.norm()
        assert abs(float(s["norm"]) - float(norm)) <= 2.0 ** -14 * float(norm)
        want = want * (1.0 / norm).clamp_max(1.0)
        assert (clipped - want).abs().max() <= 2.0 ** -14 * want.abs().max(), n
        assert torch.equal(s["top_ids"], torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :3])


def test_steps_follow_one_another(example):
    """A user's row in a later step is the one that the step before has written."""
    seen = {}
    for s in example.train(steps=6, users=12, items=130, k=32, rank=2, batch=12):
        order = s["rows"][:, 0].argsort()  # all users each step, in another order: told apart by their first number
        now = s["rows"][order]
        if seen:
            have = {tuple(r[:4].tolist()) for r in seen["written"]}
            assert {tuple(r[:4].tolist()) for r in now} == have
        seen["written"] = s["rows"] - 0.5 * s["clipped"]
        assert s["rows"].isfinite().all()
