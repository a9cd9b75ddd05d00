"""The example that runs the table and the operators together: the loss starts
at log 2 (the policy is its own reference), falls, and the rows in the table
have changed."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_preference_step_learns():
    from hash_table_cache_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("preference_step",
                                                  os.path.join(ROOT, "examples", "preference_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, norms, before, after = m.train(steps=30, items=1000, dim=40, inputs=70, pairs=6, length=9)
    assert abs(losses[0] - math.log(2)) < 1e-6
    assert losses[-1] < 0.8 * losses[0], losses
    assert all(math.isfinite(n) and n > 0 for n in norms)
    assert after.isfinite().all() and not torch.equal(before, after)
