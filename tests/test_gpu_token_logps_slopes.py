"""The gradient of token_logps for large dlogps and dentropy, on rows with masked
entries: whatever the mask, an entry whose probability is 0 has a gradient of 0."""
import math

import pytest
import torch

from tests.operators_plain import near
from tests.token_logps_plain import token_logps as plain

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    return m


@pytest.mark.parametrize("size", [1e9, 1e29, 1e37])
@pytest.mark.parametrize("mask", [-math.inf, "lowest", -1e30, -1e5])
@pytest.mark.parametrize("rows,vocab", [(6, 50), (6, 3000), (6, 40000), (5000, 3000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_slopes(hkv, rows, vocab, dtype, mask, size):
    """By warps, by blocks and by clusters' rows; a gradient that lies as the logits do and
    one that does not; one row far from 0."""
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.randn((rows, vocab), generator=g, device=DEV) * 2
    x[3] += 30000
    x[torch.rand((rows, vocab), generator=g, device=DEV) < 0.5] = torch.finfo(dtype).min if mask == "lowest" else mask
    buf = torch.zeros(rows * vocab + 1, dtype=dtype, device=DEV)
    labels = torch.randint(vocab, (rows,), generator=g, device=DEV)
    labels[1] = -100
    sign = torch.tensor([1.0, -1.0], device=DEV).repeat(rows)[:rows]
    slopes = torch.rand(rows, generator=g, device=DEV) * sign * size
    other = torch.randn(rows, generator=g, device=DEV)
    for dlogps, dentropy in ((other, slopes), (slopes, other)):
        for at in (0, 1):
            y = buf[at:at + rows * vocab].view(rows, vocab).copy_(x)
            want = plain(y, labels, 0, dlogps, dentropy)["grad"]
            near(hkv.token_logps_backward(hkv.token_logps(y, labels), dlogps, dentropy), *want, "gradient")
