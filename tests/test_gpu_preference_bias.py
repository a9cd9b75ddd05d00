"""What leans one way in a token's log probability: a sequence adds its tokens
up, so the mean error over many tokens counts, not only the largest."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    return m


def _rows(tokens, vocab, dtype, scale, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (scale * torch.randn((tokens, vocab), generator=g, device=DEV)).to(dtype)
    return x, torch.randint(vocab, (tokens,), generator=g, device=DEV)


def _logps(hkv, x, labels):
    return hkv.preference_loss(x, labels, torch.tensor([0, x.shape[0], x.shape[0]], device=DEV)).logps


@pytest.mark.parametrize("dtype", TYPES)
def test_a_vocabulary_of_one(hkv, dtype):
    x, labels = _rows(1000, 1, dtype, 5.0, 1)
    assert (_logps(hkv, x, labels) == 0).all()


@pytest.mark.parametrize("vocab", [2, 3, 7])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_certain_tokens_of_short_rows(hkv, vocab, dtype):
    """The other entries add less than 2^-40 to the sum, which is 1."""
    x, labels = _rows(1000, vocab, dtype, 2.0, vocab)
    x[torch.arange(1000, device=DEV), labels] = 45.0
    assert (_logps(hkv, x, labels) == 0).all()


@pytest.mark.parametrize("vocab", [8, 1000, 20000, 131072])
@pytest.mark.parametrize("dtype", TYPES)
def test_certain_tokens(hkv, vocab, dtype):
    """The sum is 1 but for one approximate exponential near 2^0 and one rounding:
    at most 2^-22 for a token, half a unit (2^-25) on average."""
    tokens = min(8192, 2 ** 28 // vocab)
    x, labels = _rows(tokens, vocab, dtype, 2.0, vocab)
    x[torch.arange(tokens, device=DEV), labels] += 50.0
    lp = _logps(hkv, x, labels).double()
    assert float(lp.abs().max()) <= 2.0 ** -22
    assert float(lp.mean().abs()) <= 2.0 ** -25 + 5 * float(lp.std()) / tokens ** 0.5


@pytest.mark.parametrize("scale", [0.1, 2.0, 8.0])
@pytest.mark.parametrize("vocab", [2, 50, 1000, 8192, 32768, 131072])
@pytest.mark.parametrize("dtype", TYPES)
def test_mean_error(hkv, vocab, scale, dtype):
    """Below three quarters of 2^-24 a token, and five deviations of the mean.
    (log2 e in one float alone would lean by twice that.)"""
    tokens = min(16384, 2 ** 28 // vocab)
    x, labels = _rows(tokens, vocab, dtype, scale, vocab)
    got = _logps(hkv, x, labels).double()
    want = torch.cat([x[i:i + 2048].double().log_softmax(1).gather(1, labels[i:i + 2048, None])[:, 0]
                      for i in range(0, tokens, 2048)])
    off = got - want
    assert float(off.mean().abs()) <= 0.75 * 2.0 ** -24 + 5 * float(off.std()) / tokens ** 0.5
