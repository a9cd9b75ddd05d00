"""The preference loss where entries of the vocabulary are banned by a finite
number, each row held to a bound of its own (tests/preference_bounds.py)."""
import pytest
import torch

from tests import preference_bounds as bounds

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    return m


def _logits(rows, vocab, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (2 * torch.randn((rows, vocab), generator=g, device=DEV)).to(dtype)
    return x, torch.randint(vocab, (rows,), generator=g, device=DEV)


def _check_logps(hkv, x, labels):
    """Every row counted, in a sequence of its own."""
    rows = x.shape[0]
    f = hkv.preference_loss(x, labels, torch.arange(rows + 1, device=DEV))
    lp, bound, _, _ = bounds.tokens(x, labels)
    over = (f.logps.double() - lp).abs() - bound
    assert f.logps.isfinite().all(), f"{int((~f.logps.isfinite()).sum())} of {rows} rows are not finite"
    assert float(over.max()) <= 0, f"row {int(over.argmax())}: {float(over.max()):.3g} over its bound"
    assert f.losses.isfinite().all() and f.ratios.isfinite().all()
    return f


MASKS = [-1e3, -1e4, -1e5, -1e6, -2e6, -1e8, -2e9, -1e10, -1e20, -1e30, -1e36, -1e37, -3e38]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab,first", [(64, 63), (1000, 900), (4096, 2048), (20000, 16384), (131072, 65536),
                                         (131072, 131071)])
def test_logps_beside_finite_masks(hkv, dtype, vocab, first):
    """Masks over a whole first round of every thread, over all entries but the
    label, over one part of a row that blocks share."""
    x, labels = _logits(2 * len(MASKS), vocab, dtype, vocab + first)
    for i, low in enumerate(MASKS):
        x[2 * i, :first] = low          # the first entries
        x[2 * i + 1, vocab - first:] = low  # the last
        labels[2 * i] = vocab - 1
        labels[2 * i + 1] = 0
    _check_logps(hkv, x, labels)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [1, 7, 64, 1000, 40000])
def test_logps_of_rows_that_are_all_mask(hkv, dtype, vocab):
    """A row whose mask leaves nothing has the log probability -log(vocab)."""
    low = [v for v in MASKS if dtype != F16 or v > -65504] + [torch.finfo(dtype).min]
    x, labels = _logits(2 * (len(low) // 2 + 1), vocab, dtype, vocab)
    for i, v in enumerate(low):
        x[i] = v
    _check_logps(hkv, x, labels)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logps_of_large_logits(hkv, dtype):
    """Rows of large numbers of either sign that are not masks."""
    x, labels = _logits(24, 3000, dtype, 5)
    for i, v in enumerate([1e4, -1e5, 1e6, -2e6, 1e7, 1e9, -3e9, 1e10, 1e20, -1e30, 1e36, 3e38]):
        x[2 * i] = x[2 * i] * (abs(v) / 16)
        x[2 * i + 1] = v
    _check_logps(hkv, x, labels)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_beside_finite_masks(hkv, dtype):
    x, labels = _logits(2 * len(MASKS), 5000, dtype, 9)
    at = torch.arange(2 * len(MASKS), device=DEV)
    for i, low in enumerate(MASKS):
        x[2 * i, :4096] = low
        x[2 * i + 1, torch.arange(5000, device=DEV) != labels[2 * i + 1]] = low
        labels[2 * i] = 4500
    f = _check_logps(hkv, x, labels)
    d = hkv.preference_loss_backward(f).double()
    _, _, p, e = bounds.tokens(x, labels)
    h = 0.1 * (f.ratios[:len(MASKS)] - f.ratios[len(MASKS):]).double()
    slope = -0.1 * torch.sigmoid(-h)
    g = torch.cat((slope, -slope))[:, None]
    hot = torch.zeros_like(p)
    hot[at, labels] = 1
    want = g * (hot - p)
    u = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[dtype]
    bound = g.abs() * (e + (hot - p).abs() * 2.0 ** -20 + 2.0 ** -23 * hot) * (1 + u) + want.abs() * u + 2.0 ** -132
    over = (d - want).abs() - bound
    assert float(over.max()) <= 0, f"row {int(over.amax(1).argmax())}: {float(over.max()):.3g} over its bound"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [1, 7, 64, 1001, 40000])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_of_rows_that_are_all_mask(hkv, dtype, vocab, in_place):
    """A counted row whose mask leaves nothing, or whose logits are all large,
    has a softmax that adds up to 1; rows beside it stay as they are."""
    low = [v for v in MASKS if dtype != F16 or v > -65504] + [torch.finfo(dtype).min, 3e4]
    rows = 2 * len(low)
    x, labels = _logits(rows, vocab, dtype, vocab)
    for i, v in enumerate(low):
        x[2 * i] = v
        x[2 * i, vocab // 2:] += torch.tensor(0.75, device=DEV).to(dtype)
    pairs = rows // 2
    f = hkv.preference_loss(x, labels, torch.arange(rows + 1, device=DEV))
    lp, _, p, e = bounds.tokens(x, labels)
    h = 0.1 * (f.ratios[:pairs] - f.ratios[pairs:]).double()
    slope = -0.1 * torch.sigmoid(-h)
    g = torch.cat((slope, -slope))[:, None]
    hot = torch.zeros_like(p)
    hot[torch.arange(rows, device=DEV), labels] = 1
    want = g * (hot - p)
    u = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -132
    bound = g.abs() * (e + (hot - p).abs() * 2.0 ** -20 + 2.0 ** -23 * hot) * (1 + u) + want.abs() * u + tiny
    d = hkv.preference_loss_backward(f, out=x if in_place else None).double()
    over = (d - want).abs() - bound
    assert float(over.max()) <= 0, f"row {int(over.amax(1).argmax())}: {float(over.max()):.3g} over its bound"
