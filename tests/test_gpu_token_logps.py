"""token_logps and its gradient against their 64-bit forms
(tests/token_logps_plain.py), at the lengths, strides, masks and ties where they
can go wrong."""
import math

import pytest
import torch

from tests.operators_plain import near
from tests.token_logps_plain import token_logps as plain

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


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(seed, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * scale).to(dtype)


def _strided(x, extra, shift):
    rows, cols = x.shape
    buf = torch.full((shift + rows * (cols + extra),), float("nan"), dtype=x.dtype, device=x.device)
    view = buf[shift:].view(rows, cols + extra)[:, :cols]
    view.copy_(x)
    return view


def _labels(seed, rows, vocab):
    """Some tokens without one, on either side of the vocabulary."""
    labels = torch.randint(vocab, (rows,), generator=_gen(seed), device=DEV)
    if rows > 2:
        labels[1::5] = -100
        labels[2::7] = vocab
    return labels


def _check(hkv, x, labels, top, backward=True, out=None, seed=0):
    rows = x.shape[0]
    g = _randn(seed + 50, (rows,)) if labels is not None and backward else None
    h = _randn(seed + 51, (rows,)) if backward else None
    want = plain(x, labels, top, g, h)
    f = hkv.token_logps(x, labels, top)
    near(f.entropy, *want["entropy"], "entropy")
    if labels is None:
        assert f.logps is None
    else:
        near(f.logps, *want["logps"], "logps")
    if top:
        assert torch.equal(f.top_ids, want["top_ids"]), "top_ids"
        near(f.top_logps, *want["top_logps"], "top_logps")
    else:
        assert f.top_ids is None and f.top_logps is None
    if backward:
        got = hkv.token_logps_backward(f, g, h, out=out)
        assert out is None or got is out
        near(got, *want["grad"], "gradient")
    return f


@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (2, 31), (9, 33), (70, 257), (4, 1000), (3, 1024),
                                        (2, 2049), (33, 4097), (600, 1000), (5, 8193), (3, 16384), (9, 50257),
                                        (1, 131072), (200, 20000), (2, 300001)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_rows(hkv, rows, vocab, dtype, top):
    x = _randn(rows + vocab, (rows, vocab), dtype, 3.0)
    _check(hkv, x, _labels(vocab, rows, vocab), min(top, vocab), backward=top == 5)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_short_rows(hkv, dtype):
    """More than a warp for each SM's lanes: rows of 8 KB by warps."""
    x = _randn(4, (6000, 2003), dtype, 2.0)
    _check(hkv, x, _labels(1, 6000, 2003), 20)


@pytest.mark.parametrize("rows,vocab", [(7, 300), (5, 9001)])
@pytest.mark.parametrize("extra,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (5, 0), (8, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows(hkv, rows, vocab, extra, shift, dtype):
    x = _strided(_randn(1, (rows, vocab), dtype, 2.0), extra, shift)
    labels = _labels(2, rows, vocab)
    _check(hkv, x, labels, 20)  # into a contiguous gradient, which lies differently
    for other_extra, other_shift in ((extra, shift), (2, 3)):
        out = _strided(torch.zeros((rows, vocab), dtype=dtype, device=DEV), other_extra, other_shift)
        _check(hkv, x, labels, 3, out=out)
        whole = torch.empty(0, dtype=dtype, device=DEV).set_(out.untyped_storage())
        assert int(whole.isnan().sum()) == other_shift + other_extra * rows, "elements between the rows were written"


@pytest.mark.parametrize("vocab", [50, 3000, 40000])
@pytest.mark.parametrize("dtype", TYPES)
def test_without_labels(hkv, vocab, dtype):
    x = _randn(3, (6, vocab), dtype, 2.0)
    _check(hkv, x, None, 7)
    f = hkv.token_logps(x)
    with pytest.raises(ValueError):
        hkv.token_logps_backward(f, torch.ones(6, device=DEV))


@pytest.mark.parametrize("vocab", [40, 1500, 9000, 70000])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [1, 20, 32])
def test_ties_go_to_the_lower_index(hkv, vocab, dtype, top):
    """Few different values, one value, zeros of both signs, values that repeat
    every 256 entries, rows in order."""
    x = torch.randint(-3, 4, (8, vocab), generator=_gen(9), device=DEV).to(dtype)
    x[1] = 2.5
    x[2] = 0.0
    x[2, ::3] = -0.0
    x[3] = (torch.arange(vocab, device=DEV) % 256 < 8).to(dtype)
    x[4] = torch.arange(vocab, device=DEV).to(dtype) / vocab
    x[5] = -torch.arange(vocab, device=DEV).to(dtype) / vocab
    x[6] = 0.0
    x[6, vocab // 2:] = 1.0
    _check(hkv, x, None, top, backward=False)


@pytest.mark.parametrize("vocab", [64, 1200, 33000])
@pytest.mark.parametrize("dtype", TYPES)
def test_masks(hkv, vocab, dtype):
    """-inf and finite masks that leave all, a few, one or no entries; a label that
    is banned; NaN and infinities in rows that are not counted and in ones that are."""
    low = torch.finfo(dtype).min
    x = _randn(6, (16, vocab), dtype, 2.0)
    labels = torch.randint(vocab, (16,), generator=_gen(7), device=DEV)
    for r, mask in ((0, -math.inf), (1, low), (2, max(low, -1e10)), (3, -3e4)):
        keep = x[r, 5:14].clone()
        x[r] = mask
        x[r, 5:14] = keep
        labels[r] = 7
    x[4], x[4, vocab - 1] = -math.inf, 1.5
    labels[4] = vocab - 1
    x[5] = -math.inf
    x[6] = low
    x[7] = max(low, -1e10)
    x[8], x[8, 3] = low, -math.inf
    labels[9] = 20
    x[9, 20] = -math.inf
    x[10, 9] = math.nan
    x[11, 9] = math.inf
    x[12, 9], labels[12] = math.nan, -1
    x[13], labels[13] = math.inf, vocab
    x[14] = -torch.finfo(dtype).min  # the largest, everywhere
    x[15, ::2] = -math.inf
    _check(hkv, x, labels, 20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [90, 5000, 80000])
def test_far_and_certain_rows(hkv, dtype, vocab):
    """Large logits of either sign, and rows with one entry that is all."""
    x = _randn(8, (8, vocab), dtype, 1.0)
    x[0] += 1000
    x[1] -= 2000
    x[2] += 20000
    x[3] -= 30000
    x[4, 17] = 100
    x[5, 17] = 30
    x[6, 17] = 60000
    _check(hkv, x, torch.full((8,), 17, device=DEV), 5)


@pytest.mark.parametrize("vocab", [700, 30000])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_in_place(hkv, vocab, dtype):
    x = _randn(1, (9, vocab), dtype, 2.0)
    labels = _labels(3, 9, vocab)
    g, h = _randn(5, (9,)), _randn(6, (9,))
    f = hkv.token_logps(x, labels)
    want = hkv.token_logps_backward(f, g, h)
    for a, b in ((g, None), (None, h)):
        near(hkv.token_logps_backward(f, a, b), *plain(x, labels, 0, a, b)["grad"])
    assert not hkv.token_logps_backward(f).any()
    version = x._version
    assert hkv.token_logps_backward(f, g, h, out=x) is x
    assert torch.equal(x, want) and x._version > version


def test_gradient_against_differences(hkv):
    """L = sum dlogps logps + dentropy entropy along v, |v| <= 1: the difference
    quotient of step s is off by the values' bounds over s, and by s^2 / 6 times the
    third derivative: at most 8 for a log p (a third central moment of v) and
    8 (3 + max |log p|) for the entropy, a mean of log p."""
    rows, vocab, s = 12, 300, 2.0 ** -6
    x = _randn(1, (rows, vocab), F32, 1.5)
    v = torch.rand((rows, vocab), generator=_gen(2), device=DEV) * 2 - 1
    # steps that are exact: the values are multiples of 2^-10
    x, v = (x * 1024).round() / 1024, (v * 16).round() / 16
    labels = torch.randint(vocab, (rows,), generator=_gen(3), device=DEV)
    g, h = _randn(4, (rows,)), _randn(5, (rows,))
    f = hkv.token_logps(x, labels)
    d = hkv.token_logps_backward(f, g, h)
    got = (d.double() * v.double()).sum(1)
    up, down = (hkv.token_logps(x + k * s * v, labels) for k in (1, -1))
    diff = (g.double() * (up.logps.double() - down.logps.double())
            + h.double() * (up.entropy.double() - down.entropy.double())) / (2 * s)
    want = plain(x, labels, 0, g, h)
    e = (g.abs() * want["logps"][1] + h.abs() * want["entropy"][1]) / s
    most = -torch.log_softmax(x.double(), 1).amin(1)
    e = e + s * s / 6 * (8 * g.abs() + 8 * (3 + most) * h.abs()) + want["grad"][1].sum(1)
    assert bool(((got - diff).abs() <= e).all()), ((got - diff).abs() / e).max()


def test_rows_past_32_bit_offsets(hkv):
    """Rows 2^30 elements apart: the last starts 2^31 elements in."""
    buf = torch.zeros(2 * 2 ** 30 + 5000, dtype=BF16, device=DEV)
    x = buf.as_strided((3, 5000), (2 ** 30, 1))
    x.copy_(_randn(8, (3, 5000), BF16, 2.0))
    _check(hkv, x, torch.tensor([4, 4999, 17], device=DEV), 20)


def test_a_long_vocabulary(hkv):
    """Ids past 2^24, which a float does not hold."""
    vocab = 20_000_003
    x = _randn(3, (2, vocab), BF16, 1.0)
    x[0, vocab - 2] = x[0, vocab - 1] = 30.0
    _check(hkv, x, torch.tensor([vocab - 1, 5], device=DEV), 9)


def test_no_rows(hkv):
    x = torch.empty((0, 50), device=DEV)
    f = hkv.token_logps(x, torch.empty(0, dtype=torch.int64, device=DEV), top=3)
    assert f.logps.shape == f.entropy.shape == (0,) and f.top_ids.shape == (0, 3)
    assert hkv.token_logps_backward(f).shape == (0, 50)


@pytest.mark.parametrize("rows,vocab", [(3, 100000), (400, 9000), (5000, 700)])
def test_the_same_bits_each_time(hkv, rows, vocab):
    x = _randn(5, (rows, vocab), BF16, 2.0)
    labels = _labels(6, rows, vocab)
    g = _randn(7, (rows,))
    a = hkv.token_logps(x, labels, 20)
    da = hkv.token_logps_backward(a, g, g)
    for _ in range(3):
        b = hkv.token_logps(x, labels, 20)
        for name in ("logps", "entropy", "top_logps", "top_ids"):
            assert torch.equal(getattr(a, name), getattr(b, name))
        assert torch.equal(da, hkv.token_logps_backward(b, g, g))


def test_in_a_graph_and_on_another_stream(hkv):
    rows, vocab = 20, 40000
    x, labels = _randn(1, (rows, vocab), BF16, 2.0), _labels(2, rows, vocab)
    g = _randn(3, (rows,))
    hkv.token_logps_backward(hkv.token_logps(x, labels, 5), g)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f = hkv.token_logps(x, labels, 5)
        d = hkv.token_logps_backward(f, g)
    x.copy_(_randn(9, (rows, vocab), BF16, 2.0))
    graph.replay()
    torch.cuda.synchronize()
    want = hkv.token_logps(x, labels, 5)
    assert torch.equal(f.top_ids, want.top_ids) and torch.equal(f.logps, want.logps)
    assert torch.equal(d, hkv.token_logps_backward(want, g))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        s = hkv.token_logps(x, labels, 5, stream=stream)
        ds = hkv.token_logps_backward(s, g, stream=stream)
        side.synchronize()
        assert torch.equal(s.top_ids, want.top_ids) and torch.equal(ds, d)


def _overlapping(x):
    """A matrix that begins in the middle of x's first row."""
    return x.as_strided(x.shape, x.stride(), x.storage_offset() + 20)


def test_columns_of_one_buffer(hkv):
    buf = _randn(1, (6, 80))
    x = buf[:, :40]
    labels = _labels(2, 6, 40)
    f = hkv.token_logps(x, labels)
    g = _randn(3, (6,))
    want = hkv.token_logps_backward(f, g)
    assert torch.equal(hkv.token_logps_backward(f, g, out=buf[:, 40:]), want)


def test_refusals(hkv):
    x = _randn(1, (12, 40))[:6]
    labels = torch.zeros(6, dtype=torch.int64, device=DEV)
    f = hkv.token_logps(x, labels, 2)
    for bad in (lambda: hkv.token_logps(x.double(), labels), lambda: hkv.token_logps(x[0], labels),
                lambda: hkv.token_logps(x.t(), labels), lambda: hkv.token_logps(x, labels[:5]),
                lambda: hkv.token_logps(x, labels.int()), lambda: hkv.token_logps(x, labels.cpu()),
                lambda: hkv.token_logps(x, labels, top=33), lambda: hkv.token_logps(x, labels, top=-1),
                lambda: hkv.token_logps(x[:, :4], labels, top=5), lambda: hkv.token_logps(x[:, :0], labels),
                lambda: hkv.token_logps_backward(f, torch.zeros(5, device=DEV)),
                lambda: hkv.token_logps_backward(f, torch.zeros(6, dtype=BF16, device=DEV)),
                lambda: hkv.token_logps_backward(f, dentropy=torch.zeros(6)),
                lambda: hkv.token_logps_backward(f, out=torch.zeros((6, 41), device=DEV)),
                lambda: hkv.token_logps_backward(f, out=torch.zeros((6, 40), dtype=BF16, device=DEV)),
                lambda: hkv.token_logps_backward(f, out=torch.zeros((40, 6), device=DEV).t()),
                lambda: hkv.token_logps_backward(f, out=_overlapping(x))):
        with pytest.raises((ValueError, hkv.HKVError)):
            bad()
