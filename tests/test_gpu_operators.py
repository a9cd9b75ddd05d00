"""The operators on looked-up rows against their plain 64-bit forms
(tests/operators_plain.py), at the sizes, strides and masks where they can go
wrong, and their refusals."""
import math

import pytest
import torch

from tests import operators_plain as plain

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
    yield m
    assert m.hkv_get_wait_timeouts() == (0, 0)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(seed, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * scale).to(dtype)


def _strided(x, extra, shift):
    """The same matrix with `extra` elements between rows, `shift` elements into
    its buffer; the buffer around it is NaN."""
    rows, cols = x.shape
    buf = torch.full((shift + rows * (cols + extra),), float("nan"), dtype=x.dtype, device=x.device)
    view = buf[shift:].view(rows, cols + extra)[:, :cols]
    view.copy_(x)
    return view


# --------------------------------------------------------------------------
# 4-bit copies
# --------------------------------------------------------------------------
def _check_copy(q, x):
    code, byte = plain.quantize(x)
    codes, scales = plain.layout(code, byte)
    assert torch.equal(q.codes.cpu().reshape(-1), codes.reshape(-1)), "codes differ"
    assert torch.equal(q.scales.cpu().reshape(-1), scales.reshape(-1)), "scales differ"
    want = plain.values(code, byte, x.shape[1])
    for dtype in (F32, BF16):
        got = q.dequantize(dtype).cpu().double()
        assert torch.equal(got.nan_to_num(7e77), want.nan_to_num(7e77)), f"values differ as {dtype}"
    got = q.dequantize(F16).cpu()
    assert torch.equal(got.nan_to_num(3e4), want.to(F32).to(F16).nan_to_num(3e4))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 31), (2, 33), (129, 64), (127, 96), (128, 128),
                                       (257, 300), (64, 1000), (1000, 64), (5, 4097), (33, 8), (512, 160),
                                       (300, 513)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("along", ["rows", "columns", "both"])
def test_copy(hkv, rows, cols, dtype, along):
    x = _randn(rows * 7 + cols, (rows, cols), dtype)
    x *= torch.exp(2 * torch.randn((rows, 1), generator=_gen(3), device=DEV)).to(dtype)
    q = hkv.mx_quantize(x, along)
    if along != "columns":
        _check_copy(q[0] if along == "both" else q, x)
    if along != "rows":
        _check_copy(q[1] if along == "both" else q, x.t())


@pytest.mark.parametrize("extra,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (32, 0), (5, 0), (8, 4), (2, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_copy_of_strided_rows(hkv, extra, shift, dtype):
    x = _strided(_randn(1, (130, 200), dtype), extra, shift)
    q, qt = hkv.mx_quantize(x, "both")
    _check_copy(q, x)
    _check_copy(qt, x.t())
    out = _strided(torch.zeros((130, 200), dtype=dtype, device=DEV), extra, shift)
    buf = out.untyped_storage()
    q.dequantize(out=out)
    assert torch.equal(out, q.dequantize(dtype))
    whole = torch.empty(0, dtype=dtype, device=DEV).set_(buf)
    assert int(whole.isnan().sum()) == shift + extra * 130, "bytes between the rows were written"


@pytest.mark.parametrize("dtype", TYPES)
def test_copy_rounds_ties_to_even(hkv, dtype):
    """Every level, the middle between each two, and the neighbours of the
    middles, at scales up to the ends of the range."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    eps = {F32: 2.0 ** -22, BF16: 2.0 ** -6, F16: 2.0 ** -9}[dtype]
    v = [0.0, 0.5, 1, 1.5, 2, 3, 4, 6, 7.5] + [m * f for m in mids for f in (1, 1 - eps, 1 + eps)]
    v = (v + [0.0] * 32)[:32]
    row = torch.tensor([v, [-a for a in v]], dtype=torch.float64)
    row[:, 31] = 4.0  # fixes the scale at 1
    powers = [0, 1, -1, 7] + ([100, -100, 124, -126, -130, -140] if dtype != F16 else [12, -12, -20])
    x = torch.cat([row * 2.0 ** p for p in powers]).to(dtype).to(DEV)
    _check_copy(hkv.mx_quantize(x), x)
    _check_copy(hkv.mx_quantize(x.t().contiguous(), "columns"), x)


def test_copy_of_special_values(hkv):
    """Zeros, negative zeros, NaN and infinities in some blocks only, the
    largest and the smallest floats, whole subnormal blocks."""
    x = _randn(5, (40, 130))
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = math.nan
    x[3, 64] = math.inf
    x[4, 129] = -math.inf
    x[5] = torch.finfo(F32).max
    x[6] = torch.finfo(F32).tiny
    x[7] = 2.0 ** -149
    x[8] *= 2.0 ** -128
    x[9] = -torch.finfo(F32).max
    for dtype in (F32, BF16):
        q, qt = hkv.mx_quantize(x.to(dtype), "both")
        _check_copy(q, x.to(dtype))
        _check_copy(qt, x.to(dtype).t())


def test_empty_copies(hkv):
    for shape in ((0, 5), (5, 0), (0, 0)):
        q = hkv.mx_quantize(torch.empty(shape, device=DEV), "both")
        assert q[0].shape == shape and q[1].shape == shape[::-1]
        assert q[0].dequantize().shape == shape


def test_copy_past_32_bit_offsets(hkv):
    """Rows 2^30 elements apart: the last starts 2^31 elements in."""
    buf = torch.empty(2 * 2 ** 30 + 64, dtype=BF16, device=DEV)
    x = buf.as_strided((3, 64), (2 ** 30, 1))
    x.copy_(_randn(8, (3, 64), BF16))
    q, qt = hkv.mx_quantize(x, "both")
    _check_copy(q, x)
    _check_copy(qt, x.t())
    want = q.dequantize(BF16)
    q.dequantize(out=x)
    assert torch.equal(x, want)


def test_copy_refusals(hkv):
    x = torch.zeros((4, 64), device=DEV)
    for bad in (x.cpu(), x[0], x.t(), x.double(), x.int(), x[:1].expand(4, 64)):
        with pytest.raises(ValueError):
            hkv.mx_quantize(bad)
    with pytest.raises(ValueError):
        hkv.mx_quantize(x, "diagonal")
    q = hkv.mx_quantize(x)
    with pytest.raises(ValueError):
        q.dequantize(torch.float64)
    with pytest.raises(ValueError):
        q.dequantize(out=x[:3])
    with pytest.raises(ValueError):
        hkv.MXMatrix(q.codes, q.scales, 4, 65)
    with pytest.raises(ValueError):
        hkv.MXMatrix(q.codes.float(), q.scales, 4, 64)


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------
def _check_product(hkv, a, b, dtype, out=None):
    m, n = a.shape[0], b.shape[0]
    qa, qb = hkv.mx_quantize(a), hkv.mx_quantize(b)
    y = hkv.mx_matmul(qa, qb, dtype=dtype, out=out)
    want, bound = plain.matmul(qa.dequantize().double(), qb.dequantize().double())
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -132
    bound = bound * (1 + plain.U[dtype]) + want.abs() * plain.U[dtype] + tiny
    if dtype == F16:
        want = torch.where(want.abs() > 65519, torch.sign(want) * math.inf, want)
    assert y.shape == (m, n)
    plain.near(y, want, bound, f"{m} x {n} x {a.shape[1]}")
    return y


SIZES = [(1, 1, 1), (1, 128, 64), (1, 4096, 1000), (2, 300, 32), (15, 17, 33), (16, 129, 96), (17, 64, 256),
         (31, 1000, 257), (32, 256, 512), (33, 127, 2048), (64, 384, 160), (65, 130, 511), (100, 257, 640),
         (128, 128, 128), (129, 128, 31), (200, 513, 1024), (255, 1, 300), (256, 256, 256), (257, 640, 4096),
         (384, 2000, 64), (1000, 777, 333), (2049, 130, 8), (130, 5000, 64)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_product(hkv, m, n, k, dtype):
    _check_product(hkv, _randn(m, (m, k)), _randn(n + 1, (n, k), scale=0.1), dtype)


@pytest.mark.parametrize("m,n,k", [(1, 512, 8192), (8, 128, 16384), (40, 130, 8200), (300, 300, 5000),
                                   (4099, 520, 160), (1, 40000, 64), (1100, 9000, 96)])
def test_product_of_long_rows_and_many(hkv, m, n, k):
    _check_product(hkv, _randn(m, (m, k)), _randn(n + 1, (n, k), scale=0.1), BF16)


@pytest.mark.parametrize("m,n,k", [(1300, 3100, 600), (1537, 2561, 64), (3000, 1500, 33), (193, 20001, 300),
                                   (2500, 4000, 2100), (5000, 900, 515)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_of_many_tiles(hkv, m, n, k, dtype):
    """More tiles than SMs: several tiles per block, ragged in every direction."""
    _check_product(hkv, _randn(m, (m, k)), _randn(n + 1, (n, k), scale=0.1), dtype)


@pytest.mark.parametrize("extra,shift", [(0, 1), (1, 0), (3, 3), (2, 0), (8, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_into_strided_rows(hkv, extra, shift, dtype):
    for m, n in ((5, 200), (150, 131)):
        out = _strided(torch.zeros((m, n), dtype=dtype, device=DEV), extra, shift)
        whole = torch.empty(0, dtype=dtype, device=DEV).set_(out.untyped_storage())
        _check_product(hkv, _randn(1, (m, 200)), _randn(2, (n, 200)), dtype, out)
        assert int(whole.isnan().sum()) == shift + extra * m, "bytes between the rows were written"


def test_product_scales_rows_apart(hkv):
    """Rows and blocks whose scales are far apart: a scale taken from another
    row or block would be off by powers of two."""
    for m, n, k in ((40, 300, 256), (300, 200, 320), (1, 260, 512)):
        ea = torch.randint(-12, 12, (m, k // 32), generator=_gen(m), device=DEV)
        eb = torch.randint(-12, 12, (n, k // 32), generator=_gen(n), device=DEV)
        a = _randn(1, (m, k)) * (2.0 ** ea.float()).repeat_interleave(32, 1)
        b = _randn(2, (n, k)) * (2.0 ** eb.float()).repeat_interleave(32, 1)
        _check_product(hkv, a, b, F32)


def test_product_of_special_values(hkv):
    """A block of NaNs makes its row or column NaN and nothing else; zero rows
    give zeros."""
    a, b = _randn(1, (70, 200)), _randn(2, (300, 200))
    a[3, 150] = math.nan
    a[69, 0] = math.inf
    a[5] = 0
    b[299, 33] = -math.inf
    b[7] = 0
    y = _check_product(hkv, a, b, F32)
    assert y[3].isnan().all() and y[69].isnan().all() and y[:, 299].isnan().all()
    assert (y[5, :299] == 0).all() and int(y.isnan().sum()) == 2 * 300 + 68


def test_product_without_columns_or_rows(hkv):
    e = lambda r, c: hkv.mx_quantize(torch.zeros((r, c), device=DEV))  # noqa: E731
    y = hkv.mx_matmul(e(3, 0), e(5, 0), out=torch.full((3, 5), 7.0, device=DEV))
    assert torch.equal(y, torch.zeros((3, 5), device=DEV))
    assert hkv.mx_matmul(e(0, 64), e(5, 64)).shape == (0, 5)
    assert hkv.mx_matmul(e(5, 64), e(0, 64)).shape == (5, 0)


def test_product_past_32_bit_offsets(hkv):
    """The last output row starts past 2^31 elements."""
    buf = torch.empty(2 * 2 ** 30 + 64, dtype=BF16, device=DEV)
    _check_product(hkv, _randn(1, (3, 64)), _randn(2, (64, 64)), BF16, buf.as_strided((3, 64), (2 ** 30, 1)))


def test_products_of_a_training_step(hkv):
    """Input and weight gradients through the copies along the other axis: the
    formulas' products of the values that the copies stand for."""
    m, n, k = 130, 96, 200
    x, w, dy = _randn(1, (m, k), BF16), _randn(2, (n, k), BF16), _randn(3, (m, n), BF16)
    qx, qxt = hkv.mx_quantize(x, "both")
    qw, qwt = hkv.mx_quantize(w, "both")
    qdy, qdyt = hkv.mx_quantize(dy, "both")
    for got, a, b in ((hkv.mx_matmul(qdy, qwt, F32), qdy, qwt), (hkv.mx_matmul(qdyt, qxt, F32), qdyt, qxt)):
        want, bound = plain.matmul(a.dequantize().double(), b.dequantize().double())
        plain.near(got, want, bound + 2.0 ** -130, "gradient")
    # the copies along the other axis stand for nearly the same matrices
    assert float((qwt.dequantize().t() - w.float()).norm() / w.float().norm()) < 0.2


def test_product_same_bits_every_time(hkv):
    for m, n, k in ((1, 512, 4096), (70, 300, 2000), (600, 600, 600)):
        qa, qb = hkv.mx_quantize(_randn(1, (m, k))), hkv.mx_quantize(_randn(2, (n, k)))
        first = hkv.mx_matmul(qa, qb, dtype=F32)
        for _ in range(5):
            assert torch.equal(hkv.mx_matmul(qa, qb, dtype=F32), first)


def test_product_refusals(hkv):
    q = lambda r, c: hkv.mx_quantize(torch.zeros((r, c), device=DEV))  # noqa: E731
    with pytest.raises(ValueError):
        hkv.mx_matmul(q(4, 64), q(4, 96))
    with pytest.raises(ValueError):
        hkv.mx_matmul(q(4, 64), q(4, 64), dtype=torch.float64)
    with pytest.raises(ValueError):
        hkv.mx_matmul(q(4, 64), q(4, 64), out=torch.zeros((4, 5), device=DEV))
    with pytest.raises(ValueError):
        hkv.mx_matmul(q(4, 64), q(5, 64), out=torch.zeros((5, 4), device=DEV).t())


# --------------------------------------------------------------------------
# preference loss
# --------------------------------------------------------------------------
def _pairs(lengths, vocab, dtype, seed=0, masked=0.25, scale=2.0):
    offsets = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], device=DEV)
    rows = int(offsets[-1])
    logits = _randn(seed, (rows, vocab), dtype, scale)
    labels = torch.randint(vocab, (rows,), generator=_gen(seed + 1), device=DEV)
    hide = torch.rand(rows, generator=_gen(seed + 2), device=DEV) < masked
    labels = torch.where(hide, -100, labels)
    ref = -math.log(vocab) + _randn(seed + 3, (rows,))
    return logits, labels, offsets, ref


def _check_loss(hkv, logits, labels, offsets, ref=None, beta=0.1, smoothing=0.0, average=False, dlosses=None,
                out=None):
    f = hkv.preference_loss(logits, labels, offsets, ref, beta=beta, label_smoothing=smoothing, average=average)
    want = plain.preference(logits, labels, offsets, ref, beta, smoothing, average, dlosses)
    for name in ("losses", "ratios", "logps"):
        plain.near(getattr(f, name), *want[name], name)
    plain.near(hkv.preference_loss_backward(f, dlosses, out=out), *want["grad"], "gradient")
    return f


@pytest.mark.parametrize("vocab", [1, 2, 31, 257, 1000, 4096, 32771, 131072])
@pytest.mark.parametrize("dtype", TYPES)
def test_loss(hkv, vocab, dtype):
    case = _pairs([5, 1, 7, 3, 2, 9], vocab, dtype, seed=vocab)
    _check_loss(hkv, *case, beta=0.3, smoothing=0.1, dlosses=_randn(9, (3,)))


@pytest.mark.parametrize("beta,smoothing,average", [(0.1, 0.0, False), (2.0, 0.0, True), (0.5, 1.0, False),
                                                    (0.0, 0.2, True), (-0.3, 0.5, False), (30.0, 0.0, False)])
def test_loss_parameters(hkv, beta, smoothing, average):
    case = _pairs([40, 33, 1, 64, 50, 2], 515, F32, seed=3)
    _check_loss(hkv, *case, beta=beta, smoothing=smoothing, average=average)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_of_empty_and_hidden_sequences(hkv, dtype):
    """Sequences without tokens, sequences whose tokens are all hidden, labels
    past the vocabulary, tokens after the last sequence, no reference."""
    lengths = [0, 4, 3, 5, 0, 6]
    logits, labels, offsets, _ = _pairs(lengths, 300, dtype, masked=0.0)
    labels[4:7] = -1
    labels[8] = 300
    labels[9] = 2 ** 40
    extra = torch.cat((logits, _randn(7, (3, 300), dtype)))
    labels = torch.cat((labels, torch.tensor([1, 2, 3], device=DEV)))
    for average in (False, True):
        f = _check_loss(hkv, extra, labels, offsets, None, average=average)
        assert f.ratios[0] == 0 and f.ratios[2 + 2] == 0
    d = hkv.preference_loss_backward(f)
    assert (d[18:] == 0).all() and (d[8] == 0).all()


def test_loss_of_all_hidden(hkv):
    logits, labels, offsets, ref = _pairs([3, 4], 100, F32)
    f = hkv.preference_loss(logits, torch.full_like(labels, -100), offsets, ref)
    assert abs(float(f.losses[0]) - math.log(2)) < 1e-6
    assert (hkv.preference_loss_backward(f) == 0).all()


def test_loss_ignores_what_hidden_rows_hold(hkv):
    logits, labels, offsets, ref = _pairs([6, 5], 700, F32, masked=0.0)
    labels[2] = labels[7] = -100
    for bad in (math.nan, math.inf, -math.inf):
        logits[2], ref[2] = bad, bad
        logits[7, ::3] = bad
        f = hkv.preference_loss(logits, labels, offsets, ref)
        d = hkv.preference_loss_backward(f)
        for t in (f.losses, f.ratios, f.logps, d):
            assert t.isfinite().all()
        assert (d[2] == 0).all() and (d[7] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_loss_of_banned_entries(hkv, dtype):
    """Vocabulary entries at -inf or the type's lowest value, whole aligned
    pieces of a row among them, the only allowed entry of a row the label."""
    logits, labels, offsets, ref = _pairs([4, 4], 5000, dtype, masked=0.0)
    for i, low in enumerate((-math.inf, torch.finfo(dtype).min)):
        logits[i, :4096] = low
        labels[i] = 4500
        logits[4 + i] = low
        logits[4 + i, 77] = 1.0
        labels[4 + i] = 77
        logits[2 + i, ::2] = low
        labels[2 + i] = 1
    _check_loss(hkv, logits, labels, offsets, ref)


def test_loss_of_infinite_and_nan_rows(hkv):
    """A counted row without any allowed entry, with NaN or with +inf gives NaN
    to its own pair alone; a banned label gives an infinite ratio."""
    logits, labels, offsets, ref = _pairs([3, 3, 3, 3, 2, 2, 2, 2], 400, F32, masked=0.0)
    logits[0] = -math.inf
    logits[4, 17] = math.nan
    logits[6, labels[6]] = -math.inf
    f = _check_loss(hkv, logits, labels, offsets, ref)
    assert f.losses[:2].isnan().all() and f.losses[2] == math.inf and f.losses[3].isfinite()


def test_loss_gradient_against_differences(hkv):
    """Central differences of the 64-bit loss at the largest entries of some rows."""
    logits, labels, offsets, ref = _pairs([5, 4, 6, 5], 60, F32, masked=0.2)
    up = torch.tensor([0.7, -1.3], device=DEV)
    f = hkv.preference_loss(logits, labels, offsets, ref, beta=0.4, label_smoothing=0.1)
    d = hkv.preference_loss_backward(f, up)

    def total(x):
        return float((plain.preference(x, labels, offsets, ref, 0.4, 0.1, False)["losses"][0] * up.double()).sum())

    step = 2.0 ** -12
    for row in range(0, 20, 3):
        for col in (int(logits[row].argmax()), 11):
            # 64-bit logits: dtype only picks a bound here
            x = logits.clone()
            x[row, col] += step
            hi = total(x)
            x[row, col] = logits[row, col] - step
            lo = total(x)
            span = float((logits[row, col] + step).double() - (logits[row, col] - step).double())
            # third derivative of the loss below 1: the step's error is step^2
            assert abs((hi - lo) / span - float(d[row, col])) < step ** 2 + 4e-6


@pytest.mark.parametrize("extra,shift", [(1, 0), (3, 5), (8, 0), (0, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_of_strided_logits(hkv, extra, shift, dtype):
    logits, labels, offsets, ref = _pairs([5, 3], 1000, dtype)
    x = _strided(logits, extra, shift)
    out = _strided(torch.zeros_like(logits), 2 * extra + 1, shift)
    whole = torch.empty(0, dtype=dtype, device=DEV).set_(out.untyped_storage())
    _check_loss(hkv, x, labels, offsets, ref, out=out)
    assert int(whole.isnan().sum()) == shift + (2 * extra + 1) * 8


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [515, 40000])
def test_loss_gradient_in_place(hkv, dtype, vocab):
    case = _pairs([4, 5], vocab, dtype)
    f = hkv.preference_loss(*case)
    want = hkv.preference_loss_backward(f)
    assert torch.equal(hkv.preference_loss_backward(f, out=f.logits), want)


def test_loss_of_many_tokens_and_pairs(hkv):
    """One pair of long sequences; many pairs of short ones."""
    _check_loss(hkv, *_pairs([3001, 2500], 130, F32))
    _check_loss(hkv, *_pairs([1 + i % 3 for i in range(1200)], 130, BF16))


def test_loss_past_32_bit_offsets(hkv):
    buf = torch.empty(2 * 2 ** 30 + 1000, dtype=BF16, device=DEV)
    logits, labels, offsets, ref = _pairs([1, 2], 1000, BF16, masked=0.0)
    x = buf.as_strided((3, 1000), (2 ** 30, 1))
    x.copy_(logits)
    f = _check_loss(hkv, x, labels, offsets, ref)
    want = hkv.preference_loss_backward(f)
    assert torch.equal(hkv.preference_loss_backward(f, out=x), want)


def test_loss_without_pairs_or_tokens(hkv):
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    f = hkv.preference_loss(torch.zeros((0, 10), device=DEV), none, torch.zeros(5, dtype=torch.int64, device=DEV))
    assert torch.allclose(f.losses, torch.full((2,), math.log(2), device=DEV), atol=1e-6, rtol=0)
    assert hkv.preference_loss_backward(f).shape == (0, 10)
    logits, labels, _, _ = _pairs([3, 4], 50, F32, masked=0.0)
    f = hkv.preference_loss(logits, labels, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert f.losses.numel() == 0 and (hkv.preference_loss_backward(f) == 0).all()


def test_loss_refusals(hkv):
    logits, labels, offsets, ref = _pairs([3, 4], 50, F32)
    go = hkv.preference_loss
    for bad in (lambda: go(logits.cpu(), labels, offsets), lambda: go(logits.double(), labels, offsets),
                lambda: go(logits.t(), labels, offsets), lambda: go(logits, labels[:-1], offsets),
                lambda: go(logits, labels.int(), offsets), lambda: go(logits, labels, offsets[:-1]),
                lambda: go(logits, labels, offsets.cpu()), lambda: go(logits, labels, offsets, ref.double()),
                lambda: hkv.preference_loss_backward(go(logits, labels, offsets), ref),
                lambda: hkv.preference_loss_backward(go(logits, labels, offsets), out=logits.half())):
        with pytest.raises(ValueError):
            bad()
    for kw in ({"beta": math.nan}, {"beta": math.inf}, {"label_smoothing": -0.1}, {"label_smoothing": 1.1},
               {"label_smoothing": math.nan}):
        with pytest.raises(hkv.HKVError) as e:
            go(logits, labels, offsets, **kw)
        assert e.value.status == hkv.HKV_ERR_INVALID


# --------------------------------------------------------------------------
# gradient norm and clipping
# --------------------------------------------------------------------------
def _check_clip(hkv, grads, max_norm, outs):
    """Bound: float32 sums of squares, one thread's chain no longer than the
    total over 2^14 (or 64 terms) and 64 joins; half of it is left by the root."""
    total = sum(g.numel() for g in grads)
    before = [g.double() for g in grads]
    norm = math.sqrt(sum(float(g.square().sum()) for g in before))
    u = 2.0 ** -24
    rel = (total / 2 ** 14 + 128) * u
    got = hkv.clip_grad_norm(grads, max_norm, outs)
    assert got.dtype == F32 and got.dim() == 0
    assert abs(float(got) - norm) <= rel * norm, (float(got), norm)
    if abs(norm - max_norm) <= rel * norm:
        return got
    factor = 1.0 if norm <= max_norm else max_norm / norm
    for o, b in zip(grads if outs == "in place" else outs, before):
        tiny = 2.0 ** -24 if o.dtype == F16 else 2.0 ** -132
        plain.near(o, b * factor, (b * factor).abs() * ((rel + 4 * u) * (factor != 1) + plain.U[o.dtype] * 1.01) + tiny,
                   "clipped")
    return got


SHAPES = [[1], [3], [5, 1, 1000], [4096, 4097, 4095], [100000], [70000, 1, 33, 129, 4096, 8191],
          [7] * 65, [10 + i % 40 for i in range(700)], [17] * 1030, [300] * 2100]


@pytest.mark.parametrize("sizes", SHAPES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("clips", [True, False])
def test_clip_in_place(hkv, sizes, dtype, clips):
    grads = [_randn(i, (n,), dtype, 0.1) for i, n in enumerate(sizes)]
    kept = [g.clone() for g in grads]
    norm = 0.1 * math.sqrt(sum(sizes))
    _check_clip(hkv, grads, norm * (0.05 if clips else 20.0), "in place")
    if not clips:
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
def test_clip_into_other_tensors(hkv, dtype, out):
    for clips in (True, False):
        grads = [_randn(i, (n,), dtype, 0.1) for i, n in enumerate([33, 4096, 1, 70001])]
        kept = [g.clone() for g in grads]
        outs = [torch.full_like(g, math.nan, dtype=out) for g in grads]
        _check_clip(hkv, grads, 0.5 if clips else 1e3, outs)
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_clip_of_mixed_types_and_shapes(hkv):
    """Matrices, transposes, scalars, tensors without elements and tensors that
    start in the middle of 16 bytes, side by side."""
    buf = {t: _randn(4, (40000,), t) for t in TYPES}
    grads = [buf[F32][1:1000], buf[BF16][3:5022].view(7, 717)[2:6], buf[F16][1:8194], buf[F32][5000:5001].view(()),
             buf[F32][6000:6000], buf[BF16][10001:20001].view(100, 100).t(), buf[F32][10001:10005],
             torch.zeros((0, 4), device=DEV)]
    edges = [buf[F32][:1].clone(), buf[F32][1000:5000].clone(), buf[F16][8194:].clone()]
    _check_clip(hkv, grads, 3.0, "in place")
    assert torch.equal(buf[F32][:1], edges[0]) and torch.equal(buf[F32][1000:5000], edges[1])
    assert torch.equal(buf[F16][8194:], edges[2])


def test_clip_norm_alone(hkv):
    g = _randn(1, (1000,), BF16)
    kept = g.clone()
    got = hkv.clip_grad_norm(g, 0.0, outs=())
    assert abs(float(got) - float(kept.double().norm())) < 1e-5 and torch.equal(g, kept)


def test_clip_of_special_values(hkv):
    for bad in (math.nan, math.inf):
        grads = [_randn(1, (5000,)), _randn(2, (77,), BF16)]
        grads[1][5] = bad
        norm = hkv.clip_grad_norm(grads, 1.0)
        if math.isnan(bad):
            assert norm.isnan() and all(g.isnan().all() for g in grads)
        else:
            assert norm == math.inf and (grads[0] == 0).all() and int(grads[1].isnan().sum()) == 1
    zero = [torch.zeros(100, device=DEV)]
    assert hkv.clip_grad_norm(zero, 0.0) == 0 and (zero[0] == 0).all()
    g = [_randn(3, (100,))]
    hkv.clip_grad_norm(g, 0.0)
    assert (g[0] == 0).all()
    g = [_randn(3, (100,))]
    kept = g[0].clone()
    hkv.clip_grad_norm(g, math.inf)
    assert torch.equal(g[0], kept)
    assert hkv.clip_grad_norm([torch.zeros(0, device=DEV)], 1.0) == 0


def test_clip_of_a_tensor_past_32_bits(hkv):
    g = torch.full((2 ** 31 + 77,), 2.0 ** -10, dtype=BF16, device=DEV)
    g[-1] = 64.0
    norm = hkv.clip_grad_norm(g, 1.0)
    want = math.sqrt((2 ** 31 + 76) * 2.0 ** -20 + 4096)
    assert abs(float(norm) - want) < want * 2.0 ** -20
    assert abs(float(g[-1]) * want / 64 - 1) < 2.0 ** -8
    assert float(g[2 ** 31 + 3]) == float(g[0]) and abs(float(g[0]) * want / 2.0 ** -10 - 1) < 2.0 ** -8


def test_clip_same_bits_every_time(hkv):
    grads = [_randn(i, (n,)) for i, n in enumerate([100001, 5, 77777, 300000])]
    first = hkv.clip_grad_norm(grads, 1.0, outs=())
    assert all(torch.equal(hkv.clip_grad_norm(grads, 1.0, outs=()), first) for _ in range(5))


def test_clip_refusals(hkv):
    g = _randn(1, (8, 8))
    for bad in (lambda: hkv.clip_grad_norm([], 1.0), lambda: hkv.clip_grad_norm([g.cpu()], 1.0),
                lambda: hkv.clip_grad_norm([g.double()], 1.0), lambda: hkv.clip_grad_norm([g[:, :4]], 1.0),
                lambda: hkv.clip_grad_norm([g, g], 1.0, outs=[g]), lambda: hkv.clip_grad_norm([g], 1.0, outs=[g.t()]),
                lambda: hkv.clip_grad_norm([g[0].expand(8, 8)], 1.0), lambda: hkv.clip_grad_norm([g], 1.0, "nowhere")):
        with pytest.raises(ValueError):
            bad()
    for limit in (-1.0, math.nan):
        with pytest.raises(hkv.HKVError) as e:
            hkv.clip_grad_norm([g], limit)
        assert e.value.status == hkv.HKV_ERR_INVALID


# --------------------------------------------------------------------------
# streams and graphs
# --------------------------------------------------------------------------
def _step(hkv, x, w, labels, offsets, outs, stream=None):
    q = hkv.mx_quantize(x, stream=stream)
    y = hkv.mx_matmul(q, hkv.mx_quantize(w, stream=stream), dtype=F32, stream=stream)
    f = hkv.preference_loss(y, labels, offsets, stream=stream)
    d = hkv.preference_loss_backward(f, stream=stream)
    norm = hkv.clip_grad_norm([d], 1e-3, outs=outs, stream=stream)
    return y, f.losses, d, norm


def test_operators_on_another_stream(hkv):
    """Each call on a stream of its own choosing, behind a long-running copy."""
    x, w = _randn(1, (70, 256)), _randn(2, (900, 256))
    _, labels, offsets, _ = _pairs([40, 30], 900, F32)
    want_out, out = (torch.zeros((70, 900), device=DEV) for _ in range(2))
    want = _step(hkv, x, w, labels, offsets, [want_out])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.empty(2 ** 28, device=DEV)
    with torch.cuda.stream(side):
        big.fill_(1)
        late = torch.empty_like(x)
        big.mul_(2)
        late.copy_(x)
    for s in (side, side.cuda_stream):
        got = _step(hkv, late, w, labels, offsets, [out], stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out, want_out)


def test_operators_in_a_graph(hkv):
    x, w = _randn(1, (70, 256)), _randn(2, (900, 256))
    _, labels, offsets, _ = _pairs([40, 30], 900, F32)
    want_out, out = (torch.zeros((70, 900), device=DEV) for _ in range(2))
    other = _randn(9, (70, 256))
    want = _step(hkv, other, w, labels, offsets, [want_out])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = _step(hkv, x, w, labels, offsets, [out])
    x.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out, want_out)
