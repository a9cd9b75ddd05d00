"""Variants of the operators' kernels that the sizes elsewhere do not come to:
products of pairs of blocks and of eight storing warps into rows of y that
start anywhere, gradients and logits that lie differently in memory, clipped
tensors whose outs start elsewhere, and the C layer's own wrappers."""
import ctypes
import math

import pytest
import torch

from tests import operators_plain as plain
from tests import preference_bounds as bounds

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


def _randn(seed, shape, dtype=F32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _room(rows, cols, extra, shift, dtype):
    """A matrix with `extra` elements between rows, `shift` into a buffer of NaNs."""
    buf = torch.full((shift + rows * (cols + extra),), math.nan, dtype=dtype, device=DEV)
    return buf, buf[shift:].view(rows, cols + extra)[:, :cols]


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------
# m, n, k: pairs of blocks (more than five steps of k, tiles of pairs for more
# than every SM), then single blocks with eight storing warps (more than five
# steps, fewer tiles)
BRANCHES = [(2500, 4000, 2100), (2500, 4001, 2100), (1555, 7777, 1400), (400, 5000, 1500), (400, 5001, 1500),
            (385, 6144, 1311), (700, 3001, 4000)]


@pytest.mark.parametrize("m,n,k", BRANCHES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("extra,shift", [(0, 0), (3, 0), (5, 1), (8, 8)])
def test_product_into_rows_that_start_anywhere(hkv, m, n, k, dtype, extra, shift):
    a, b = hkv.mx_quantize(_randn(m, (m, k))), hkv.mx_quantize(_randn(n + 1, (n, k), scale=0.1))
    buf, out = _room(m, n, extra, shift, dtype)
    y = hkv.mx_matmul(a, b, out=out)
    want, bound = plain.matmul(a.dequantize().double(), b.dequantize().double())
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -132
    plain.near(y, want, bound * (1 + plain.U[dtype]) + want.abs() * plain.U[dtype] + tiny, f"{m} x {n} x {k}")
    assert int(buf.isnan().sum()) == shift + extra * m, "memory between the rows was written"


@pytest.mark.parametrize("k", [64, 700])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("extra,shift", [(1, 0), (0, 3)])
def test_product_of_short_k_into_rows_that_start_anywhere(hkv, k, dtype, extra, shift):
    """Twelve storing warps; more tiles than SMs, ragged on both sides."""
    m, n = 1537, 4099
    a, b = hkv.mx_quantize(_randn(k, (m, k))), hkv.mx_quantize(_randn(k + 1, (n, k), scale=0.1))
    buf, out = _room(m, n, extra, shift, dtype)
    y = hkv.mx_matmul(a, b, out=out)
    want, bound = plain.matmul(a.dequantize().double(), b.dequantize().double())
    tiny = 2.0 ** -24 if dtype == F16 else 2.0 ** -132
    plain.near(y, want, bound * (1 + plain.U[dtype]) + want.abs() * plain.U[dtype] + tiny, f"{k}")
    assert int(buf.isnan().sum()) == shift + extra * m, "memory between the rows was written"


# --------------------------------------------------------------------------
# copies of half-precision rows that start anywhere
# --------------------------------------------------------------------------
@pytest.mark.parametrize("extra,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (5, 0), (2, 2)])
def test_half_precision_copies_of_strided_rows(hkv, extra, shift):
    _, x = _room(130, 200, extra, shift, F16)
    x.copy_(_randn(1, (130, 200), F16))
    for q, v in zip(hkv.mx_quantize(x, "both"), (x, x.t())):
        codes, scales = plain.layout(*plain.quantize(v))
        assert torch.equal(q.codes.cpu().reshape(-1), codes.reshape(-1))
        assert torch.equal(q.scales.cpu().reshape(-1), scales.reshape(-1))
    q = hkv.mx_quantize(x)
    buf, out = _room(130, 200, extra, shift, F16)
    assert torch.equal(q.dequantize(out=out), q.dequantize(F16))
    assert int(buf.isnan().sum()) == shift + extra * 130


# --------------------------------------------------------------------------
# preference loss
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,stride", [(1000, 1003), (1000, 1024), (20001, 20032), (50257, 50304)])
@pytest.mark.parametrize("where", ["new", "strided", "in place"])
def test_gradient_of_the_first_columns_of_a_wider_matrix(hkv, dtype, vocab, stride, where):
    """Logits that are a view of a padded matrix: the default out starts its rows
    elsewhere."""
    rows = 24
    buf = torch.full((rows * stride,), math.nan, dtype=dtype, device=DEV)
    x = buf.view(rows, stride)[:, :vocab]
    x.copy_(_randn(vocab, (rows, vocab), dtype, 2.0))
    labels = torch.randint(vocab, (rows,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    up = _randn(2, (rows // 2,))
    f = hkv.preference_loss(x, labels, torch.arange(rows + 1, device=DEV), beta=0.5, label_smoothing=0.1)
    lp, e_lp, p, e = bounds.tokens(x, labels)
    assert float(((f.logps.double() - lp).abs() - e_lp).max()) <= 0
    h = 0.5 * (f.ratios[:rows // 2] - f.ratios[rows // 2:]).double()
    slope = 0.5 * (torch.sigmoid(h) - 0.9) * up.double()
    g = torch.cat((slope, -slope))[:, None]
    hot = torch.zeros_like(p)
    hot[torch.arange(rows, device=DEV), labels] = 1
    want = g * (hot - p)
    u, tiny = plain.U[dtype], 2.0 ** -24 if dtype == F16 else 2.0 ** -132
    # beside the softmax: the slope (two exponentials, of h rounded to 4 u |h|)
    e_g = 0.5 * up.double().abs() * (2.0 ** -21 + 4 * 2.0 ** -24 * h.abs())
    bound = (g.abs() * (e + 2.0 ** -22) + torch.cat((e_g, e_g))[:, None]) * (1 + u) + want.abs() * u + tiny
    room, out = None, None
    if where == "strided":
        room, out = _room(rows, vocab, 2 * (stride - vocab) + 1, 1, dtype)
    d = hkv.preference_loss_backward(f, up, out=x if where == "in place" else out)
    over = (d.double() - want).abs() - bound
    assert float(over.max()) <= 0, f"row {int(over.amax(1).argmax())}: {float(over.max()):.3g} over its bound"
    assert int(buf.isnan().sum()) == rows * (stride - vocab)
    assert room is None or int(room.isnan().sum()) == 1 + rows * (2 * (stride - vocab) + 1)


# --------------------------------------------------------------------------
# clipping
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("clips", [True, False])
def test_clip_into_a_buffer_without_padding(hkv, dtype, out, clips):
    """Outs that start anywhere beside gradients that do not, and the other way."""
    sizes = [33, 4097, 1, 70001, 8, 16385, 4096, 5]
    for shifted in (False, True):
        grads = [_randn(i, (n + 8,), dtype, 0.1)[i % 8 if shifted else 0:][:n] for i, n in enumerate(sizes)]
        flat = torch.full((sum(sizes) + 3,), math.nan, dtype=out, device=DEV)
        outs = list(flat[1:-2].split(sizes))
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        limit = norm * (0.3 if clips else 3.0)
        got = hkv.clip_grad_norm(grads, limit, outs=outs)
        # float32 sums: chains of no more than 64 terms and 64 joins, halved by the root
        rel = 64 * 2.0 ** -24
        assert abs(float(got) - norm) <= rel * norm
        want = torch.cat(grads).double() * (0.3 if clips else 1.0)
        u, tiny = plain.U[out], 2.0 ** -24 if out == F16 else 2.0 ** -132
        bound = want.abs() * ((rel + 4 * 2.0 ** -24) * clips + u * 1.01) + tiny
        plain.near(flat[1:-2], want, bound, "clipped")
        assert flat[0].isnan() and flat[-2:].isnan().all()


# --------------------------------------------------------------------------
# the C layer's wrappers
# --------------------------------------------------------------------------
def test_c_wrappers_do_what_the_operators_do(hkv):
    x = _randn(1, (70, 200), BF16)
    q, qt = hkv.mx_quantize(x, "both")
    like = [torch.empty_like(t) for t in (q.codes, q.scales, qt.codes, qt.scales)]
    assert hkv.hkv_mx_quantize(70, 200, x, hkv.HKV_BF16, 200, *like) == 0
    assert all(torch.equal(a, b) for a, b in zip(like, (q.codes, q.scales, qt.codes, qt.scales)))
    y = torch.empty((70, 200), device=DEV)
    assert hkv.hkv_mx_dequantize(70, 200, q.codes, q.scales, y, hkv.HKV_F32, 200) == 0
    assert torch.equal(y, q.dequantize())
    y = torch.empty((70, 70), dtype=F16, device=DEV)
    assert hkv.hkv_mx_matmul(70, 70, 200, q.codes, q.scales, q.codes, q.scales, y, hkv.HKV_F16, 70) == 0
    assert torch.equal(y, hkv.mx_matmul(q, q, dtype=F16))

    labels = torch.randint(200, (70,), device=DEV)
    offsets = torch.tensor([0, 10, 30, 60, 70], device=DEV)
    ref = _randn(3, (70,))
    f = hkv.preference_loss(x, labels, offsets, ref, beta=0.3, label_smoothing=0.2, average=True)
    losses, ratios, logps, lse, grad = (torch.empty(n, device=DEV) for n in (2, 4, 70, 70, 70))
    pair = torch.empty(70, dtype=torch.int32, device=DEV)
    assert hkv.hkv_preference_loss(2, 70, 200, x, hkv.HKV_BF16, 200, labels, offsets, ref, 0.3, 0.2, True, losses,
                                   ratios, logps, lse, grad, pair) == 0
    assert torch.equal(losses, f.losses) and torch.equal(ratios, f.ratios) and torch.equal(logps, f.logps)
    d = torch.empty_like(x)
    up = _randn(4, (2,))
    assert hkv.hkv_preference_loss_backward(2, 70, 200, x, hkv.HKV_BF16, 200, labels, lse, grad, pair, up, d, 200) == 0
    assert torch.equal(d, hkv.preference_loss_backward(f, up))

    g, out = _randn(5, (1000,)), torch.empty(1000, dtype=BF16, device=DEV)
    norm = torch.empty((), device=DEV)
    work = torch.empty(hkv.CLIP_WORK_BYTES, dtype=torch.uint8, device=DEV)
    one = (hkv.Grad * 1)(hkv.Grad(g.data_ptr(), out.data_ptr(), 1000, hkv.HKV_F32, hkv.HKV_BF16))
    assert hkv.hkv_clip_grad_norm(1, ctypes.cast(one, ctypes.c_void_p), 1.0, norm, work) == 0
    want = torch.empty_like(out)
    assert torch.equal(hkv.clip_grad_norm(g, 1.0, outs=want), norm) and torch.equal(out, want)
