"""Host-side refusals of the operators on looked-up rows: bad arguments return
HKV_ERR_INVALID before any CUDA call (no GPU needed)."""
import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 0x80000000
P = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from hash_table_cache_gb300 import _build
    import hash_table_cache_gb300 as hkv
    _build.build()
    return hkv.load()


def _with(base, **change):
    return [change.get(k, v) for k, v in base.items()]


QUANTIZE = dict(rows=4, cols=64, x=P, type=0, stride=64, codes=P, scales=P, codes_t=P, scales_t=P, stream=None)
DEQUANTIZE = dict(rows=4, cols=64, codes=P, scales=P, y=P, type=0, stride=64, stream=None)
MATMUL = dict(m=4, n=5, k=64, ac=P, asc=P, bc=P, bs=P, y=P, type=1, stride=5, stream=None)
LOSS = dict(pairs=2, rows=9, vocab=10, logits=P, type=0, stride=10, labels=P, offsets=P, ref=None, beta=0.1,
            smoothing=0.0, average=0, losses=P, ratios=P, logps=P, lse=P, row_grad=P, row_pair=P, stream=None)
BACKWARD = dict(pairs=2, rows=9, vocab=10, logits=P, type=0, stride=10, labels=P, lse=P, row_grad=P, row_pair=P,
                dlosses=None, dlogits=P, dstride=10, stream=None)


@pytest.mark.parametrize("name,base,bad", [
    ("hkv_mx_quantize", QUANTIZE, [
        dict(rows=BIG), dict(cols=BIG), dict(stride=63), dict(type=3), dict(type=-1), dict(x=None), dict(x=P + 2),
        dict(codes=None), dict(scales=None), dict(codes_t=None), dict(codes=P + 8), dict(scales_t=P + 1),
        dict(codes=None, scales=None, codes_t=None, scales_t=None), dict(type=1, x=P + 1)]),
    ("hkv_mx_dequantize", DEQUANTIZE, [
        dict(rows=BIG), dict(cols=BIG), dict(stride=63), dict(type=9), dict(codes=None), dict(scales=None),
        dict(y=None), dict(y=P + 2), dict(codes=P + 4), dict(scales=P + 4)]),
    ("hkv_mx_matmul", MATMUL, [
        dict(m=BIG), dict(n=BIG), dict(k=BIG), dict(stride=4), dict(type=3), dict(ac=None), dict(asc=None),
        dict(bc=None), dict(bs=None), dict(y=None), dict(y=P + 1), dict(ac=P + 8), dict(bs=P + 8)]),
    ("hkv_preference_loss", LOSS, [
        dict(pairs=BIG), dict(rows=BIG), dict(vocab=0), dict(vocab=BIG), dict(logits=None), dict(logits=P + 2),
        dict(type=3), dict(stride=9), dict(labels=None), dict(offsets=None), dict(beta=math.nan),
        dict(beta=math.inf), dict(smoothing=-0.5), dict(smoothing=1.5), dict(smoothing=math.nan),
        dict(losses=None), dict(ratios=None), dict(logps=None), dict(lse=None), dict(row_grad=None),
        dict(row_pair=None), dict(labels=P + 4), dict(offsets=P + 4), dict(ref=P + 2)]),
    ("hkv_preference_loss_backward", BACKWARD, [
        dict(pairs=BIG), dict(rows=BIG), dict(vocab=0), dict(logits=None), dict(type=3), dict(stride=9),
        dict(labels=None), dict(lse=None), dict(row_grad=None), dict(row_pair=None), dict(dlogits=None),
        dict(dlogits=P + 2), dict(dstride=9), dict(dstride=11), dict(dlosses=P + 1)]),
])
def test_refusals(lib, name, base, bad):
    for change in bad:
        assert getattr(lib, name)(*_with(base, **change)) == -1, (name, change)


def test_clip_refusals(lib):
    import hash_table_cache_gb300 as hkv
    go = lib.hkv_clip_grad_norm
    good = dict(data=P, out=P, n=10, type=0, out_type=0)

    def call(count=1, limit=1.0, norm=P, work=P, grads=True, **change):
        e = hkv.Grad(**{**good, **change})
        return go(count, ctypes.addressof(e) if grads else None, limit, norm, work, None)

    for change in (dict(limit=-1.0), dict(limit=math.nan), dict(norm=None), dict(work=None), dict(norm=P + 2),
                   dict(work=P + 1), dict(grads=False), dict(count=BIG), dict(type=3), dict(out_type=3),
                   dict(data=None), dict(data=P + 2), dict(out=P + 2), dict(out_type=1), dict(n=1 << 41)):
        assert call(**change) == -1, change


def test_wait_timeouts_wants_a_pointer(lib):
    assert lib.hkv_get_wait_timeouts(None) == -1


def test_sizes_and_constants_match_the_header():
    import hash_table_cache_gb300 as hkv
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    assert int(re.search(r"#define HKV_CLIP_WORK_BYTES (\d+)", text).group(1)) == hkv.CLIP_WORK_BYTES
    assert re.search(r"HKV_F32 = 0, HKV_BF16 = 1, HKV_F16 = 2", text)
    assert (hkv.HKV_F32, hkv.HKV_BF16, hkv.HKV_F16) == (0, 1, 2)
    assert ctypes.sizeof(hkv.Grad) == 32


def test_cpu_tensors_are_refused():
    import torch
    import hash_table_cache_gb300 as hkv
    x = torch.zeros((4, 64))
    for bad in (lambda: hkv.mx_quantize(x), lambda: hkv.clip_grad_norm([x], 1.0),
                lambda: hkv.MXMatrix(torch.zeros(128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64),
                lambda: hkv.preference_loss(x, torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            bad()
