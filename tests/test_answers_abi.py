"""Host-side refusals of the operators that answer many users: bad arguments
return HKV_ERR_INVALID before any CUDA call (no GPU needed)."""
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


LOGPS = dict(rows=9, vocab=10, logits=P, type=0, stride=10, labels=P, top=3, logps=P, entropy=P, top_logps=P,
             top_ids=P, lse=P, stream=None)
LOGPS_BACKWARD = dict(rows=9, vocab=10, logits=P, type=0, stride=10, labels=P, lse=P, entropy=P, dlogps=P, dentropy=P,
                      dlogits=4 * P, dstride=10, stream=None)


def _refused(lib, name, base, bad):
    for change in bad:
        assert set(change) <= set(base)
        assert getattr(lib, name)(*[change.get(k, v) for k, v in base.items()]) == -1, (name, change)


def test_token_logps(lib):
    _refused(lib, "hkv_token_logps", LOGPS, [
        dict(rows=BIG), dict(vocab=0), dict(vocab=BIG), dict(logits=None), dict(logits=P + 2), dict(type=3), dict(type=-1),
        dict(stride=9), dict(labels=None), dict(logps=None), dict(entropy=None), dict(top=11), dict(top=33, vocab=50, stride=50),
        dict(top_logps=None), dict(top_ids=None), dict(labels=P + 4), dict(logps=P + 2), dict(entropy=P + 1),
        dict(top_logps=P + 2), dict(top_ids=P + 4), dict(lse=P + 2)])
    _refused(lib, "hkv_token_logps_backward", LOGPS_BACKWARD, [
        dict(rows=BIG), dict(vocab=0), dict(logits=None), dict(logits=P + 2), dict(type=3), dict(stride=9), dict(labels=None),
        dict(lse=None), dict(entropy=None), dict(dlogits=None), dict(dlogits=4 * P + 2), dict(dstride=9), dict(dlogits=P, dstride=11), dict(dlogits=P + 4), dict(dlogits=P - 40),
        dict(lse=P + 2), dict(entropy=P + 2), dict(dlogps=P + 2), dict(dentropy=P + 2), dict(labels=P + 4)])
    good = [dict(LOGPS, rows=0)[k] for k in LOGPS]
    assert lib.hkv_token_logps(*good) == 0


def _adapters(hkv, **change):
    v = dict(count=3, down=P, down_step=512, down_stride=64, up=P, up_step=384, up_stride=8, scales=P, rank=8) | change
    return hkv.Adapters(*[v[n] for n, _ in hkv.Adapters._fields_])


FORWARD = dict(tokens=9, k=64, n=48, type=0, adapters=None, requests=2, offsets=P, which=P, x=P, x_stride=64, base=2 * P,
               base_stride=48, y=3 * P, y_stride=48, hidden=P, stream=None)
BACKWARD = dict(tokens=9, k=64, n=48, type=0, adapters=None, requests=2, offsets=P, which=P, x=P, x_stride=64, dy=2 * P,
                dy_stride=48, hidden=P, base=3 * P, base_stride=64, dx=4 * P, dx_stride=64, ddown=P, dup=P, dhidden=P,
                stream=None)
BAD_ADAPTERS = [dict(count=BIG), dict(rank=0), dict(rank=65), dict(down=None), dict(up=None), dict(down_stride=63),
                dict(up_stride=7), dict(down_stride=1 << 32), dict(up_stride=1 << 32), dict(down_step=1 << 41),
                dict(up_step=1 << 41), dict(down=P + 2), dict(up=P + 1), dict(scales=P + 2)]
BAD = [dict(tokens=BIG), dict(k=0), dict(n=0), dict(k=BIG), dict(n=BIG), dict(type=3), dict(requests=BIG), dict(offsets=None),
       dict(which=None), dict(offsets=P + 4), dict(which=P + 4), dict(x=None), dict(x=P + 2), dict(x_stride=63),
       dict(x_stride=1 << 32), dict(hidden=None), dict(hidden=P + 8), dict(base=P + 2), dict(adapters=None)]


def test_adapters(lib):
    import ctypes
    import hash_table_cache_gb300 as hkv
    good = _adapters(hkv)
    at = ctypes.addressof(good)
    for name, base, bad in (
            ("hkv_adapter_matmul", FORWARD, BAD + [
                dict(base_stride=47), dict(y=None), dict(y=3 * P + 2), dict(y_stride=47), dict(y_stride=1 << 32), dict(y=P),
                dict(y=P + 256), dict(y=2 * P, y_stride=49), dict(y=2 * P + 4)]),
            ("hkv_adapter_matmul_backward", BACKWARD, BAD + [
                dict(base_stride=63), dict(dy=None), dict(dy=2 * P + 2), dict(dy_stride=47), dict(dx=None), dict(dx=4 * P + 1),
                dict(dx_stride=63), dict(dhidden=None), dict(dhidden=P + 8), dict(ddown=P + 2),
                dict(dup=P + 2), dict(dx=P), dict(dx=2 * P), dict(dx=3 * P, dx_stride=65)])):
        _refused(lib, name, dict(base, adapters=at), bad)
        for change in BAD_ADAPTERS:
            wrong = _adapters(hkv, **change)
            _refused(lib, name, dict(base, adapters=ctypes.addressof(wrong)), [{}])
    assert lib.hkv_adapter_matmul(*dict(FORWARD, adapters=at, tokens=0).values()) == 0
    nothing = _adapters(hkv, count=0, down=None, up=None, scales=None)
    assert lib.hkv_adapter_matmul_backward(*dict(BACKWARD, adapters=ctypes.addressof(nothing), tokens=0).values()) == 0


def test_the_structure_is_the_header_s():
    import ctypes
    import hash_table_cache_gb300 as hkv
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    assert re.search(r"\(rank\) <= 16 \? 16 : \(rank\) <= 32 \? 32 : 64\) \* \(\(type\) == HKV_F32 \? 6 : 4\)", text)
    assert [hkv.adapter_hidden_bytes(3, r, t) for r, t in ((1, 0), (17, 1), (33, 2), (64, 0))] == [288, 384, 768, 1152]
    assert ctypes.sizeof(hkv.Adapters) == 72 and hkv.Adapters.rank.offset == 64 and hkv.Adapters.scales.offset == 56


def test_constants_match_the_header():
    import hash_table_cache_gb300 as hkv
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    assert int(re.search(r"#define HKV_MAX_TOP (\d+)", text).group(1)) == hkv.MAX_TOP
    assert int(re.search(r"#define HKV_MAX_RANK (\d+)", text).group(1)) == hkv.MAX_RANK


def test_cpu_tensors_are_refused():
    import torch
    import hash_table_cache_gb300 as hkv
    with pytest.raises(ValueError):
        hkv.token_logps(torch.zeros((4, 64)), torch.zeros(4, dtype=torch.int64))
