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
                      dlogits=P, dstride=10, stream=None)


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
        dict(lse=None), dict(entropy=None), dict(dlogits=None), dict(dlogits=P + 2), dict(dstride=9), dict(dstride=11),
        dict(lse=P + 2), dict(entropy=P + 2), dict(dlogps=P + 2), dict(dentropy=P + 2), dict(labels=P + 4)])
    good = [dict(LOGPS, rows=0)[k] for k in LOGPS]
    assert lib.hkv_token_logps(*good) == 0


def test_constants_match_the_header():
    import hash_table_cache_gb300 as hkv
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    assert int(re.search(r"#define HKV_MAX_TOP (\d+)", text).group(1)) == hkv.MAX_TOP


def test_cpu_tensors_are_refused():
    import torch
    import hash_table_cache_gb300 as hkv
    with pytest.raises(ValueError):
        hkv.token_logps(torch.zeros((4, 64)), torch.zeros(4, dtype=torch.int64))
