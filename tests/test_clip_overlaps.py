"""Gradients and outs that overlap are refused on the host, before any launch
(no GPU needed; the addresses are never read)."""
import ctypes
import itertools

import pytest

P = 1 << 20
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    return m


def _status(hkv, entries):
    """entries: (data, out, n, type, out_type)"""
    grads = (hkv.Grad * len(entries))(*[hkv.Grad(*e) for e in entries])
    return hkv.load().hkv_clip_grad_norm(len(entries), ctypes.addressof(grads), 1.0, P, P, None)


@pytest.mark.parametrize("entries", [
    # listed twice, first or last element shared, one inside another
    [(P, P, 100, F32, F32), (P, P, 100, F32, F32)],
    [(P, P, 100, F32, F32), (P + 396, P + 396, 100, F32, F32)],
    [(P, P, 100, F32, F32), (P + 40, P + 40, 1, F32, F32)],
    [(P, P, 100, F32, F32), (P + 198, P + 198, 10, BF16, BF16)],
    # outs of different gradients
    [(P, P + 4096, 100, F32, F32), (P + 1024, P + 4492, 100, F32, F32)],
    [(P, P + 4096, 100, F32, BF16), (P + 1024, P + 4096 + 198, 100, F32, BF16)],
    # an out over another gradient, over a part of its own, exchanged, over one
    # that is there for its norm alone
    [(P, P + 4096, 100, F32, F32), (P + 4096, P + 8192, 100, F32, F32)],
    [(P, P + 4, 100, F32, F32)],
    [(P, P + 2, 100, BF16, BF16)],
    [(P, P + 4096, 100, F32, F32), (P + 4096, P, 100, F32, F32)],
    [(P, P, 100, F32, F32), (P + 396, P + 4096, 100, F32, F32)],
    [(P, P, 100, F32, F32), (P + 396, None, 100, F32, F32)],
])
def test_overlaps_are_refused(hkv, entries):
    apart = [(P + 65536, P + 65536, 7, F32, F32), (P + 131072, P + 131080, 0, F32, F32),
             (P + 70000, None, 100, F32, F32)]
    for order in itertools.permutations(entries + apart):
        assert _status(hkv, list(order)) == hkv.HKV_ERR_INVALID


def test_many_with_one_overlap(hkv):
    many = [(P + 4096 * i, P + 4096 * i, 1024, F32, F32) for i in range(700)]
    for i, j in ((0, 699), (3, 4), (350, 20)):
        entries = list(many)
        entries[i] = entries[j]
        assert _status(hkv, entries) == hkv.HKV_ERR_INVALID
        assert _status(hkv, entries[::-1]) == hkv.HKV_ERR_INVALID
