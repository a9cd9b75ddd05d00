"""Buffers that hkv_adapter_matmul and its backward call write must not overlap what they
read, nor one another: refused on the host, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from tests import test_answers_abi as abi

MB = 1 << 20  # an aligned address that is never dereferenced; every buffer below is smaller


@pytest.fixture(scope="module")
def lib():
    from hash_table_cache_gb300 import _build
    import hash_table_cache_gb300 as hkv
    _build.build()
    return hkv.load()


# float32, 9 rows of 64 and 48 numbers in rows of 80; 3 adapters of rank 8; h: 9 rows of 96 bytes
FORWARD = dict(tokens=9, k=64, n=48, type=0, adapters=None, requests=2, offsets=MB, which=2 * MB, x=3 * MB, x_stride=80,
               base=4 * MB, base_stride=80, y=5 * MB, y_stride=80, hidden=6 * MB, stream=None)
BACKWARD = dict(tokens=9, k=64, n=48, type=0, adapters=None, requests=2, offsets=MB, which=2 * MB, x=3 * MB, x_stride=80,
                dy=4 * MB, dy_stride=80, hidden=5 * MB, base=6 * MB, base_stride=80, dx=7 * MB, dx_stride=80, ddown=8 * MB,
                dup=9 * MB, dhidden=10 * MB, stream=None)
HIDDEN, DDOWN, DUP, ROWS = 9 * 96, 3 * 8 * 64 * 4, 3 * 48 * 8 * 4, 8 * 320


def _adapters(hkv, **change):
    v = dict(count=3, down=20 * MB, down_step=512, down_stride=64, up=21 * MB, up_step=384, up_stride=8, scales=22 * MB,
             rank=8) | change
    return hkv.Adapters(*[v[n] for n, _ in hkv.Adapters._fields_])


def _status(lib, name, args):
    import hash_table_cache_gb300 as hkv
    w = _adapters(hkv)
    return getattr(lib, name)(*(args | dict(adapters=ctypes.addressof(w))).values())


@pytest.mark.parametrize("name", ["x", "base", "y"])
def test_forward(lib, name):
    at = FORWARD[name]
    for hidden in (at, at + 64, at - HIDDEN + 16, at + ROWS + 16):  # the start, inside, its end, its last row
        assert _status(lib, "hkv_adapter_matmul", FORWARD | dict(hidden=hidden)) == -1, hidden - at


@pytest.mark.parametrize("written,size", [("dhidden", HIDDEN), ("ddown", DDOWN), ("dup", DUP)])
@pytest.mark.parametrize("name,end", [("x", ROWS), ("dy", ROWS), ("base", ROWS), ("dx", ROWS), ("hidden", HIDDEN - 96),
                                      ("dhidden", HIDDEN - 96), ("ddown", DDOWN - 96), ("dup", DUP - 96)])
def test_backward(lib, written, size, name, end):
    if name == written:
        return
    at = BACKWARD[name]
    for to in (at, at + 64, at - size + 16, at + end + 16):
        assert _status(lib, "hkv_adapter_matmul_backward", BACKWARD | {written: to}) == -1, to - at


def test_what_was_refused_is_refused_for_its_own_reason(lib):
    """The other refusals, with buffers apart."""
    import hash_table_cache_gb300 as hkv
    good = _adapters(hkv)
    for name, base, bad in (
            ("hkv_adapter_matmul", FORWARD, [dict(y=None), dict(y_stride=47), dict(y=3 * MB + 256), dict(y=4 * MB + 4)]),
            ("hkv_adapter_matmul_backward", BACKWARD, [dict(dy=None), dict(dy_stride=47), dict(dhidden=None),
                                                       dict(dhidden=10 * MB + 8), dict(ddown=8 * MB + 2),
                                                       dict(dup=9 * MB + 2), dict(dx=3 * MB), dict(dx=6 * MB + 4)])):
        apart = {"x": 3 * MB + 2, "offsets": MB + 4, "which": 2 * MB + 4, "hidden": base["hidden"] + 8, "base": base["base"] + 2}
        for change in abi.BAD + bad:
            change = {k: apart[k] if k in apart and v is not None else v for k, v in change.items()}
            args = dict(base, adapters=ctypes.addressof(good)) | change
            assert getattr(lib, name)(*args.values()) == -1, (name, change)
        for change in abi.BAD_ADAPTERS:
            change = {k: v + 19 * MB if k in ("down", "up", "scales") and v else v for k, v in change.items()}
            wrong = _adapters(hkv, **change)
            assert getattr(lib, name)(*(base | dict(adapters=ctypes.addressof(wrong))).values()) == -1, (name, change)


def test_beside_one_another(lib):
    """What only lies close is taken: nothing is launched without rows and adapters, and
    then no buffer holds anything."""
    import hash_table_cache_gb300 as hkv
    none = _adapters(hkv, count=0)
    args = BACKWARD | dict(tokens=0, adapters=ctypes.addressof(none), dhidden=5 * MB, ddown=3 * MB, dup=3 * MB)
    assert lib.hkv_adapter_matmul_backward(*args.values()) == 0
    assert lib.hkv_adapter_matmul(*(FORWARD | dict(tokens=0, adapters=ctypes.addressof(none), hidden=3 * MB)).values()) == 0
