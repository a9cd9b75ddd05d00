"""adapter_matmul and its gradients against their 64-bit forms
(tests/adapters_plain.py), at the shapes, strides and requests where they can go
wrong."""
import math

import pytest
import torch

from tests.adapters_plain import adapter_matmul as plain
from tests.operators_plain import near

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
    torch.cuda.empty_cache()


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


def _int(values):
    return torch.tensor(values, dtype=torch.int64, device=DEV)


class Case:
    """Inputs of one call: `lengths` of the requests and their adapters, `before` and
    `behind` rows of none."""

    def __init__(self, dtype, k, n, rank, lengths, which, count=3, before=0, behind=0, seed=0, scales=True, base=True):
        ends = [before]
        for v in lengths:
            ends.append(ends[-1] + v)
        self.offsets, self.which = _int(ends), _int(which)
        tokens = ends[-1] + behind
        self.x = _randn(seed, (tokens, k), dtype)
        self.down = _randn(seed + 1, (count, rank, k), dtype, k ** -0.5)
        self.up = _randn(seed + 2, (count, n, rank), dtype, rank ** -0.5)
        self.scales = torch.rand(count, generator=_gen(seed + 3), device=DEV) + 0.5 if scales else None
        self.base = _randn(seed + 4, (tokens, n), dtype) if base else None
        self.dy = _randn(seed + 5, (tokens, n), dtype)
        self.dx_base = _randn(seed + 6, (tokens, k), dtype) if base else None

    def call(self, hkv, out=None, **how):
        return hkv.adapter_matmul(self.x, self.down, self.up, self.offsets, self.which, self.scales, base=self.base,
                                  out=out, **how)

    def check(self, hkv, backward=True, out=None, dx=None):
        want = plain(self.x, self.down, self.up, self.offsets, self.which, self.scales, self.base,
                     self.dy if backward else None, self.dx_base)
        f = self.call(hkv, out)
        assert out is None or f.out is out
        near(f.out, *want["out"], "out")
        if backward:
            got = hkv.adapter_matmul_backward(f, self.dy, base=self.dx_base, out=dx)
            for name, v in zip(("dx", "ddown", "dup"), got):
                near(v, *want[name], name)
        return f


@pytest.mark.parametrize("k,n", [(1, 1), (8, 5), (64, 64), (70, 130), (128, 96), (513, 260), (1000, 77), (2048, 24),
                                 (40, 3000), (4096, 4096)])
@pytest.mark.parametrize("rank", [1, 8, 13, 16, 24, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_shapes(hkv, k, n, rank, dtype):
    Case(dtype, k, n, rank, [5, 0, 1, 70, 3], [2, 1, 0, 0, -1], before=2, behind=3, seed=k + n + rank).check(hkv)


@pytest.mark.parametrize("lengths,which", [
    ([1], [0]), ([1] * 7, [0, 2, 1, 1, -1, 3, 0]), ([1] * 300, [i % 5 - 1 for i in range(300)]),
    ([16] * 20, [1] * 20), ([17, 15, 16, 33, 31, 64, 65, 63], [0, 0, 0, 1, 1, 2, 2, 2]), ([500], [2]), ([200, 200], [1, 1]),
    ([0, 0, 0], [0, 1, 2]), ([0, 130, 0, 1, 0], [0, 1, 2, 1, 2]), ([3, 4], [-1, 7]), ([], []),
    ([2] * 1100, [i * 7 % 3 for i in range(1100)]), ([40] * 70, [0] * 70),
    ([0, 0, 1, 0, 2, 0, 0, 1] * 150, [i % 4 - 1 for i in range(1200)]),  # more requests than tokens
    ([1] * 900, [i % 3 for i in range(900)]), ([3] * 40, [i % 3 for i in range(40)])])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", [8, 33])
def test_requests(hkv, lengths, which, dtype, rank):
    Case(dtype, 320, 192, rank, lengths, which, before=1, behind=20).check(hkv)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_scales_and_base(hkv, dtype):
    Case(dtype, 200, 264, 8, [30, 2, 90], [1, -1, 2], before=3, behind=5, scales=False, base=False).check(hkv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths", [[1, 1, 1, 1], [40, 3, 0, 100]])
def test_in_place(hkv, dtype, lengths):
    """base itself is written; rows of no adapter are left as they are, whatever they hold."""
    c = Case(dtype, 136, 200, 16, lengths, [0, -1, 1, 2], before=2, behind=70)
    want = plain(c.x, c.down, c.up, c.offsets, c.which, c.scales, c.base, c.dy, c.dx_base)
    idle = torch.ones(len(c.x), dtype=torch.bool, device=DEV)
    ends = c.offsets.tolist()
    for a, b, w in zip(ends, ends[1:], c.which.tolist()):
        idle[a:b] = w < 0
    c.base[idle] = math.nan
    c.dx_base[idle] = math.nan
    version = c.base._version
    f = c.call(hkv, out=c.base)
    assert f.out is c.base and c.base._version > version
    dx, _, _ = hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base, out=c.dx_base)
    assert dx is c.dx_base
    for got, name in ((c.base, "out"), (dx, "dx")):
        assert got[idle].isnan().all()
        near(got[~idle], *(v[~idle] for v in want[name]), name)


@pytest.mark.parametrize("extra,shift", [(0, 1), (1, 0), (3, 5), (8, 8), (5, 0), (8, 4), (2, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rank", [7, 16])
def test_strides(hkv, extra, shift, dtype, rank):
    c = Case(dtype, 168, 136, rank, [33, 1, 5, 80], [0, 1, 2, 0], before=1, behind=2)
    c.x, c.base, c.dy, c.dx_base = (_strided(t, extra, shift) for t in (c.x, c.base, c.dy, c.dx_base))
    # adapters as the rows of a table's buffer, one after the other and something else between
    bank = torch.full((3, shift + rank * (168 + 136) + extra), math.nan, dtype=dtype, device=DEV)
    down = bank[:, shift:shift + rank * 168].unflatten(1, (rank, 168))
    up = bank[:, shift + rank * 168:shift + rank * 304].unflatten(1, (136, rank))
    down.copy_(c.down)
    up.copy_(c.up)
    c.down, c.up = down, up
    out, dx = (_strided(torch.zeros_like(t), extra, shift) for t in (c.base, c.x))
    c.check(hkv, out=out, dx=dx)
    for t in (out, dx):
        whole = torch.empty(0, dtype=dtype, device=DEV).set_(t.untyped_storage())
        assert int(whole.isnan().sum()) == shift + extra * len(t), "elements between the rows were written"


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_adapters_apart(hkv, dtype):
    """Rows of the factors further apart than they are long."""
    c = Case(dtype, 96, 80, 8, [50, 2], [0, 2])
    big = torch.full((3, 8, 120), math.nan, dtype=dtype, device=DEV)
    big[:, :, :96] = c.down
    tall = torch.full((3, 80, 24), math.nan, dtype=dtype, device=DEV)
    tall[:, :, 8:16] = c.up
    c.down, c.up = big[:, :, :96], tall[:, :, 8:16]
    c.check(hkv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lengths", [[1, 1, 1], [50, 20, 90]])
def test_what_is_not_of_a_request_has_no_effect(hkv, dtype, lengths):
    """NaN and infinities in rows of no request, in adapters of none, and in another
    request's rows."""
    c = Case(dtype, 264, 328, 12, lengths, [0, -1, 2], before=3, behind=9)
    want = plain(c.x, c.down, c.up, c.offsets, c.which, c.scales, c.base, c.dy, c.dx_base)
    ends = c.offsets.tolist()
    for t in (c.x, c.dy):
        t[:ends[0]] = math.nan
        t[ends[1]:ends[2]] = math.inf
        t[ends[3]:] = -math.inf
    c.down[1], c.up[1], c.scales[1] = math.nan, math.inf, math.nan
    f = c.call(hkv)
    got = dict(zip(("dx", "ddown", "dup"), hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base)), out=f.out)
    for name, v in got.items():
        near(v, *want[name], name)
    c.x[ends[0]] = math.nan  # one row of the first request
    f = c.call(hkv)
    assert f.out[ends[0]].isnan().all()
    assert torch.equal(f.out[ends[0] + 1:], got["out"][ends[0] + 1:])
    dx, ddown, _ = hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base)
    assert torch.equal(dx, got["dx"]) and ddown[0].isnan().all() and torch.equal(ddown[2], got["ddown"][2])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rank", [5, 16, 32, 48, 64])
@pytest.mark.parametrize("k,n", [(8, 16), (16, 8), (24, 40), (64, 128), (72, 200), (520, 1000), (1032, 136)])
def test_long_requests(hkv, dtype, rank, k, n):
    """Tiles that end in every part of their 64 rows, columns and ranks that end inside a
    box of the loads."""
    Case(dtype, k, n, rank, [64, 1, 63, 65, 0, 127, 128, 200], [0, 1, 2, 0, 1, -1, 2, 0], before=5, behind=70,
         seed=rank).check(hkv)


@pytest.mark.parametrize("lengths", [[300, 40], [70] * 6])
def test_one_adapter_for_all(hkv, lengths):
    """One adapter seen as several, a step of 0 between them; every request's gradient
    is its own all the same."""
    which = list(range(len(lengths)))
    c = Case(BF16, 256, 320, 16, lengths, which, count=len(lengths))
    c.down, c.up = (t[:1].expand(t.shape) for t in (c.down, c.up))
    c.check(hkv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rank", [8, 9])
def test_many_more_requests_than_rows(hkv, dtype, rank):
    lengths = [0] * 3000
    for i, v in ((5, 1), (700, 40), (701, 2), (2990, 17)):
        lengths[i] = v
    Case(dtype, 64, 72, rank, lengths, [i % 4 - 1 for i in range(3000)], before=3, behind=4).check(hkv)


@pytest.mark.parametrize("k,n", [(1, 1), (9, 300), (264, 520), (70, 130), (513, 257), (2048, 1023), (31, 4100)])
@pytest.mark.parametrize("rank", [1, 8, 13, 16, 31, 32, 48, 63, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_alone(hkv, k, n, rank, dtype):
    """Requests of one row, and of two by one adapter or several."""
    Case(dtype, k, n, rank, [1] * 37, [i * 5 % 7 - 1 for i in range(37)], count=7, before=1, behind=2, seed=k + rank).check(hkv)
    Case(dtype, k, n, rank, [2, 0, 3, 1, 2], [1, 0, -1, 1, 2], seed=n + rank).check(hkv)


@pytest.mark.parametrize("k,n", [(64, 260), (37, 1100), (130, 130)])
@pytest.mark.parametrize("rank", [2, 8, 9])
@pytest.mark.parametrize("dtype", TYPES)
def test_more_rows_alone_than_tiles_take(hkv, k, n, rank, dtype):
    """Eight rows to a request and nine, of more requests than a small call's."""
    for length in (4, 5, 8, 9):
        Case(dtype, k, n, rank, [length] * 260, [i * 7 % 5 - 1 for i in range(260)], count=4, behind=1, seed=length).check(hkv)


@pytest.mark.parametrize("k,n", [(264, 520), (261, 77)])
@pytest.mark.parametrize("rank", [5, 24, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows_to_an_adapter(hkv, k, n, rank, dtype):
    """More rows and requests than a step of the sums takes, adapters without any, and the
    lengths around the rule's borders."""
    lengths = [i * 7 % 6 for i in range(600)]
    Case(dtype, k, n, rank, lengths, [i * i % 61 - 1 for i in range(600)], count=60, before=2, behind=1).check(hkv)
    Case(dtype, k, n, rank, [3], [150], count=191).check(hkv)
    for length in (15, 16, 17, 32):
        Case(dtype, k, n, rank, [length] * 3, [2, 0, 1], seed=length).check(hkv)


@pytest.mark.parametrize("k,n", [(1, 1), (70, 130), (513, 257), (1000, 77), (40, 3000)])
@pytest.mark.parametrize("rank", [1, 13, 16, 24, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_to_an_adapter(hkv, k, n, rank, dtype):
    Case(dtype, k, n, rank, [5, 0, 150, 70, 3, 90], [2, 1, 0, 0, -1, 1], before=2, behind=3, seed=k + n + rank).check(hkv)


@pytest.mark.parametrize("extra,shift", [(0, 1), (3, 5), (8, 8), (8, 4)])
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("rank", [7, 40])
def test_strides_of_rows_alone(hkv, extra, shift, dtype, rank):
    """What lies between the rows and around the factors' is neither used nor written."""
    c = Case(dtype, 168, 136, rank, [1, 1, 2, 1], [0, 1, 2, 0], before=1, behind=2)
    c.x, c.base, c.dy, c.dx_base = (_strided(t, extra, shift) for t in (c.x, c.base, c.dy, c.dx_base))
    bank = torch.full((3, shift + rank * (168 + 136) + extra), math.nan, dtype=dtype, device=DEV)
    down = bank[:, shift:shift + rank * 168].unflatten(1, (rank, 168))
    up = bank[:, shift + rank * 168:shift + rank * 304].unflatten(1, (136, rank))
    down.copy_(c.down)
    up.copy_(c.up)
    c.down, c.up = down, up
    out, dx = (_strided(torch.zeros_like(t), extra, shift) for t in (c.base, c.x))
    c.check(hkv, out=out, dx=dx)
    for t in (out, dx):
        whole = torch.empty(0, dtype=dtype, device=DEV).set_(t.untyped_storage())
        assert int(whole.isnan().sum()) == shift + extra * len(t), "elements between the rows were written"
    # NaN behind the last rank of every row, and behind the last column
    tall = torch.full((3, 136, rank + 3), math.nan, dtype=dtype, device=DEV)
    tall[:, :, :rank] = up
    wide = torch.full((3, rank, 168 + 5), math.nan, dtype=dtype, device=DEV)
    wide[:, :, :168] = down
    c.down, c.up = wide[:, :, :168], tall[:, :, :rank]
    c.check(hkv)


@pytest.mark.parametrize("rank", [3, 20, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_many_adapters_of_few_requests(hkv, dtype, rank):
    """Adapters of no request get zeros, whatever their gradients' memory held; two
    requests of one adapter meet in one sum; rows shared by as many blocks as there are."""
    junk = torch.full((3 << 20,), math.nan, device=DEV)
    del junk
    for lengths, which in (([3000, 40], [33, 2]), ([700, 0, 90, 64], [5, 30, 5, -1]), ([2, 1], [36, 36]), ([130], [99])):
        Case(dtype, 72, 41, rank, lengths, which, count=37, before=1, behind=2).check(hkv)
    Case(dtype, 1100, 1030, rank, [1, 50], [69, 0], count=70).check(hkv)


def test_numbers_at_the_ends_of_the_range(hkv):
    """Hidden numbers above float16's largest and below its smallest, and float32's
    with all digits in use."""
    for big in (2.0 ** 9, 2.0 ** -12):
        c = Case(F16, 640, 72, 8, [20, 1], [0, 1], count=2)
        c.x, c.down, c.up = c.x * big, c.down * big, c.up / big / (big if big > 1 else 1)
        c.check(hkv, backward=False)
    c = Case(F32, 300, 200, 8, [40, 3], [0, 1], count=2)
    c.x = c.x.exp2().pow(20)
    c.dy = c.dy * torch.exp2(20 * torch.randn((43, 1), generator=_gen(4), device=DEV))
    c.check(hkv)


@pytest.mark.parametrize("rank", [6, 40])
def test_gradients_against_differences(hkv, rank):
    """L = sum dy out is linear in each of x, down and up, so the difference quotient
    of any step is the derivative: it is off by out's bounds over the step and by the
    gradient's bound."""
    c = Case(F32, 90, 70, rank, [30, 2, 1], [1, 0, 1], count=2, base=False)
    f = c.call(hkv)
    grads = hkv.adapter_matmul_backward(f, c.dy)
    want = plain(c.x, c.down, c.up, c.offsets, c.which, c.scales, None, c.dy)
    for i, name in enumerate(("x", "down", "up")):
        t = getattr(c, name)
        v = _randn(20 + i, t.shape) / t.numel() ** 0.5 * float(t.norm())
        quotient = e = 0.0
        for sign in (1, -1):
            setattr(c, name, t + sign * v)
            moved = getattr(c, name).double() - t.double()
            quotient += sign * (c.dy.double() * c.call(hkv).out.double()).sum() / 2
            bound = plain(c.x, c.down, c.up, c.offsets, c.which, c.scales)["out"][1]
            e += (c.dy.double().abs() * bound).sum() / 2
            # the step that the rounding of t + v makes
            e += ((moved - sign * v.double()).abs() * grads[i].double().abs()).sum()
        setattr(c, name, t)
        e += (want[("dx", "ddown", "dup")[i]][1] * v.double().abs()).sum()
        got = (grads[i].double() * v.double()).sum()
        assert abs(float(got - quotient)) <= float(e), (name, float(got), float(quotient), float(e))


def test_past_32_bit_offsets(hkv):
    """Rows of x 2^30 elements apart, adapters 2^31 elements apart."""
    c = Case(BF16, 64, 72, 8, [2, 1], [1, 0], count=2)
    buf = torch.empty(2 * 2 ** 30 + 64, dtype=BF16, device=DEV)
    x = buf.as_strided((3, 64), (2 ** 30, 1))
    x.copy_(c.x)
    c.x = x
    bank = torch.empty(2 ** 31 + 4096, dtype=BF16, device=DEV)
    down, up = bank.as_strided((2, 8, 64), (2 ** 31, 64, 1)), bank.as_strided((2, 72, 8), (2 ** 31, 8, 1), 512)
    down.copy_(c.down)
    up.copy_(c.up)
    c.down, c.up = down, up
    c.check(hkv)
    del c, buf, bank
    torch.cuda.empty_cache()
    # outputs whose rows end past 2^31 elements
    c = Case(BF16, 16, 65536, 8, [40000], [0], count=1, base=False)
    f = c.call(hkv)
    some = _int([0, 1, 32767, 32768, 39999])
    want = plain(c.x[some], c.down, c.up, _int([0, 5]), _int([0]), c.scales)
    near(f.out[some], *want["out"], "out")


@pytest.mark.parametrize("lengths", [[1] * 40, [130, 70, 3]])
def test_the_same_bits_each_time(hkv, lengths):
    c = Case(BF16, 2048, 1536, 24, lengths, [i % 3 for i in range(len(lengths))])
    f = c.call(hkv)
    a = (f.out, *hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base))
    for _ in range(4):
        f = c.call(hkv)
        b = (f.out, *hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base))
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_in_a_graph_and_on_another_stream(hkv):
    """Another batch of the captured sizes: other lengths, adapters and inputs."""
    c = Case(BF16, 512, 384, 16, [30, 9, 25], [0, 1, 2], behind=6)
    other = Case(BF16, 512, 384, 16, [2, 61, 7], [2, -1, 2], behind=0, seed=40)
    hkv.adapter_matmul_backward(c.call(hkv), c.dy)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f = c.call(hkv)
        got = hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base)
    for name in ("x", "down", "up", "scales", "base", "dy", "dx_base", "offsets", "which"):
        getattr(c, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    g = c.call(hkv)
    want = hkv.adapter_matmul_backward(g, c.dy, base=c.dx_base)
    assert torch.equal(f.out, g.out) and all(torch.equal(u, v) for u, v in zip(got, want))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        s = c.call(hkv, stream=stream)
        d = hkv.adapter_matmul_backward(s, c.dy, base=c.dx_base, stream=stream)
        side.synchronize()
        assert torch.equal(s.out, g.out) and all(torch.equal(u, v) for u, v in zip(d, want))


@pytest.mark.parametrize("k,n", [(512, 384), (511, 385)])
def test_rows_alone_in_a_graph(hkv, k, n):
    """Replayed with other adapters: the idle ones' zeros follow which adapters these are."""
    c = Case(BF16, k, n, 16, [1] * 9, [i % 3 for i in range(9)], count=40, before=1, behind=2)
    other = Case(BF16, k, n, 16, [1] * 9, [39, -1, 7, 7, 0, 12, 39, 5, -1], count=40, before=1, behind=2, seed=40)
    hkv.adapter_matmul_backward(c.call(hkv), c.dy)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f = c.call(hkv)
        got = hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base)
    for name in ("x", "down", "up", "scales", "base", "dy", "dx_base", "offsets", "which"):
        getattr(c, name).copy_(getattr(other, name))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    want = plain(c.x, c.down, c.up, c.offsets, c.which, c.scales, c.base, c.dy, c.dx_base)
    for v, name in zip((f.out, *got), ("out", "dx", "ddown", "dup")):
        near(v, *want[name], name)
    side = torch.cuda.Stream()
    g = c.call(hkv, stream=side)
    d = hkv.adapter_matmul_backward(g, c.dy, base=c.dx_base, stream=side)
    side.synchronize()
    assert torch.equal(g.out, f.out) and all(torch.equal(u, v) for u, v in zip(got, d))


def test_two_calls_at_once(hkv):
    """Calls on two streams that share the adapters and nothing else."""
    cases = [Case(BF16, 1024, 1024, 16, [300, 5], [0, 2], seed=s) for s in (0, 60)]
    cases[1].down, cases[1].up = cases[0].down, cases[0].up
    want = [c.call(hkv).out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [c.call(hkv, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(f.out, w) for f, w in zip(got, want))


def test_bad_offsets_stay_inside(hkv):
    """Offsets outside the batch are cut to it; the rows of good requests come out."""
    c = Case(BF16, 128, 128, 8, [10, 20], [0, 1])
    good = c.call(hkv).out
    c.offsets[0], c.offsets[2] = -50, 10 ** 12
    assert torch.equal(c.call(hkv).out, good)


def test_columns_of_one_buffer(hkv):
    """x, base and out side by side in one buffer."""
    c = Case(BF16, 64, 96, 8, [20, 4], [0, 1])
    want = c.call(hkv).out
    buf = torch.empty((24, 64 + 96 + 96), dtype=BF16, device=DEV)
    buf[:, :64], buf[:, 64:160] = c.x, c.base
    c.x, c.base = buf[:, :64], buf[:, 64:160]
    assert torch.equal(c.call(hkv, out=buf[:, 160:]).out, want)
    assert torch.equal(c.call(hkv, out=buf[:, 64:160]).out, want)


def test_no_tokens_and_no_adapters(hkv):
    c = Case(F32, 40, 30, 4, [], [])
    f = c.check(hkv)
    assert f.out.shape == (0, 30)
    c = Case(F32, 40, 30, 4, [3], [0], count=0)
    f = c.check(hkv)
    assert torch.equal(f.out, c.base)


def test_refusals(hkv):
    c = Case(BF16, 64, 48, 8, [5, 4], [0, 1])
    f = c.call(hkv)

    def call(**change):
        v = dict(x=c.x, down=c.down, up=c.up, offsets=c.offsets, which=c.which, scales=c.scales, base=c.base) | change
        return hkv.adapter_matmul(**v)

    def back(dy=c.dy, **how):
        return hkv.adapter_matmul_backward(f, dy, **how)

    square = _randn(1, (9, 64), BF16)
    for bad in (lambda: call(x=c.x.double()), lambda: call(x=c.x.float()), lambda: call(x=c.x[0]), lambda: call(x=c.x.t()),
                lambda: call(down=c.down[0]), lambda: call(down=c.down[:2]), lambda: call(down=c.down[:, :7]),
                lambda: call(down=c.down.float()), lambda: call(down=c.down[:, :, ::2], x=c.x[:, ::2].contiguous()),
                lambda: call(up=c.up[:, :, :7]), lambda: call(up=c.up.cpu()), lambda: call(up=c.up.transpose(1, 2)),
                lambda: call(offsets=c.offsets[:2]), lambda: call(offsets=c.offsets.int()), lambda: call(which=c.which.cpu()),
                lambda: call(which=c.which.float()), lambda: call(scales=c.scales[:2]), lambda: call(scales=c.scales.double()),
                lambda: call(base=c.base[:, :40]), lambda: call(base=c.base.float()), lambda: call(out=c.base[:5]),
                lambda: call(down=_randn(1, (3, 65, 64), BF16), up=_randn(2, (3, 48, 65), BF16)),
                lambda: call(down=c.down[:, :0], up=c.up[:, :, :0]),
                lambda: call(up=_randn(1, (3, 64, 8), BF16), base=None, x=square, out=square),
                lambda: call(base=c.base[:, :47], up=c.up[:, :47], out=c.base[:, 1:]),
                lambda: back(c.dy[:, :40]), lambda: back(c.dy.float()), lambda: back(out=c.x), lambda: back(base=c.dy),
                lambda: back(out=torch.empty((9, 64), device=DEV))):
        with pytest.raises((ValueError, hkv.HKVError)):
            bad()
