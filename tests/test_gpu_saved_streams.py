"""Backward calls on another stream than the forward call's: what the forward call has
saved stays as it is until they are done with it, also when the result is dropped and its
memory's stream goes on."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    yield m
    torch.cuda.empty_cache()


def _randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


ROWS = 1 << 18  # what a call saves is an allocation of its own: 1 MB and more


def _adapters(hkv):
    x, dy = _randn(1, ROWS, 16, dtype=torch.bfloat16), _randn(2, ROWS, 24, dtype=torch.bfloat16)
    down, up = _randn(3, 2, 8, 16, dtype=torch.bfloat16), _randn(4, 2, 24, 8, dtype=torch.bfloat16)
    offsets, which = torch.tensor([0, ROWS // 2, ROWS], device=DEV), torch.tensor([1, 0], device=DEV)
    return (lambda s: hkv.adapter_matmul(x, down, up, offsets, which, stream=s),
            lambda f, s: hkv.adapter_matmul_backward(f, dy, stream=s), lambda f: [f._hidden])


def _logps(hkv):
    x, g = _randn(5, ROWS, 8), _randn(6, ROWS)
    labels = torch.arange(ROWS, device=DEV) % 9
    return (lambda s: hkv.token_logps(x, labels, stream=s),
            lambda f, s: (hkv.token_logps_backward(f, g, g, stream=s),), lambda f: [f._lse, f.entropy])


def _preference(hkv):
    x, labels = _randn(7, ROWS, 8), torch.arange(ROWS, device=DEV) % 9
    offsets = torch.arange(0, ROWS + 1, 1024, device=DEV)
    return (lambda s: hkv.preference_loss(x, labels, offsets, stream=s),
            lambda f, s: (hkv.preference_loss_backward(f, stream=s),), lambda f: [f._saved])


def _matrix(hkv):
    x = _randn(8, ROWS // 64, 512)
    one = hkv.mx_quantize(_randn(9, 16, 512))
    return (lambda s: hkv.mx_quantize(x, stream=s),
            lambda f, s: (hkv.mx_matmul(f, one, stream=s), f.dequantize(stream=s)), lambda f: [f._base[0]])


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("make", [_adapters, _logps, _preference, _matrix])
def test_saved_memory_on_another_stream(hkv, make, given):
    """The later stream is the current one, or one that is given."""
    forward, backward, saved = make(hkv)
    side, later = torch.cuda.Stream(), torch.cuda.Stream()

    def back(f):
        if given:
            return backward(f, later)
        with torch.cuda.stream(later):
            return backward(f, None)

    want = [None, None]  # the second one's memory is the later call's: nothing is allocated while a stream is busy
    busy = torch.empty(2 ** 29, device=DEV)
    busy.mul_(2.0)
    torch.full((5,), 0xFF, dtype=torch.uint8, device=DEV)  # all kernels are loaded
    for i in range(2):
        f = forward(side)
        torch.cuda.synchronize()
        want[i] = back(f)
        torch.cuda.synchronize()
        del f
    del want[1]
    f = forward(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(later):
        for _ in range(200):  # some tenths of a second
            busy.mul_(2.0)
    got = back(f)
    sizes = [t.untyped_storage().nbytes() for t in saved(f)]
    del f
    with torch.cuda.stream(side):
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes]
    side.synchronize()
    assert not later.query(), "the stream was done too early to show anything"
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want[0]))
    del junk


@pytest.mark.parametrize("make", [_adapters, _logps, _preference, _matrix])
def test_captured_after_an_eager_forward_call(hkv, make):
    """The capturing stream is another than the forward call's."""
    forward, backward, _ = make(hkv)
    f = forward(None)
    want = backward(f, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = backward(f, None)
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    del f, graph
    assert forward(None) is not None
    torch.cuda.synchronize()
