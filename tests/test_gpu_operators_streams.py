"""Calls on a stream of the caller's choosing: memory of tensors that are
dropped after the call, and streams of another device."""
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
    return m


def _busy(stream):
    """Some hundredths of a second of work ahead on the stream."""
    big = torch.empty(2 ** 29, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(40):
            big.mul_(2.0)
    return big


N = 1 << 20  # elements: an allocation of its own


def _quantize(hkv, side):
    x = torch.ones((1024, N // 1024), device=DEV)
    return hkv.mx_quantize(x, stream=side), [x]


def _dequantize(hkv, side):
    q = hkv.mx_quantize(torch.ones((4096, 1024), device=DEV))
    out = torch.empty((4096, 1024), device=DEV)
    return q.dequantize(out=out, stream=side), [q.codes]


def _wrapped(hkv, side):
    q = hkv.mx_quantize(torch.ones((4096, 1024), device=DEV))
    m = hkv.MXMatrix(q.codes.clone(), q.scales.clone(), 4096, 1024)
    return m.dequantize(stream=side), [m.codes]


def _matmul(hkv, side):
    a, b = (hkv.mx_quantize(torch.ones((4096, 1024), device=DEV)) for _ in range(2))
    return hkv.mx_matmul(a, b, stream=side), [a.codes, b.codes]


def _loss(hkv, side):
    x = torch.zeros((1024, N // 1024), device=DEV)
    labels = torch.zeros(1024, dtype=torch.int64, device=DEV)
    f = hkv.preference_loss(x, labels, torch.arange(1025, device=DEV), stream=side)
    f.logits = None
    return f, [x]


def _backward(hkv, side):
    x = torch.zeros((1024, N // 1024), device=DEV)
    labels = torch.zeros(1024, dtype=torch.int64, device=DEV)
    f = hkv.preference_loss(x, labels, torch.arange(1025, device=DEV))
    d = hkv.preference_loss_backward(f, stream=side)
    f.logits = None
    return d, [x]


def _clip(hkv, side):
    g, out = ([torch.ones(N, device=DEV) for _ in range(3)] for _ in range(2))
    return hkv.clip_grad_norm(g, 1.0, outs=out, stream=side), g + out


@pytest.mark.parametrize("call", [_quantize, _dequantize, _wrapped, _matmul, _loss, _backward, _clip])
@pytest.mark.parametrize("handle", [False, True])
def test_dropped_tensors_are_not_used_again_too_early(hkv, call, handle):
    """While the stream has not come to the call, a new allocation on the current
    stream does not get the memory of what the call reads or writes."""
    call(hkv, None)  # loads the kernels
    side = torch.cuda.Stream()
    keep = _busy(side)
    result, read = call(hkv, side.cuda_stream if handle else side)
    taken = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in read}
    del read
    assert not side.query(), "the stream was done too early to show anything"
    fresh = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in taken.values() for _ in range(4)]
    assert not {t.data_ptr() for t in fresh} & set(taken)
    assert not side.query(), "the stream was done too early to show anything"
    side.synchronize()
    del keep, result


def test_a_stream_of_another_device_is_refused(hkv):
    class Elsewhere:
        cuda_stream = 0
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError):
        hkv.mx_quantize(torch.zeros((4, 64), device=DEV), stream=Elsewhere())


@pytest.mark.parametrize("stream", [0, "default", "current"])
def test_the_default_stream_by_any_name(hkv, stream):
    x = torch.randn((70, 300), device=DEV)
    want = hkv.mx_quantize(x).dequantize()
    s = {"default": torch.cuda.default_stream(), "current": torch.cuda.current_stream()}.get(stream, stream)
    assert torch.equal(hkv.mx_quantize(x, stream=s).dequantize(stream=s), want)


def test_a_given_stream_in_a_graph(hkv):
    """The capturing stream named in every call, on tensors of another stream."""
    x, grads = torch.randn((70, 256), device=DEV), [torch.randn(5000, device=DEV)]
    outs = [torch.zeros(5000, device=DEV)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        q = hkv.mx_quantize(x, stream=side)
        y = hkv.mx_matmul(q, q, dtype=torch.float32, stream=side)
        norm = hkv.clip_grad_norm(grads, 1.0, outs=outs, stream=side)
    x.normal_()
    grads[0].normal_()
    graph.replay()
    torch.cuda.synchronize()
    q = hkv.mx_quantize(x)
    assert torch.equal(y, hkv.mx_matmul(q, q, dtype=torch.float32))
    want = torch.zeros_like(outs[0])
    assert torch.equal(norm, hkv.clip_grad_norm(grads, 1.0, outs=[want])) and torch.equal(outs[0], want)
