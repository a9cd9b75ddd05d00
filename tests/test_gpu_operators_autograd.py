"""What the operators write counts as written for autograd, and results carry
no gradient function."""
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


def _loss(hkv, logits):
    rows = logits.shape[0]
    return hkv.preference_loss(logits, torch.arange(rows, device=DEV), torch.arange(rows + 1, device=DEV))


def test_written_tensors_have_a_new_version(hkv):
    x = torch.randn((6, 64), device=DEV)
    q = hkv.mx_quantize(x)
    for call in (lambda t: q.dequantize(out=t), lambda t: hkv.preference_loss_backward(_loss(hkv, x), out=t)):
        out = torch.zeros_like(x)
        before = out._version
        call(out)
        assert out._version > before
    out = torch.zeros((6, 6), device=DEV)
    before = out._version
    hkv.mx_matmul(q, q, out=out)
    assert out._version > before
    grads = [torch.randn(5, device=DEV), torch.randn((3, 4), device=DEV)]
    outs = [torch.zeros_like(g) for g in grads]
    before = [t._version for t in grads + outs]
    hkv.clip_grad_norm(grads, 1.0, outs=())
    hkv.clip_grad_norm(grads, 0.1, outs=outs)
    assert [t._version for t in grads] == before[:2]
    assert all(t._version > v for t, v in zip(outs, before[2:]))
    hkv.clip_grad_norm(grads, 0.1)
    assert all(t._version > v for t, v in zip(grads, before))


def test_autograd_notices_logits_that_hold_their_gradient(hkv):
    w = torch.randn((4, 10), device=DEV, requires_grad=True)
    logits = (w * 2.0).exp()  # saves its result
    f = _loss(hkv, logits.detach())
    hkv.preference_loss_backward(f, out=f.logits)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        logits.sum().backward()


def test_autograd_notices_clipped_tensors(hkv):
    w = torch.randn(100, device=DEV, requires_grad=True)
    g = torch.randn(100, device=DEV)
    y = (w * g).sum()  # saves g
    hkv.clip_grad_norm([g], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inputs_that_require_a_gradient_give_results_without_one(hkv):
    x = torch.randn((4, 64), device=DEV, requires_grad=True)
    assert not hkv.mx_quantize(x).dequantize().requires_grad
    f = _loss(hkv, x)
    assert not f.losses.requires_grad and not hkv.preference_loss_backward(f).requires_grad


def test_inference_mode(hkv):
    with torch.inference_mode():
        g = [torch.ones(100, device=DEV)]
        assert float(hkv.clip_grad_norm(g, 1.0)) == 10.0
    hkv.clip_grad_norm(g, 0.5)  # an inference tensor outside: the kernel writes it all the same
    assert abs(float(g[0][0]) - 0.05) < 1e-6
