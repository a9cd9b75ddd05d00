"""What a kept result keeps of the device's memory."""
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


def test_losses_and_logps_keep_no_more_than_themselves(hkv):
    rows, pairs = 4000, 3
    x = torch.randn((rows, 50), device=DEV)
    labels = torch.randint(50, (rows,), device=DEV)
    f = hkv.preference_loss(x, labels, torch.arange(2 * pairs + 1, device=DEV) * 600)
    assert f.losses.untyped_storage().nbytes() <= 3 * pairs * 4
    assert f.ratios.untyped_storage().nbytes() <= 3 * pairs * 4
    assert f.logps.untyped_storage().nbytes() == 4 * rows


@pytest.mark.parametrize("along", ["rows", "columns", "both"])
def test_each_copy_has_memory_of_its_own(hkv, along):
    rows, cols = 700, 4100
    got = hkv.mx_quantize(torch.randn((rows, cols), device=DEV), along)
    copies = got if along == "both" else (got,)
    for q in copies:
        own = q.rows * -(-q.cols // 32) * 16 + -(-q.rows // 128) * -(-q.cols // 128) * 512
        assert q.codes.untyped_storage().nbytes() < own + 512
        assert q.scales.untyped_storage().data_ptr() == q.codes.untyped_storage().data_ptr()
    assert along != "both" or copies[0].codes.untyped_storage().data_ptr() != copies[1].codes.untyped_storage().data_ptr()


def test_clipping_takes_any_order_without_overlaps(hkv):
    """Outs and gradients side by side in one buffer, in every order; gradients
    that are only read may be listed twice."""
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        part = torch.randn(24 * 1000, generator=g, device=DEV).split(1000)
        order = torch.randperm(24, generator=torch.Generator().manual_seed(seed)).tolist()
        grads, outs = [part[i] for i in order[:12]], [part[i] for i in order[12:]]
        want = torch.cat(grads).double()
        norm = hkv.clip_grad_norm(grads, 1.0, outs=outs)
        assert abs(float(norm) - float(want.norm())) <= 1e-5 * float(want.norm())
        assert float((torch.cat(outs).double() - want / want.norm()).abs().max()) < 1e-6
        hkv.clip_grad_norm(grads[::-1], 1.0)
        assert float((torch.cat(grads).double() - want / want.norm()).abs().max()) < 1e-6
    x = torch.ones(50, device=DEV)
    assert abs(float(hkv.clip_grad_norm([x, x], 1.0, outs=())) - 10.0) < 1e-5
    with pytest.raises(hkv.HKVError):
        hkv.clip_grad_norm([x, x], 1.0)
    with pytest.raises(hkv.HKVError):
        hkv.clip_grad_norm([x, x.view(5, 10)], 1.0, outs=[torch.zeros_like(x), x])
    assert (x == 1).all()
    hkv.clip_grad_norm([x, x], 100.0, outs=[torch.zeros_like(x), torch.zeros_like(x)])
