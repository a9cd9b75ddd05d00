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
