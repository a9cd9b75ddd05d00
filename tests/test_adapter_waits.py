"""The waits of the adapters' kernels on tcgen05, as their source has them (a wait that
runs out cannot be tried on a GPU that works): bounded, with one answer for a warp where
the warp goes on together, and no block ends while a load is in flight."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def source():
    text = open(os.path.join(ROOT, "hash_table_cache_gb300", "csrc", "adapter_tensor.cuh")).read()
    return re.sub(r"//[^\n]*", "", text)


def _kernel(source, name):
    start = source.index(f"    {name}(const __grid_constant__")
    end = source.find("template <", start)
    return source[start:end if end > 0 else None]


def test_every_wait_is_bounded(source):
    body = source[source.index("bool slow_wait("):source.index("bool wait(")]
    assert re.search(r"while \(!mbar_try_wait\(bar, parity\)\)\s*if \(now_ns\(\) - begin > kWaitNs\)", body)
    assert "return false" in body and "g_wait_timeouts" in body
    rest = source[source.index("bool wait_warp("):]
    assert "mbar_try_wait" not in rest and not re.search(r"while \(!", rest)
    assert "__all_sync(0xFFFFFFFFu, wait(bar, parity))" in rest[:rest.index("elect(")]


@pytest.mark.parametrize("name", ["first_tensor_kernel", "second_tensor_kernel", "grads_tensor_kernel"])
def test_loads_are_waited_for(source, name):
    """Both roles that can give up wait for the full barriers of the loads that follow."""
    kernel = _kernel(source, name)
    for given_up in re.findall(r"!ok\b[^;]*?\{?[^;]*?for \(uint32_t i = (step[^;]*);[^{]*?wait\(&full\[i % S::kStages\], i / S::kStages & 1\)",
                               kernel):
        assert given_up in ("step - S::kStages", "step + 1", "step")
    assert len(re.findall(r"wait\(&full\[i % S::kStages\], i / S::kStages & 1\)", kernel)) == 2


@pytest.mark.parametrize("name", ["first_tensor_kernel", "second_tensor_kernel", "grads_tensor_kernel"])
def test_reads_of_sums_follow_a_warp_s_wait(source, name):
    kernel = _kernel(source, name)
    at = kernel.index("tcgen05.ld.sync.aligned")
    assert "wait_warp(&done, 0)" in kernel[:at] or "wait_warp(&ready[b]" in kernel[:at]
    assert kernel.index("tcgen05.alloc") < kernel.index("pdl_wait()") < at < kernel.index("tcgen05.dealloc")
