"""What the adapters' kernels on tcgen05 do where a wait runs out, and when their limited
waits begin, as their source has them (neither can be tried on a GPU that works)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DRAIN = r"for \(uint32_t i = ([^;]*); [^;]*; \+\+i\)\s*if \(!wait\(&full\[i % S::kStages\], i / S::kStages & 1\)\) break;"


@pytest.fixture(scope="module")
def source():
    text = open(os.path.join(ROOT, "hash_table_cache_gb300", "csrc", "adapter_tensor.cuh")).read()
    return re.sub(r"//[^\n]*", "", text)


def _kernel(source, name):
    start = source.index(f"    {name}(const __grid_constant__")
    end = source.find("template <", start)
    return source[start:end if end > 0 else None]


def _roles(kernel):
    """The loading thread's part and the multiplying one's."""
    load = kernel.index("if (warp == 0")
    multiply = kernel.index("} else if (warp == 1", load)
    end = kernel.find("} else if (warp >= 2)", multiply)
    return kernel[load:multiply], kernel[multiply:end if end > 0 else None]


@pytest.mark.parametrize("name,starts", [
    ("first_tensor_kernel", ["step - S::kStages", "step + 1"]),  # loaded and not known to be there; not yet waited for
    ("second_tensor_kernel", ["step - S::kStages", "step"]),  # (the wait that ran out may be another barrier's)
    ("grads_tensor_kernel", ["step - S::kStages", "step + 1"])])
def test_who_gives_up_waits_for_the_loads(source, name, starts):
    kernel = _kernel(source, name)
    assert re.findall(DRAIN, kernel) == starts
    for at in re.finditer(DRAIN, kernel):
        assert "!ok" in kernel[max(0, at.start() - 160):at.start()], "a drain that is not a given-up role's"


def test_who_gives_up_waits_for_the_planes(source):
    load, multiply = _roles(_kernel(source, "second_tensor_kernel"))
    for role in (load, multiply):
        given_up = role[role.rindex("if (!ok)"):]
        assert given_up.index("wait(&planes, 0);") < re.search(DRAIN, given_up).start()


def test_limited_waits_begin_when_the_first_product_is_done(source):
    """The second product's kernel starts before: how long the first one still takes is no
    part of a limited wait, whether the tile has an adapter or not."""
    load, multiply = _roles(_kernel(source, "second_tensor_kernel"))
    adding = _kernel(source, "second_tensor_kernel")
    adding = adding[adding.index("} else if (warp >= 2)"):]
    for role in (multiply, adding):
        first = re.search(r"\bwait(_warp)?\(&", role).start()
        assert "pdl_wait();" in role[:first]
    # the loading thread's first limited wait is for the stage that it loaded first
    assert re.search(r"if \(round > 0 && !wait\(&empty\[s\]", load)
    last_of_the_first_round = r"if \(step \+ 1 == S::kStages \|\| \(step \+ 1 == steps && steps < S::kStages\)\) \{\s*pdl_wait\(\);"
    assert re.search(last_of_the_first_round, load)
    for name in ("first_tensor_kernel", "grads_tensor_kernel"):
        kernel = _kernel(source, name)
        assert kernel.index("pdl_wait();") < re.search(r"\bwait(_warp)?\(&", kernel).start()
