"""adapter_matmul and its gradients on batches whose lengths and adapters are uneven (the
kernels are chosen from means), with more adapters than a block has threads, and from two
threads at once."""
import threading

import pytest
import torch

from tests.test_gpu_adapters import TYPES, Case, hkv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,which,count", [
    ([500] + [1] * 255, [i % 64 for i in range(256)], 64),  # a prompt among single tokens: by row
    ([1] * 60 + [2100] + [1] * 40, [i % 7 - 1 for i in range(101)], 7),  # in tiles of 64 rows
    ([1] * 60 + [900] + [1] * 40, [i % 7 - 1 for i in range(101)], 7),  # of 16
    ([13] * 300, [5] * 300, 256), ([13] * 300, [i * i % 256 for i in range(300)], 256),  # a popular adapter, and none
    ([3800] + [1] * 255, list(range(256)), 256)])
@pytest.mark.parametrize("rank", [8, 40])
@pytest.mark.parametrize("dtype", TYPES)
def test_uneven(hkv, lengths, which, count, rank, dtype):  # noqa: F811
    Case(dtype, 136, 264, rank, lengths, which, count=count, before=1, behind=3).check(hkv)


@pytest.mark.parametrize("requests,count", [(1000, 1000), (700, 1400), (1400, 700)])
@pytest.mark.parametrize("longest", [1, 4])
@pytest.mark.parametrize("dtype", TYPES)
def test_many_adapters_in_use(hkv, requests, count, longest, dtype):  # noqa: F811
    lengths = [1 + i % longest for i in range(requests)]
    Case(dtype, 72, 40, 9, lengths, [i * 7 % count for i in range(requests)], count=count, behind=1).check(hkv)


def test_two_threads(hkv):  # noqa: F811
    """Each with a stream and a batch of its own; single rows, short and long requests."""
    cases = [[Case(torch.bfloat16, 512, 384, 16, lengths, [i % 3 for i in range(len(lengths))], seed=seed)
              for lengths in ([1] * 30, [12] * 24, [200, 130])] for seed in (0, 60)]

    def both(c, stream):
        f = c.call(hkv, stream=stream)
        return (f.out, *hkv.adapter_matmul_backward(f, c.dy, base=c.dx_base, stream=stream))

    want = [[both(c, None) for c in of] for of in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(of, expected):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got = [both(c, stream) for c in of]
                stream.synchronize()
                wrong.extend(1 for g, w in zip(got, expected) for u, v in zip(g, w) if not torch.equal(u, v))
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=pair) for pair in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
