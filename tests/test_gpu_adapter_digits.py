"""How many digits of float32 matrices the adapters' kernels take: sums of one term each,
so that nothing but the products' own error is left.

A tile kernel takes a number in three parts of 8 digits, the first two cut off: the second
is below 2^-7 of the number, the third below 2^-15.  Of a product the three smallest of the
nine products of parts are left out: together below 2 2^-22 + 2^-30 of it.  The others are
added in a chain of the five lower ones (each below 2^-6 of the product, and what the tensor
core cuts off an addition is 2^-23 of that) and the highest, which is exact; joining the two
rounds by 2^-24.  So a product is off by at most 2^-21 + 2^-23 of itself, and an output,
a product of a product (h and dh go on with all 24 digits), by twice that and by its
square."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
EACH = 2.0 ** -21 + 2.0 ** -23


@pytest.fixture(scope="module")
def hkv():
    import hash_table_cache_gb300 as m
    from hash_table_cache_gb300 import _build
    _build.build()
    m.load()
    return m


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


# long requests, short ones, rows alone; many rows to an adapter and few
@pytest.mark.parametrize("lengths,count", [([90, 110], 2), ([12] * 24, 2), ([12] * 24, 24), ([1] * 40, 3)])
@pytest.mark.parametrize("rank", [8, 24, 40])
@pytest.mark.parametrize("k,n", [(320, 304), (301, 333)])
def test_products_of_float32(hkv, lengths, count, rank, k, n):
    tokens, requests = sum(lengths), len(lengths)
    at = torch.arange(tokens, device=DEV)
    offsets = torch.tensor([0, *lengths], device=DEV).cumsum(0)
    which = torch.arange(requests, device=DEV) % count
    a = which.repeat_interleave(torch.tensor(lengths, device=DEV))
    # a row of x and of dy has one number in a column of its own, a row of up one rank
    col, out = at * 13 % k, at * 11 % n
    assert len(set(col.tolist())) == len(set(out.tolist())) == tokens
    x, dy = torch.zeros((tokens, k), device=DEV), torch.zeros((tokens, n), device=DEV)
    x[at, col], dy[at, out] = _randn(1, tokens), _randn(2, tokens)
    down, up = _randn(3, count, rank, k), torch.zeros((count, n, rank), device=DEV)
    j = torch.arange(n, device=DEV)
    up[:, j, j % rank] = _randn(4, count, n)
    f = hkv.adapter_matmul(x, down, up, offsets, which)
    dx, ddown, dup = hkv.adapter_matmul_backward(f, dy)

    xs, ds = x.double()[at, col], dy.double()[at, out]
    d, u = down.double(), up.double()
    h = xs[:, None] * d[a, :, col]  # [tokens, rank]
    dh = ds[:, None] * u[a, out]
    want = {"out": h[:, j % rank] * u[a][:, j, j % rank], "dx": (dh[:, :, None] * d[a]).sum(1),
            "ddown": torch.zeros_like(d), "dup": torch.zeros_like(u)}
    want["ddown"][a, :, col] = dh * xs[:, None]
    want["dup"][a, out] = ds[:, None] * h
    bound = 2 * EACH + EACH ** 2
    for got, name in ((f.out, "out"), (dx, "dx"), (ddown, "ddown"), (dup, "dup")):
        off = (got.double() - want[name]).abs()
        worst = float((off / want[name].abs().clamp_min(1e-300)).max())
        assert bool((off <= bound * want[name].abs()).all()), f"{name}: {worst:.3g} of it, not {bound:.3g}"
