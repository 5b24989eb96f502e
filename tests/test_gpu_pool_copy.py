"""Slots copied inside pools: every width of access, sizes, skipped pairs, many pools."""
import pytest
import torch

import gated_delta_rule_gdn_amd as g

pytestmark = pytest.mark.gpu


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def bytes_of(gen, *shape, dtype=torch.uint8):
    n = torch.empty(shape, dtype=dtype).element_size() * torch.Size(shape).numel()
    return torch.randint(0, 256, (n,), generator=gen, dtype=torch.uint8).view(dtype).view(shape).cuda()


def run(pools, src, dst):
    src, dst = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (src, dst))
    want = [t.clone() for t in pools]
    for a, b in zip(src.tolist(), dst.tolist()):
        for w, p in zip(want, pools):
            if 0 <= a < len(p) and 0 <= b < len(p):
                w[b] = p[a]
    g.pool_copy(pools, src, dst)
    assert all(torch.equal(p.view(torch.uint8), w.view(torch.uint8)) for p, w in zip(pools, want))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 8, 15, 16, 17, 48, 255, 256, 1000, 1024, 4095, 4096, 4112, 16384, 16400,
                               65537, 131072])
def test_slot_sizes(n):
    gen = torch.Generator().manual_seed(n)
    run([bytes_of(gen, 9, n)], [0, 3, 3, 8], [5, 1, 7, 2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int8, torch.float64])
def test_types_and_shapes(dtype):
    gen = torch.Generator().manual_seed(1)
    run([bytes_of(gen, 6, 3, 5, dtype=dtype), bytes_of(gen, 6, 64, dtype=dtype)], [0, 4], [3, 5])


def test_pools_at_odd_addresses():
    gen = torch.Generator().manual_seed(2)
    raw = bytes_of(gen, 7 * 64 + 9)
    for at in (1, 2, 4, 8, 9):
        run([raw[at:at + 7 * 64].view(7, 64)], [6, 0], [1, 2])


def test_pairs_outside_the_pool_are_skipped():
    gen = torch.Generator().manual_seed(3)
    run([bytes_of(gen, 5, 640)], [-1, 0, 5, 1, 2 ** 31 - 1, 2, -2 ** 31], [3, 5, 0, -1, 4, 2, 2 ** 31 - 1])


def test_one_source_many_destinations():
    gen = torch.Generator().manual_seed(4)
    run([bytes_of(gen, 40, 272)], [7] * 30, list(range(8, 38)))


@pytest.mark.parametrize("pools", [1, 63, 64, 65, 130])
def test_many_pools_of_different_sizes(pools):
    gen = torch.Generator().manual_seed(pools)
    run([bytes_of(gen, 4, 16 * (1 + 37 * i % 11)) for i in range(pools)], [1, 2], [0, 3])


def test_many_pairs():
    """More pairs than one dimension of the grid takes."""
    gen = torch.Generator().manual_seed(5)
    n = 40000
    order = torch.randperm(2 * n, generator=gen)
    pool = bytes_of(gen, 2 * n, 20)
    src, dst = order[:n].to(torch.int32).cuda(), order[n:].to(torch.int32).cuda()
    want = pool.clone()
    want[dst.long()] = pool[src.long()]
    g.pool_copy(pool, src, dst)
    assert torch.equal(pool, want)


def test_slots_beyond_four_gigabytes():
    pool = torch.zeros(5, (1 << 30) + 4, dtype=torch.uint8, device="cuda")
    pool[4, -1], pool[4, 0], pool[4, 1 << 29] = 7, 8, 9
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g.pool_copy(pool, i(4), i(3))
    assert torch.equal(pool[3], pool[4]) and not pool[:3].any()


def test_more_pieces_than_a_grid_dimension_takes():
    """A slot of 2^20 workgroups and a few, byte by byte, in a pool beside a small one."""
    n = (1 << 29) + 1539
    pool = torch.zeros(2, n, dtype=torch.uint8, device="cuda")
    pool[0, :1000], pool[0, -1000:], pool[0, 1 << 28] = 3, 5, 7
    small = torch.tensor([[1, 2, 3], [4, 5, 6]], dtype=torch.uint8, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g.pool_copy([pool, small], i(0), i(1))
    assert torch.equal(pool[1], pool[0]) and torch.equal(small[1], small[0])


def test_nothing_to_do():
    gen = torch.Generator().manual_seed(6)
    pool = bytes_of(gen, 3, 16)
    want = pool.clone()
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    g.pool_copy(pool, i, i.clone())
    g.pool_copy([], i, i.clone())
    g.pool_copy(torch.zeros(0, 8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                torch.ones(1, dtype=torch.int32, device="cuda"))
    g.pool_copy(torch.zeros(3, 0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                torch.ones(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(pool, want)


def test_refusals():
    pool = torch.zeros(4, 8, device="cuda")
    i = torch.tensor([0], dtype=torch.int32, device="cuda")
    j = torch.tensor([1], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        g.pool_copy([pool, torch.zeros(5, 8, device="cuda")], i, j)
    with pytest.raises(ValueError):
        g.pool_copy(pool.t(), i, j)
    with pytest.raises(TypeError):
        g.pool_copy(pool, i.long(), j.long())
    with pytest.raises(ValueError):
        g.pool_copy(pool, i, torch.cat((j, j)))
    with pytest.raises(g.GDN2Error):
        g.pool_copy([pool, pool], i, j)
    with pytest.raises(ValueError):
        g.pool_copy(torch.zeros(4, 8), i, j)
