"""Page ids that no pool has, in a block table that is released: they are reported and never come back as a free page."""
import numpy as np
import pytest
import torch

from tests.test_gpu_pool import build

pytestmark = pytest.mark.gpu


# one block of the release's, and several whose shares hold some bad ids, none, or nothing else
@pytest.mark.parametrize("n,page,width,bad", [(1, 16, 3, "all"), (3, 16, 4, "one"), (40, 32, 20, "some"), (64, 16, 700, "some"),
                                              (64, 16, 700, "one"), (6, 64, 2200, "end"), (2500, 16, 3, "some"),
                                              (70, 16, 300, "all")], ids=str)
def test_bad_pages_are_left_out_of_the_stack(fcp, n, page, width, bad):
    r, m, pool, ints = build(fcp, n + width, n, page, width, 5)
    held = [(i, x) for i in range(n) for x in range(m.pages(m.lens[i]))]
    if bad == "some":
        at = [held[x] for x in r.choice(len(held), max(2, len(held) // 50), replace=False)]
    elif bad == "end":
        at = held[-3000:]
    else:
        at = held if bad == "all" else [held[len(held) // 2]]
    n_pages = pool.free_pages.numel()
    for j, (i, x) in enumerate(at):
        m.table[i][x] = [-1, n_pages, (1 << 31) - 1, -(1 << 31), 1 << 20][j % 5]
    pool.block_table.copy_(ints(m.table).view(n, width))
    keep = np.where(r.rand(n) < 0.2, -1, r.randint(0, width * page // 2 + 1, n)) if bad == "some" else np.zeros(n, int)
    m.release([int(x) for x in keep])
    lost = sum(not 0 <= x < n_pages for x in m.free)
    assert lost  # some of them are among what is given back
    m.free = [x for x in m.free if 0 <= x < n_pages]
    pool.release(ints(keep.tolist()))
    with pytest.raises(fcp.FcpError, match="0x51"):
        pool.check_device_error()
    assert pool.lens.tolist() == m.lens and pool.block_table.tolist() == m.table
    assert pool.n_free.item() == len(m.free) and pool.free_pages[:len(m.free)].tolist() == m.free
    # whoever takes pages next gets pages
    new = [min(max(width * page - x, 0), 3 * page) for x in m.lens]
    m.begin()
    want = m.admit(new, sum(new))
    slots = torch.zeros(sum(new), dtype=torch.int64, device="cuda")
    before = [list(row) for row in pool.block_table.tolist()]
    bad_left = any(not 0 <= before[i][x] < n_pages for i in range(n) for x in range(m.pages(m.lens[i] - want[0][i])))
    pool.admit(ints(new), None, slots)
    if not bad_left:  # a bad page that a sequence kept is reported again where its new tokens go there
        pool.check_device_error()
    assert pool.granted.tolist() == want[0] and pool.cu_new.tolist() == want[1]
    assert pool.block_table.tolist() == m.table
    # a release without a bad page, right after, is as ever
    pool.status[:1].zero_()
    keep = [m.lens[i] - want[0][i] for i in range(n)]
    m.release(keep)
    pool.release(ints(keep))
    pool.check_device_error()
    assert pool.lens.tolist() == m.lens and pool.block_table.tolist() == m.table
    assert pool.n_free.item() == len(m.free) and pool.free_pages[:len(m.free)].tolist() == m.free


def test_two_releases_in_one_graph(fcp):
    """What one call found is not the next one's: a bad page, and then none, replayed."""
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pool = fcp.PagePool(100, 16, 2, 40)
    first, second, new = ints([0, -1]), ints([0, 0]), ints([100, 50])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.release(first)
        pool.release(second)
    for lost in (1, 0, 2):
        height = int(pool.n_free)
        pool.admit(new, total_new=150)
        pool.check_device_error()
        for x in range(lost):
            pool.block_table[0, 3 * x] = -9
        graph.replay()
        if lost:
            with pytest.raises(fcp.FcpError, match="0x51"):
                pool.check_device_error()
        pool.check_device_error()
        assert int(pool.n_free) == height - lost
        free = pool.free_pages[:height - lost].tolist()
        assert len(set(free)) == len(free) and all(0 <= x < 100 for x in free)
        assert pool.lens.tolist() == [0, 0] and (pool.block_table == -1).all()
