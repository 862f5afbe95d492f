"""The page pool against its definition, one sequence at a time in Python."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


class Model:
    """What fcp_page_pool says, in lists."""

    def __init__(self, free, lens, table, page):
        self.free, self.lens, self.table, self.page = list(free), list(lens), [list(r) for r in table], page

    def pages(self, n):
        return -(-n // self.page)

    def release(self, keep):
        for i, k in enumerate(keep):
            left = min(self.lens[i], k) if k >= 0 else self.lens[i]
            for x in range(self.pages(left), self.pages(self.lens[i])):
                self.free.append(self.table[i][x])
                self.table[i][x] = -1
            self.lens[i] = left

    def admit(self, new, total):
        granted, cu, rows, slots, positions = [], [0], 0, [-1] * total, [-1] * total
        no_pages = no_rows = False
        wanted = 0  # pages of every sequence so far that could have them
        for i, n in enumerate(new):
            need = self.pages(self.lens[i] + n) - self.pages(self.lens[i])
            if self.pages(self.lens[i] + n) > len(self.table[i]) or n < 0:
                n = need = 0
            wanted += need
            no_pages = no_pages or wanted > self.n_free0
            if need and no_pages:
                n = 0
            if n and (no_rows or rows + n > total):
                no_rows, n = True, 0
            for j in range(n):
                p = self.lens[i] + j
                if p % self.page == 0:
                    self.table[i][p // self.page] = self.free.pop()
                positions[rows + j] = p
                slots[rows + j] = self.table[i][p // self.page] * self.page + p % self.page
            self.lens[i] += n
            rows += n
            granted.append(n)
            cu.append(rows)
        return granted, cu, positions, slots

    @property
    def n_free0(self):
        return self._n0

    def begin(self):
        self._n0 = len(self.free)


def build(fcp, seed, n, page, width, spare, n_pages=None):
    r = np.random.RandomState(seed)
    lens = [int(x) for x in r.randint(0, width * page + 1, n)]
    held = [-(-x // page) for x in lens]
    n_pages = sum(held) + spare if n_pages is None else n_pages
    ids = list(map(int, r.permutation(n_pages)))
    table = []
    for h in held:
        table.append([ids.pop() for _ in range(h)] + [-1] * (width - h))
    m = Model(ids, lens, table, page)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pool = fcp.PagePool.wrap(ints(ids + [-5] * (n_pages - len(ids))), ints([len(ids)]), ints(lens),
                             ints(table).view(n, width), page)
    return r, m, pool, ints


def same(pool, m):
    pool.check_device_error()
    assert pool.lens.tolist() == m.lens
    assert pool.n_free.item() == len(m.free)
    assert pool.free_pages[:len(m.free)].tolist() == m.free
    assert pool.block_table.tolist() == m.table


CASES = [(1, 16, 3, 2, 8), (5, 16, 4, 0, 40), (128, 64, 9, 40, 700), (300, 16, 130, 900, 5000), (1030, 32, 2, 50, 3000),
         (2500, 16, 3, 300, 2100), (70, 4096, 2, 5, 9000), (7, 16, 700, 100, 1024),
         (6, 64, 2200, 9000, 400000)]


@pytest.mark.parametrize("n,page,width,spare,total", CASES, ids=str)
def test_a_run_of_steps(fcp, n, page, width, spare, total):
    """Admissions and releases in turn, with sequences that wait, end, are cut back inside a page or do not fit:
    too few pages, too few rows, too short a row of the table."""
    r, m, pool, ints = build(fcp, n + page, n, page, width, spare)
    positions, slots = ints([9] * total), torch.full((total,), 9, dtype=torch.int64).cuda()
    for step in range(6):
        new = r.choice([0, 1, 1, 3, 17, 2 * page, width * page], n, p=[.2, .3, .2, .1, .1, .05, .05]) if step % 2 else r.randint(0, 3, n)
        if step == 4:
            new[n // 2] = (1 << 31) - 1  # more than any row holds
        m.begin()
        want = m.admit([int(x) for x in new], total)
        pool.admit(ints(new.tolist()), positions, slots)
        assert pool.granted.tolist() == want[0]
        assert pool.cu_new.tolist() == want[1]
        assert positions.tolist() == want[2]
        assert slots.tolist() == want[3]
        same(pool, m)
        keep = np.where(r.rand(n) < 0.3, -1, np.maximum(0, np.array(m.lens) - r.randint(0, 2 * page, n)))
        keep[r.rand(n) < 0.2] = 0
        if step == 2:
            keep[:] = (1 << 31) - 1  # nothing to cut
        if step == 5:
            keep[:] = 0
        m.release([int(x) for x in keep])
        pool.release(ints(keep.tolist()))
        same(pool, m)
    assert m.lens == [0] * n


def test_one_launch_without_outputs_and_empty_pools(fcp):
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    pool = fcp.PagePool(10, 16, 3, 4)
    pool.admit(ints([17, 0, 1]), total_new=18)
    assert pool.block_table.tolist() == [[0, 1, -1, -1], [-1] * 4, [2, -1, -1, -1]] and pool.cu_new.tolist() == [0, 17, 17, 18]
    pool.admit(ints([1, 0, 0]), total_new=0)  # no row for it
    assert pool.granted.tolist() == [0, 0, 0] and pool.lens.tolist() == [17, 0, 1] and pool.cu_new.tolist() == [0] * 4
    pool.release(ints([0, 0, 0]))
    assert pool.n_free.item() == 10 and pool.free_pages[-3:].tolist() == [0, 1, 2]
    empty = fcp.PagePool(0, 16, 2, 0)
    rows = ints([3, 3])
    empty.admit(ints([1, 0]), rows)
    empty.release(ints([0, 0]))
    assert empty.granted.tolist() == [0, 0] and rows.tolist() == [-1, -1]
    none = fcp.PagePool(4, 16, 0, 3)
    none.admit(ints([]), rows)
    none.release(ints([]))
    assert none.cu_new.tolist() == [0] and rows.tolist() == [-1, -1]
    for p in (pool, empty, none):
        p.check_device_error()


def test_broken_state_is_reported_and_nothing_else_touched(fcp):
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for what, code in (("len", 0x50), ("long", 0x50), ("new", 0x50), ("free", 0x50), ("low", 0x50), ("page", 0x51)):
        pool = fcp.PagePool(8, 16, 3, 2)
        pool.admit(ints([20, 20, 5]), total_new=64)
        new = [1, 1, 14]
        if what == "len":
            pool.lens[1] = -4
        elif what == "long":
            pool.lens[1] = 33
        elif what == "new":
            new[1] = -1
        elif what == "free":
            pool.n_free.fill_(9)
        elif what == "low":
            pool.n_free.fill_(-1)
        else:
            pool.free_pages[int(pool.n_free) - 1] = 8
        table = pool.block_table.clone()
        pool.admit(ints(new), total_new=64)
        with pytest.raises(fcp.FcpError, match=hex(code)):
            pool.check_device_error()
        pool.check_device_error()  # read and cleared
        if what in ("free", "low"):  # no page is handed out
            assert pool.granted.tolist() == [1, 1, 0] and torch.equal(pool.block_table, table)
        elif what == "page":
            assert pool.granted.tolist() == [1, 1, 14]
        else:
            assert pool.granted.tolist() == [1, 0, 14] and torch.equal(pool.block_table[:2], table[:2])
    # a release that would pass the pool's size gives nothing back; one of a bad length leaves it out
    pool = fcp.PagePool(8, 16, 3, 2)
    pool.admit(ints([20, 20, 5]), total_new=64)
    pool.n_free.fill_(6)
    before = pool.block_table.clone(), pool.lens.clone()
    pool.release(ints([0, 0, 0]))
    with pytest.raises(fcp.FcpError, match="0x50"):
        pool.check_device_error()
    assert torch.equal(pool.block_table, before[0]) and torch.equal(pool.lens, before[1]) and pool.n_free.item() == 6
    pool.n_free.fill_(3)
    pool.lens[0] = 99
    pool.release(ints([0, 0, 0]))
    with pytest.raises(fcp.FcpError, match="0x50"):
        pool.check_device_error()
    assert pool.lens.tolist() == [99, 0, 0] and pool.n_free.item() == 6
    pool.block_table[0, 0] = 77
    pool.lens[0] = 20
    pool.release(ints([0, 0, 0]))
    with pytest.raises(fcp.FcpError, match="0x51"):
        pool.check_device_error()


def test_captured_steps(fcp):
    """A release and an admission in one graph: each replay goes on from where the last one ended, on whatever
    `keep` and `new` hold then, on a stream that the pool was not made on."""
    n, total = 40, 300
    r, m, pool, ints = build(fcp, 3, n, 16, 20, 400)
    keep, new = ints([-1] * n), ints([0] * n)
    positions, slots = ints([0] * total), torch.zeros(total, dtype=torch.int64).cuda()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pool.release(keep)
        pool.admit(new, positions, slots)
    for _ in range(5):
        k = [int(x) for x in np.where(r.rand(n) < 0.4, 0, r.randint(0, 200, n))]
        w = [int(x) for x in r.randint(0, 14, n)]
        keep.copy_(ints(k))
        new.copy_(ints(w))
        graph.replay()
        m.release(k)
        m.begin()
        want = m.admit(w, total)
        assert (pool.granted.tolist(), pool.cu_new.tolist(), positions.tolist(), slots.tolist()) == want
        same(pool, m)


def test_pool_cache_and_attention_together(fcp):
    """A server's steps over a 4-bit cache: a prompt in chunks, drafts of which some are refused, an end and a
    new beginning. The attention is that over what the cache holds."""
    from oracle import paged as R
    from tests import paged4_util as U

    hq, hkv, d, page, n, T = 4, 2, 64, 16, 3, 64
    g = torch.Generator().manual_seed(0)
    cache = fcp.PagedCache(30, page, hkv, d, torch.float4_e2m1fn_x2, v_unit=0.5)
    pool, att = fcp.PagePool(30, page, n, 9), fcp.PagedAttention(cache, hq)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    batch = pool.batch(T, max_new=50)
    for keep, new in (([-1] * 3, [50, 0, 14]), ([-1] * 3, [13, 40, 1]), ([61, 38, 15], [4, 4, 0]), ([0, -1, 10], [30, 1, 1])):
        pool.release(ints(keep))
        pool.admit(ints(new), total_new=T)
        q, k, v = (torch.randn(h, T, d, generator=g).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
        fcp.cache_write(cache, batch, k, v)
        o, _ = att.forward(batch, q)
        pool.check_device_error()
        cache.check_device_error()
        assert pool.granted.tolist() == new
        kp, vp = (U.values(p, s, u) for p, s, u in ((cache.k_pages, cache.k_scales, 1.0), (cache.v_pages, cache.v_scales, 0.5)))
        table, lens, row = pool.block_table.cpu().numpy(), pool.lens.tolist(), 0
        for i, x in enumerate(new):
            for h in range(hq if x else 0):
                pos = np.arange(lens[i])
                kk, vv = (y[table[i, pos // page], h // 2, pos % page] for y in (kp, vp))
                ro, _, spread, _, _ = R.attend(q[h, row:row + x].double().cpu().numpy(), kk, vv, x, True)
                err = np.abs(o[h, row:row + x].double().cpu().numpy() - ro)
                assert (err <= 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread).all()
            row += x
