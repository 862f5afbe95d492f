"""A server's step as one graph: pages given back and taken, q and k turned by their positions, k and v
written in 4 bits, the attention; and steps of several layers over one pool."""
import numpy as np
import pytest
import torch

from oracle import paged as R
from oracle import paged4 as R4
from oracle import rotary as RR
from tests import paged4_util as U

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float4_e2m1fn_x2, torch.float8_e4m3fn, torch.bfloat16], ids=["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("most", [4, 60], ids=["steps", "prompts"])
def test_a_servers_step_in_a_graph(fcp, dtype, most):
    hq, hkv, d, page, n, T, n_pages = 8, 2, 128, 16, 4, 64, 60
    four = dtype == torch.float4_e2m1fn_x2
    units = dict(k_unit=0.5, v_unit=2.0) if four else {}
    layers = [fcp.PagedCache(n_pages, page, hkv, d, dtype, **units) for _ in range(2)]
    pool, rot = fcp.PagePool(n_pages, page, n, 14), fcp.Rotary(64, base=500000.0, scaling=dict(kind="linear", factor=4.0))
    att = [fcp.PagedAttention(c, hq) for c in layers]
    batch = pool.batch(T, max_new=most)
    keep, new, positions, slots = ints([-1] * n), ints([0] * n), ints([7] * T), torch.full((T,), 7, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(h):
        return torch.zeros(h, T, d, dtype=torch.bfloat16, device="cuda")

    q, k, v, turned, o = ([rows(h) for _ in layers] for h in (hq, hkv, hkv, hq, hq))
    lse = [torch.zeros(hq, T, device="cuda") for _ in layers]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.release(keep)
        pool.admit(new, positions, slots)
        for i, cache in enumerate(layers):
            fcp.rotary_write(cache, batch, rot, q[i], k[i], v[i], turned[i])
            att[i].forward(batch, turned[i], o[i], lse[i])
    steps = [([-1] * n, [10, 0, 50, 4]), ([-1] * n, [4, 3, 1, 0]), ([12, -1, 50, 0], [1, 4, 4, 2]), ([0, 2, -1, -1], [4, 1, 0, 3])]
    for kp, nw in steps:
        nw = [min(x, most) for x in nw]
        keep.copy_(ints(kp))
        new.copy_(ints(nw))
        for x in (*q, *k, *v):
            x.normal_(generator=g)
        graph.replay()
        pool.check_device_error()
        assert pool.granted.tolist() == nw
        total = sum(nw)
        pos, slot = positions.cpu().numpy(), slots.cpu().numpy()
        assert (pos[total:] == -1).all() and (slot[total:] == -1).all()
        table, lens = pool.block_table.cpu().numpy(), pool.lens.tolist()
        for i, cache in enumerate(layers):
            cache.check_device_error()
            want, size = RR.turn(q[i][:, :total].double().cpu().numpy(), pos[:total], rot.radians, rot.magnitude, False)
            err = np.abs(turned[i][:, :total].double().cpu().numpy() - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size).all()
            pages = []
            for x, unit in (("k", 0.5), ("v", 2.0)):
                p, s = getattr(cache, x + "_pages"), getattr(cache, x + "_scales")
                if four:
                    y = U.values(p, s, unit)
                else:
                    y = p.double().cpu().numpy() * (1 if s is None else s.double().cpu().numpy()[..., None])
                pages.append(y)
            # the rows at the slots are v as the cache's definition keeps it
            rows_v = v[i][:, :total].double().cpu().numpy()
            at = pages[1][slot[:total] // page, :, slot[:total] % page].swapaxes(0, 1)
            if four:
                assert np.array_equal(at, R4.value(*R4.quantise(rows_v, 2.0), 2.0))
            elif dtype == torch.bfloat16:
                assert np.array_equal(at, rows_v)
            row = 0
            for j, x in enumerate(nw):
                for h in range(hq if x else 0):
                    p = np.arange(lens[j])
                    kk, vv = (y[table[j, p // page], h // 4, p % page] for y in pages)
                    ro, _, spread, _, _ = R.attend(turned[i][h, row:row + x].double().cpu().numpy(), kk, vv, x, True)
                    err = np.abs(o[i][h, row:row + x].double().cpu().numpy() - ro)
                    assert (err <= 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread).all()
                row += x


def test_two_steps_at_once_on_two_streams(fcp):
    """Two servers' steps, each with a pool, caches and an attention of its own, side by side: the same as one
    after the other."""
    hq, hkv, d, page, n, T = 8, 2, 64, 32, 40, 300
    rot = fcp.Rotary(64)

    def server(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache, pool = fcp.PagedCache(900, page, hkv, d, torch.float4_e2m1fn_x2), fcp.PagePool(900, page, n, 40)
        att, batch = fcp.PagedAttention(cache, hq), pool.batch(T, max_new=20)
        q, k, v = ([torch.randn(h, T, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(12)] for h in (hq, hkv, hkv))
        new = [torch.randint(0, 8, (n,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32) for _ in range(12)]
        keep = torch.full((n,), 60, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()

        def step(i):
            pool.release(keep)
            pool.admit(new[i], total_new=T)
            turned = fcp.rotary_write(cache, batch, rot, q[i], k[i], v[i])
            return att.forward(batch, turned, torch.zeros_like(turned), torch.zeros(hq, T, device="cuda"))

        return step, pool, cache

    streams = [torch.cuda.Stream() for _ in range(2)]
    servers, outs = [server(s) for s in (1, 2)], [[], []]
    for i in range(12):
        for s, (step, _, _) in enumerate(servers):
            with torch.cuda.stream(streams[s]):
                outs[s].append(step(i))
    torch.cuda.synchronize()
    for s, seed in enumerate((1, 2)):
        servers[s][1].check_device_error()
        servers[s][2].check_device_error()
        step, pool, _ = server(seed)
        for i in range(12):
            o, lse = step(i)
            total = int(pool.cu_new[-1])
            assert torch.equal(o[:, :total], outs[s][i][0][:, :total]) and torch.equal(lse[:, :total], outs[s][i][1][:, :total])


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_a_pool_and_frequencies_dropped_while_another_stream_works(fcp, kind):
    """What a pool and a Rotary allocated is not handed out again while a stream that their batch was used on has
    work left: here their memory is asked for and overwritten before that work has run."""
    hq, hkv, d, page, n, T = 4, 2, 64, 16, 50, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(h, T, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv, hkv))
    new = ints([2] * n)
    cache = fcp.PagedCache(200, page, hkv, d, torch.float4_e2m1fn_x2)
    att = fcp.PagedAttention(cache, hq)

    def begin():
        pool, rot = fcp.PagePool(200, page, n, 40), fcp.Rotary(d)
        pool.admit(new, total_new=T)
        torch.cuda.synchronize()
        return pool.batch(T, max_new=2), rot

    out = [[torch.zeros_like(q), torch.zeros_like(q), torch.zeros(hq, T, device="cuda")] for _ in range(2)]
    batch, rot = begin()
    fcp.rotary_write(cache, batch, rot, q, k, v, out[0][0])
    att.forward(batch, out[0][0], *out[0][1:])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side if kind == "stream" else side.cuda_stream
    batch, rot = begin()
    sizes = [x.numel() for x in (batch.lens, batch.cu_new, batch.block_table)] + [2 * rot.turns.numel()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e8))
    fcp.rotary_write(cache, batch, rot, q, k, v, out[1][0], stream=stream)
    att.forward(batch, out[1][0], *out[1][1:], stream=stream)
    del batch, rot
    junk = [torch.full((x,), 77, dtype=torch.int32, device="cuda") for x in sizes for _ in range(20)]
    torch.cuda.synchronize()
    cache.check_device_error()
    for x, y in zip(*out):
        assert torch.equal(x, y)
    del junk
