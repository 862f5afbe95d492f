"""The paged cache where its inputs are far from ordinary."""
import numpy as np
import pytest
import torch

from oracle import paged as R
from tests import paged_util as U
from tests.paged_util import Batch
from tests.test_gpu_paged import attend

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- NaN in V
NAN_V = [
    # position, batch (sequence 0 holds the NaN)
    (94, Batch([10, 10], [100, 100], hq=2, hkv=1)),                        # among the new tokens, few rows each
    (96, Batch([6, 1], [100, 40], hq=8, hkv=2, d=128, page=32)),
    (85, Batch([40, 40], [100, 100], hq=2, hkv=1)),                        # chunks
    (290, Batch([200, 33], [300, 290], hq=8, hkv=2, d=128, page=64)),      # several tiles and units
    (3, Batch([100, 100], [100, 100], hq=4, hkv=1, d=128)),
    (5960, Batch([70, 5], [6000, 300], hq=4, hkv=1, page=128)),            # keys split over many blocks
    (200, Batch([70, 90], [6000, 300], hq=4, hkv=1, d=128, page=128)),     # seen by every row, in another block
    (250, Batch([60, 60], [300, 300], hq=2, hkv=1, causal=False)),
    (127, Batch([50, 3], [160, 3], hq=2, hkv=1, max_new=1)),               # the other kernel than the batch asks for
    (0, Batch([2, 3], [2, 3], hq=2, hkv=1, max_new=90)),
]


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("at,b", NAN_V, ids=lambda x: str(x))
def test_a_nan_in_v_reaches_its_readers(fcp, at, b, c):
    """A NaN row of V makes o of every row that sees it NaN and leaves lse as it is. Other sequences keep
    every bit, and in an e4m3 cache so do the rows that do not see it, whichever kernel runs."""
    b = Batch(**{**b.__dict__, "cache": c, "seed": at})
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    want = attend(fcp, b, t, cache, batch)
    for p in {at, max(at - 1, 0)}:  # one bad row, then two beside one another
        page, off = int(t["table"][0, p // b.page]), p % b.page
        if c == "bf16":
            t["v_pages"][page, :, off, 7] = float("nan")
        else:
            t["v_scales"].view(torch.uint8)[page, :, off] = 255
    first = max(at - 1, 0)
    o, lse, _ = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    n, length = b.new[0], b.lens[0]
    sees = (torch.arange(n) + length - n >= first).cuda() if b.causal else torch.ones(n, dtype=torch.bool, device="cuda")
    assert torch.equal(lse, want[1])
    assert torch.equal(o[:, n:], want[0][:, n:])
    if c == "bf16":  # rows before it: documented as not kept apart; other channels are not touched
        assert o[:, :n, 7][:, sees].isnan().all()
        keep = torch.arange(b.d, device="cuda") != 7
        assert torch.equal(o[:, :n][..., keep], want[0][:, :n][..., keep])
    else:
        assert o[:, :n][:, sees].isnan().all()
        assert torch.equal(o[:, :n][:, ~sees], want[0][:, :n][:, ~sees])


# ---------------------------------------------------------------- V's scales far apart
@pytest.mark.parametrize("new", [1, 2, 3, 8, 50], ids=lambda n: f"new{n}")
@pytest.mark.parametrize("apart", [6, 11, 18, 24, 40, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_small_rows_of_v_beside_large_ones(fcp, new, apart, d):
    """Every ninth row of V is 2^apart larger than the rest, and zero but for one channel: the other
    channels are sums over the small rows alone, which must not be lost beside it."""
    b = Batch([new, 1], [300, 77], hq=4, hkv=1, d=d, page=32, cache="e4m3", seed=apart)
    t = U.make(b)
    codes, byte = t["v_pages"].view(torch.uint8), t["v_scales"].view(torch.uint8)
    large = torch.zeros_like(byte, dtype=torch.bool)
    large[:, :, 4::9] = True
    large &= byte != 255
    byte.copy_(torch.where(large, 117 + apart // 2, torch.where(byte == 255, 255, byte - (apart + 1) // 2)).to(torch.uint8))
    codes.masked_fill_(large[..., None] & (torch.arange(d, device="cuda") != 5), 0)
    cache, batch = U.handles(fcp, b, t)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)


# ---------------------------------------------------------------- offsets that fall back
BROKEN = [
    # cu, total, the sequences that own rows
    ([0, 2, 5, 1000, 8, 10], 10, [0, 1, 4]),
    ([0, 9, 2, 4, 3], 8, [2]),
    ([5, 7, 1, 3, 900, 7, 9], 9, [0, 2, 5]),
    ([-4, 5, 7, 2, 2, 5, 99], 7, [1, 4]),
]


def _broken(c, cu, total, owners, many, seed=0):
    """A batch of len(cu) - 1 sequences with these offsets; many: that many empty sequences more in front
    and behind, so that offsets are searched in two steps."""
    n = len(cu) - 1
    new = [max(0, cu[i + 1] - cu[i]) if 0 <= cu[i] <= cu[i + 1] <= total else 0 for i in range(n)]
    b = Batch([0] * many + new + [0] * many, [20 + i % 30 for i in range(n + 2 * many)], hq=2, hkv=2, cache=c, seed=seed)
    t = U.make(b)
    t["cu"] = torch.tensor([cu[0]] * many + cu + [cu[-1]] * many, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(seed)
    for x, h in (("q", b.hq), ("k", b.hkv), ("v", b.hkv)):
        t[x] = torch.randn(h, total, b.d, generator=g).to(torch.bfloat16).cuda()
    cache = fcp_cache(t)
    return b, t, cache


def fcp_cache(t):
    import context_parallelism_fcp_gb300 as pkg

    return pkg.PagedCache.wrap(t["k_pages"], t["v_pages"], t["k_scales"], t["v_scales"])


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("many", [0, 700])
@pytest.mark.parametrize("cu,total,owners", BROKEN, ids=lambda x: None)
def test_rows_behind_a_bad_offset_are_written_and_read(fcp, cu, total, owners, many, c):
    """A bad offset in front of a good sequence: its rows are found, and every other byte stays."""
    b, t, cache = _broken(c, cu, total, owners, many)
    batch = fcp.CacheBatch(t["cu"], t["lens"], t["table"], total, max_new=total)
    table = t["table"].cpu().numpy()
    place = {}  # packed row -> page, row of the page
    for i in owners:
        n = cu[i + 1] - cu[i]
        for j in range(n):
            pos = b.lens[many + i] - n + j
            assert cu[i] + j not in place and pos >= 0
            place[cu[i] + j] = int(table[many + i, pos // b.page]), pos % b.page
    # read
    k, v = torch.full_like(t["k"], 3.0), torch.full_like(t["v"], -3.0)
    fcp.cache_read(cache, batch, k, v)
    with pytest.raises(fcp.FcpError, match="0x50"):
        cache.check_device_error()
    for got, fill, x in ((k, 3.0, "k"), (v, -3.0, "v")):
        stored = U.values(t[x + "_pages"], t[x + "_scales"])
        want = np.full(got.shape, fill)
        for row, (pg, off) in place.items():
            want[:, row] = stored[pg, :, off]
        assert np.array_equal(got.double().cpu().numpy(), want)
    # write
    names = [x for x in ("k_pages", "v_pages", "k_scales", "v_scales") if t[x] is not None]
    before = {x: t[x].clone() for x in names}
    fcp.cache_write(cache, batch, t["k"], t["v"])
    with pytest.raises(fcp.FcpError, match="0x50"):
        cache.check_device_error()
    for x in "kv":
        rows = t[x].cpu()
        if c == "bf16":
            want = before[x + "_pages"].view(torch.int16).cpu().clone()
            for row, (pg, off) in place.items():
                want[pg, :, off] = rows[:, row].view(torch.int16)
            assert torch.equal(t[x + "_pages"].view(torch.int16).cpu(), want)
        else:
            want, byte = (before[x + y].view(torch.uint8).cpu().numpy().copy() for y in ("_pages", "_scales"))
            for row, (pg, off) in place.items():
                for h in range(b.hkv):
                    want[pg, h, off], byte[pg, h, off] = R.quantise_row(rows[h, row].double().numpy())
            assert np.array_equal(t[x + "_pages"].view(torch.uint8).cpu().numpy(), want)
            assert np.array_equal(t[x + "_scales"].view(torch.uint8).cpu().numpy(), byte)


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_new", [1, 100], ids=["few", "chunk"])
@pytest.mark.parametrize("cu,total,owners", BROKEN, ids=lambda x: None)
def test_rows_behind_a_bad_offset_are_attended(fcp, cu, total, owners, max_new, c):
    """The same batches' attention: the good sequences' rows are theirs alone, others stay."""
    b, t, cache = _broken(c, cu, total, owners, 0)
    batch = fcp.CacheBatch(t["cu"], t["lens"], t["table"], total, max_new=max_new)
    b.pad = total - sum(b.new)  # the outputs have `total` rows
    o, lse, before = attend(fcp, b, t, cache, batch)
    with pytest.raises(fcp.FcpError, match="0x50"):
        cache.check_device_error()
    rest = torch.ones(total, dtype=torch.bool, device="cuda")
    for i in owners:
        a, e = cu[i], cu[i + 1]
        rest[a:e] = False
        one = Batch([e - a], [b.lens[i]], hq=b.hq, hkv=b.hkv, cache=c)
        u = dict(t, table=t["table"][i:i + 1], q=t["q"][:, a:e])
        U.check_attention(one, u, o[:, a:e], lse[:, a:e])
    assert torch.equal(o[:, rest], before[0][:, rest]) and torch.equal(lse[:, rest], before[1][:, rest])


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("page_id", [1 << 30, -1])
def test_pages_outside_the_cache(fcp, page_id, c):
    """Attention counts the keys of a page outside the cache as zeros, in K and in V; a write and a read
    leave their rows out; the rest of the batch is what it was."""
    b = Batch([3, 40, 2], [70, 80, 33], hq=4, hkv=2, cache=c, pad=2)
    t = U.make(b)
    bad = [(0, 1), (1, 4), (2, 2)]  # sequence, entry: the second holds new tokens of its own
    held = dict(t)
    for x in ("k_pages", "v_pages"):
        held[x] = torch.cat([t[x].view(torch.uint8 if c == "e4m3" else torch.bfloat16),
                             torch.zeros_like(t[x][:1].view(torch.uint8 if c == "e4m3" else torch.bfloat16))]).view(t[x].dtype)
        if c == "e4m3":
            y = x[0] + "_scales"
            held[y] = torch.cat([t[y].view(torch.uint8), torch.full_like(t[y][:1].view(torch.uint8), 127)]).view(t[y].dtype)
    zero = t["k_pages"].shape[0]  # a page of zeros that the oracle looks at in their place
    table = t["table"].clone()
    held["table"] = t["table"].clone()
    for i, e in bad:
        table[i, e] = page_id
        held["table"][i, e] = zero
    t["table"] = table
    cache = fcp_cache(t)
    for max_new in (1, 100):
        batch = fcp.CacheBatch(t["cu"], t["lens"], t["table"], b.total, max_new=max_new)
        o, lse, before = attend(fcp, b, t, cache, batch)
        with pytest.raises(fcp.FcpError, match="0x51"):
            cache.check_device_error()
        U.check_attention(b, held, o, lse, *before)
    places = [x for x in R.places(b.new, b.lens, table.cpu().numpy(), b.page) if 0 <= x[3] < zero]
    assert 0 < len(places) < sum(b.new)
    k, v = torch.full_like(t["k"], 3.0), torch.full_like(t["v"], -3.0)
    fcp.cache_read(cache, batch, k, v)
    with pytest.raises(fcp.FcpError, match="0x51"):
        cache.check_device_error()
    for got, fill, x in ((k, 3.0, "k"), (v, -3.0, "v")):
        stored, want = U.values(t[x + "_pages"], t[x + "_scales"]), np.full(got.shape, fill)
        for row, _, _, pg, off in places:
            want[:, row] = stored[pg, :, off]
        assert np.array_equal(got.double().cpu().numpy(), want)
    names = [x for x in ("k_pages", "v_pages", "k_scales", "v_scales") if t[x] is not None]
    before = {x: t[x].clone() for x in names}
    fcp.cache_write(cache, batch, t["k"], t["v"])
    with pytest.raises(fcp.FcpError, match="0x51"):
        cache.check_device_error()
    written = torch.zeros(t["k_pages"].shape[0], b.page, dtype=torch.bool)
    for _, _, _, pg, off in places:
        written[pg, off] = True
    for x in names:
        raw = lambda y: y.view(torch.int16 if y.element_size() == 2 else torch.uint8).transpose(1, 2).cpu()  # noqa: E731
        now, old = raw(t[x]), raw(before[x])
        assert torch.equal(now[~written], old[~written]), x
    fcp.cache_read(cache, batch, k, v)
    with pytest.raises(fcp.FcpError, match="0x51"):
        cache.check_device_error()
    for row, *_ in places:
        if c == "bf16":
            assert torch.equal(k[:, row], t["k"][:, row]) and torch.equal(v[:, row], t["v"][:, row])
        else:
            for got, x in ((k, t["k"]), (v, t["v"])):
                for h in range(b.hkv):
                    codes, byte = R.quantise_row(x[h, row].double().cpu().numpy())
                    assert np.array_equal(got[h, row].double().cpu().numpy(), R.row_value(codes, byte))


# ---------------------------------------------------------------- idle sequences
@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40], ids=["few", "chunk"])
def test_thousands_of_idle_sequences(fcp, c, new):
    """Busy sequences before, between and behind 30000 idle ones each: right, and in a time that is not that
    of reading them one after another in one thread (100 ns each: 3 ms)."""
    gap = 30000
    new_, lens = [new, 0, new, 0, new], [300, 0, 700, 0, 20 + new]
    b = Batch(new_, lens, hq=4, hkv=2, d=128, cache=c, seed=new)
    t = U.make(b)
    busy = [0, gap + 1, 2 * gap + 2]
    n = 2 * gap + 3
    table = torch.full((n, t["table"].shape[1]), -7, dtype=torch.int32, device="cuda")
    lens_all = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    count = torch.zeros(n, dtype=torch.int32, device="cuda")
    for at, i in zip(busy, (0, 2, 4)):
        table[at], lens_all[at], count[at] = t["table"][i], t["lens"][i], new
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).int()
    cache = fcp_cache(t)
    batch = fcp.CacheBatch(cu, lens_all, table, b.total, max_new=new)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)
    att, times = fcp.PagedAttention(cache, b.hq), []
    for _ in range(4):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        torch.cuda.synchronize()
        start.record()
        att.forward(batch, t["q"], o, lse)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert min(times) < 1.5, times


# ---------------------------------------------------------------- streams
def _busy(stream, seconds=0.05):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(2e9 * seconds))


@pytest.mark.parametrize("kind", ["stream", "current", "handle", "external"])
def test_objects_dropped_while_another_stream_works(fcp, kind):
    """A cache and an attention made on one stream, used on another and dropped at once: their memory is not
    handed out while the work is under way."""
    b = Batch([1, 2], [3000, 700], hq=8, hkv=2, d=128)
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    want = fcp.PagedAttention(cache, b.hq).forward(batch, t["q"])
    o, lse = torch.zeros_like(t["q"]), torch.zeros(b.hq, b.total, device="cuda")
    cache = fcp.PagedCache(*t["k_pages"].shape[:1], b.page, b.hkv, b.d)
    cache.k_pages.copy_(t["k_pages"])
    cache.v_pages.copy_(t["v_pages"])
    att = fcp.PagedAttention(cache, b.hq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = torch.cuda.ExternalStream(side.cuda_stream) if kind == "external" else side
    _busy(side)
    if kind == "current":
        with torch.cuda.stream(side):
            att.forward(batch, t["q"], o, lse)
    else:
        att.forward(batch, t["q"], o, lse, stream=side.cuda_stream if kind == "handle" else other)
    mine = {x.data_ptr() for x in (att.workspace, cache.status, cache.k_pages, cache.v_pages)}
    n, pages = att.workspace.numel(), cache.k_pages.numel()
    del cache, att
    over = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    over += [torch.empty(pages, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    over += [torch.empty(64, dtype=torch.int32, device="cuda") for _ in range(8)]
    if not side.query():
        assert not mine & {x.data_ptr() for x in over}
    else:  # an object used on a stream of unknown life waits for the device when it is dropped
        assert kind in ("handle", "external")
    for x in over:
        x.view(torch.uint8).fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_objects_made_on_a_busy_stream(fcp):
    """Memory that the first stream has yet to write (a dropped tensor's, a new cache's zeros) is not used by
    another stream before that is done."""
    b = Batch([1, 2], [3000, 700], hq=8, hkv=2, d=128, page=64)
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    want = fcp.PagedAttention(cache, b.hq).forward(batch, t["q"])
    whole = fcp.CacheBatch(torch.tensor([0, 3000, 3700], dtype=torch.int32).cuda(), t["lens"], t["table"], 3700, max_new=3000)
    k, v = (torch.empty(2, 3700, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fcp.cache_read(cache, whole, k, v)
    o, lse = torch.zeros_like(t["q"]), torch.zeros(b.hq, b.total, device="cuda")
    n = fcp.lib().fcp_paged_attn_workspace_bytes(b.d)
    torch.cuda.synchronize()
    first, side = torch.cuda.current_stream(), torch.cuda.Stream()
    dropped = torch.empty(n, dtype=torch.uint8, device="cuda")
    _busy(first)
    dropped.fill_(255)
    del dropped
    other = fcp.PagedCache(cache.n_pages, b.page, b.hkv, b.d)
    att = fcp.PagedAttention(other, b.hq)
    with torch.cuda.stream(side):
        fcp.cache_write(other, whole, k, v)
        att.forward(batch, t["q"], o, lse)
    torch.cuda.synchronize()
    other.check_device_error()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_objects_made_inside_a_capture(fcp):
    """Nothing in making a cache or an attention stops a capture, and a graph replays with them."""
    b = Batch([1, 40], [300, 70], hq=4, hkv=2, d=64)
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    want = fcp.PagedAttention(cache, b.hq).forward(batch, t["q"])
    o, lse = torch.zeros_like(t["q"]), torch.zeros(b.hq, b.total, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = fcp.PagedCache.wrap(t["k_pages"], t["v_pages"])
        att = fcp.PagedAttention(again, b.hq)
        att.forward(batch, t["q"], o, lse)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    again.check_device_error()
