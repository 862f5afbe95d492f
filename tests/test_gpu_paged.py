"""The paged cache and its attention against the float64 definitions (oracle/paged.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged as R
from tests import paged_util as U
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- write and read
MOVES = [
    Batch([1], [1]),
    Batch([3, 0, 17, 1], [3, 40, 33, 64], pad=2),
    Batch([5, 2, 64], [4, 1, 64], hkv=3, hq=3, page=32, d=128),          # tokens before position 0 are left out
    Batch([1] * 70, list(range(1, 71)), hkv=1, hq=1, page=64, d=128),
    Batch([129, 1], [300, 1], hkv=5, hq=5, d=128, page=128, pad=1),
    Batch([0, 0, 7], [0, 3, 7], page=256),
]
MOVES = [b.__class__(**{**b.__dict__, "cache": c}) for b in MOVES for c in ("bf16", "e4m3")]


@pytest.mark.parametrize("b", MOVES, ids=str)
def test_write_stores_the_definition_and_nothing_else(fcp, b):
    t = U.make(b)
    before = {x: t[x].clone() for x in ("k_pages", "v_pages", "k_scales", "v_scales") if t[x] is not None}
    cache, batch = U.handles(fcp, b, t)
    fcp.cache_write(cache, batch, t["k"], t["v"])
    cache.check_device_error()
    table = t["table"].cpu().numpy()
    for x in "kv":
        pages, rows = t[x + "_pages"], t[x].cpu()
        if b.cache == "bf16":
            want = before[x + "_pages"].view(torch.int16).cpu().clone()
            for row, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
                want[pg, :, off] = rows[:, row].view(torch.int16)
            assert torch.equal(pages.view(torch.int16).cpu(), want)
        else:
            want, byte = (before[x + y].view(torch.uint8).cpu().numpy().copy() for y in ("_pages", "_scales"))
            for row, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
                for h in range(b.hkv):
                    want[pg, h, off], byte[pg, h, off] = R.quantise_row(rows[h, row].double().numpy())
            assert np.array_equal(pages.view(torch.uint8).cpu().numpy(), want)
            assert np.array_equal(t[x + "_scales"].view(torch.uint8).cpu().numpy(), byte)


@pytest.mark.parametrize("b", MOVES, ids=str)
def test_read_returns_the_stored_values(fcp, b):
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    k, v = torch.full_like(t["k"], 7.0), torch.full_like(t["v"], -7.0)
    before = k.clone(), v.clone()
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    table = t["table"].cpu().numpy()
    for got, old, x in ((k, before[0], "k"), (v, before[1], "v")):
        want = old.double().cpu().numpy()
        stored = U.values(t[x + "_pages"], t[x + "_scales"])
        for row, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
            want[:, row] = stored[pg, :, off]
        assert np.array_equal(got.double().cpu().numpy(), want)  # exact: a code has 4 significant bits


def test_every_code_and_scale_reads_back_exactly(fcp):
    """All 254 finite codes at scales across the range, subnormal codes included; scales whose products
    leave bf16's normal range are rounded once, as a float32 product is."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F] + [0, 1], dtype=torch.uint8)
    bytes_ = [0, 1, 2, 8, 60, 110, 120, 127, 130, 134, 200, 240, 246, 255]
    pages = codes.view(1, 4, 1, 64).expand(len(bytes_), 4, 16, 64).contiguous().cuda()
    scales = torch.tensor(bytes_, dtype=torch.uint8).view(-1, 1, 1).expand(len(bytes_), 4, 16).contiguous().cuda()
    cache = fcp.PagedCache.wrap(pages.view(torch.float8_e4m3fn), pages.clone().view(torch.float8_e4m3fn),
                                scales.view(torch.float8_e8m0fnu), scales.clone().view(torch.float8_e8m0fnu))
    n = 16 * len(bytes_)
    batch = fcp.CacheBatch(*(torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, n], [n], [list(range(len(bytes_)))])),
                           n, max_new=n)
    k, v = (torch.empty(4, n, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    want = torch.from_numpy(R.e4m3_values()[codes.numpy()].reshape(4, 1, 1, 64)) * \
        torch.tensor([np.nan if x == 255 else 2.0 ** (x - 127) for x in bytes_], dtype=torch.float64).view(1, -1, 1, 1)
    want = want.expand(4, len(bytes_), 16, 64).reshape(4, n, 64).to(torch.float32).to(torch.bfloat16)
    for got in (k, v):
        got = got.cpu()
        same = (got == want) | (got.isnan() & want.isnan())
        assert same.all(), (got[~same][:8], want[~same][:8])


@pytest.mark.parametrize("d", [64, 128])
def test_quantising_extreme_rows(fcp, d):
    """Rows of zeros, of one tiny or one huge value, with the borders 448 * 2^k, -0, infinities, NaN."""
    rows = torch.zeros(16, d, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(3)
    rows[1, 5] = 1e-38
    rows[2] = torch.finfo(torch.bfloat16).max
    rows[3, 0], rows[3, 1] = 448.0, 0.0009765625
    rows[4, 0], rows[4, 1] = 450.0, -1.0
    rows[5] = torch.randn(d, generator=g).to(torch.bfloat16)
    rows[5, d - 1] = float("inf")
    rows[6] = 1.0
    rows[6, 3] = float("nan")
    rows[7] = -0.0
    rows[8] = 9.2e-41
    rows[9] = torch.linspace(-500, 500, d).to(torch.bfloat16)
    rows[10] = torch.exp2(-torch.arange(d).float() / 3).to(torch.bfloat16)
    rows[11] = (torch.randn(d, generator=g) * 1e30).to(torch.bfloat16)
    rows[12] = -torch.finfo(torch.bfloat16).tiny
    rows[13, 0] = float("-inf")
    cache = fcp.PagedCache(1, 16, 1, d, torch.float8_e4m3fn)
    batch = fcp.CacheBatch(*(torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 16], [16], [[0]])), 16, max_new=16)
    x = rows[None].cuda().contiguous()
    fcp.cache_write(cache, batch, x, x)
    k, v = torch.empty_like(x), torch.empty_like(x)
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    for r in range(16):
        codes, byte = R.quantise_row(rows[r].double().numpy())
        assert np.array_equal(cache.k_pages.view(torch.uint8)[0, 0, r].cpu().numpy(), codes), r
        assert int(cache.k_scales.view(torch.uint8)[0, 0, r]) == int(cache.v_scales.view(torch.uint8)[0, 0, r]) == byte, r
        if byte == 255:
            assert k[0, r].isnan().all()
    # writing what was read stores the same values again
    codes, scales = cache.k_pages.view(torch.uint8).clone(), cache.k_scales.view(torch.uint8).clone()
    keep = scales[0, 0] != 255
    fcp.cache_write(cache, batch, k, v)
    again = U.values(cache.k_pages, cache.k_scales)
    first = U.values(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu))
    normal = np.abs(first) >= 2.0 ** -126  # below it bf16 cannot hold every product
    same = (again == first) | ~normal
    assert same[0, 0][keep.cpu().numpy()].all()


# ---------------------------------------------------------------- attention, few rows
FEW = [
    Batch([1], [1]),
    Batch([1], [2], hq=1, hkv=1, d=128),
    Batch([1, 1, 1], [15, 16, 17], d=128),
    Batch([1, 0, 1, 1], [130, 50, 127, 1000], hq=8, hkv=1, d=128, page=32, pad=3),
    Batch([1, 1], [4097, 3], hq=16, hkv=2, page=64),
    Batch([1], [2500], hq=3, hkv=3, page=256, d=128, causal=False),
    Batch([4, 2, 1, 3], [300, 2, 129, 3], hq=8, hkv=2, d=128),               # 4 x 4 rows
    Batch([5, 7], [100, 700], hq=6, hkv=2, page=128),                          # 21 rows: two tiles
    Batch([4, 1], [260, 513], hq=8, hkv=1, d=128, causal=False),               # 32 rows
    Batch([3, 2], [1, 0], hq=2, hkv=1, d=128),                                 # rows before position 0 see nothing
    Batch([2, 1], [0, 5], causal=False),                                       # a sequence with no cached rows
    Batch([1] * 300, [(i * 37) % 260 for i in range(300)], hq=2, hkv=1),
    Batch([9, 40, 1], [200, 41, 77], hq=8, hkv=2, max_new=1),                  # a wrong max_new is only slow
    Batch([1], [20000], hq=2, hkv=1, page=512, std=3.0),
]
FEW = [b.__class__(**{**b.__dict__, "cache": c, "seed": i}) for i, b in enumerate(FEW) for c in ("bf16", "e4m3")]


def attend(fcp, b, t, cache, batch):
    o = torch.full((b.hq, b.total, b.d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.hq, b.total), 5.0, device="cuda")
    att = fcp.PagedAttention(cache, b.hq, causal=b.causal)
    att.workspace.fill_(255)  # NaN: nothing may be read that this call did not write
    before = o.clone(), lse.clone()
    att.forward(batch, t["q"], o, lse)
    return o, lse, before


@pytest.mark.parametrize("b", FEW, ids=str)
def test_attention_of_few_rows(fcp, b):
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_attention_is_the_same_every_time(fcp, c):
    b = Batch([1, 4, 1], [5000, 700, 64], hq=8, hkv=2, d=128, cache=c)
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    first = attend(fcp, b, t, cache, batch)
    for _ in range(3):
        again = attend(fcp, b, t, cache, batch)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------- attention, chunks
CHUNK = [
    Batch([40], [40]),
    Batch([40], [40], hq=1, hkv=1, d=128),
    Batch([17, 33, 65, 16], [17, 100, 65, 400], hq=8, hkv=1, d=128, pad=2),
    Batch([128, 1, 0, 129], [128, 300, 77, 1000], hq=4, hkv=4, d=128, page=32),
    Batch([200, 64], [1500, 64], hq=6, hkv=2, page=64),
    Batch([300], [300], hq=5, hkv=1, d=128, page=128, causal=False),
    Batch([90, 130], [60, 129], hq=3, hkv=1, d=128),                     # rows before position 0 see nothing
    Batch([70, 5], [0, 700], causal=False),                              # a sequence with no cached rows
    Batch([34, 1, 1, 1], [5000, 4000, 129, 128], hq=8, hkv=1, d=128, page=256),
    Batch([1] * 40 + [35], [(i * 53) % 300 for i in range(40)] + [35], hq=2, hkv=1),
    Batch([513], [2049], hq=2, hkv=1, page=512, std=3.0, pad=1),
    Batch([3, 2], [900, 100], hq=4, hkv=2, d=128, max_new=500),          # a wrong max_new is only slow
    Batch([35, 20], [300, 20], hq=300, hkv=2),                           # 150 heads to a KV head
]
CHUNK = [b.__class__(**{**b.__dict__, "cache": c, "seed": 50 + i}) for i, b in enumerate(CHUNK) for c in ("bf16", "e4m3")]


@pytest.mark.parametrize("b", CHUNK, ids=str)
def test_attention_of_chunks(fcp, b):
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)


# ---------------------------------------------------------------- what goes wrong elsewhere
@pytest.mark.parametrize("new", [1, 3, 60], ids=["few8", "few16", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_with_scales_across_the_range(fcp, new, d):
    """Rows whose scales differ by many powers of two, in K and in V, some too large for one bf16 product:
    the weights and sums must not over- or underflow on the way."""
    b = Batch([new, new], [200, 333], hq=4, hkv=1, d=d, page=32, cache="e4m3", seed=new)
    t = U.make(b)
    g = torch.Generator().manual_seed(9)
    for x, lo, hi in (("k", 110, 119), ("v", 90, 165)):
        byte = t[x + "_scales"].view(torch.uint8)
        new_byte = torch.randint(lo, hi, byte.shape, generator=g, dtype=torch.int32).to(torch.uint8).cuda()
        byte.copy_(torch.where(byte == 255, byte, new_byte))
    # a sequence in the range where V's rows are tiny, another with one huge row of K that gets all the weight
    table = t["table"].cpu()
    t["k_scales"].view(torch.uint8)[int(table[1, 2]), :, 5] = 137
    cache, batch = U.handles(fcp, b, t)
    o, lse, before = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    U.check_attention(b, t, o, lse, *before)


@pytest.mark.parametrize("new", [1, 50], ids=["few", "chunk"])
@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_a_nan_row_reaches_its_readers(fcp, new, c):
    """A NaN in a key makes every row that sees it NaN, and no other sequence's."""
    b = Batch([new, new], [100, 100], hq=2, hkv=1, cache=c, page=16)
    t = U.make(b)
    page, off = int(t["table"][0, 1]), 3  # position 19 of sequence 0
    if c == "bf16":
        t["k_pages"][page, 0, off, 7] = float("nan")
    else:
        t["k_scales"].view(torch.uint8)[page, 0, off] = 255
    cache, batch = U.handles(fcp, b, t)
    o, lse, _ = attend(fcp, b, t, cache, batch)
    cache.check_device_error()
    sees = torch.arange(new) + 100 - new >= 19
    assert o[:, :new].isnan().all(-1).cpu().equal(sees[None].expand(2, -1)) and lse[:, :new].isnan().cpu().equal(
        sees[None].expand(2, -1))
    assert not o[:, new:].isnan().any() and not lse[:, new:].isnan().any()


@pytest.mark.parametrize("max_new", [1, 100], ids=["few", "chunk"])
@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_broken_batches_are_reported_and_harm_nothing(fcp, max_new, c):
    """Offsets that fall back or pass the rows, lengths past the block table, page ids outside the cache:
    the calls finish, the error word tells, what is right is computed and no other row is touched."""
    b = Batch([2, 3, 1, 2, 2], [40, 30, 20, 33, 50], hq=4, hkv=2, cache=c, max_new=max_new, pad=4)
    for what, code in (("cu", 0x50), ("back", 0x50), ("len", 0x50), ("negative", 0x50), ("page", 0x51),
                       ("low page", 0x51)):
        t = U.make(b)
        good = U.make(b)
        if what == "cu":
            # sequence 2 has no row, 3 has 5 .. 7, and 4 would pass the rows: rows 8 and on are no one's
            t["cu"][3:] = torch.tensor([5, 8, 99], dtype=torch.int32)
            good["cu"][3:] = torch.tensor([5, 8, 8], dtype=torch.int32)
            bad = {4}
        elif what == "back":
            t["cu"][5] = 3
            bad = {4}
        elif what == "len":
            t["lens"][1] = 16 * t["table"].shape[1] + 1
            bad = {1}
        elif what == "negative":
            t["lens"][3] = -1
            bad = {3}
        else:
            t["table"][4, 0] = 1 << 30 if what == "page" else -1
            bad = {4}
        cache, batch = U.handles(fcp, b, t)
        o, lse, before = attend(fcp, b, t, cache, batch)
        with pytest.raises(fcp.FcpError, match=hex(code)):
            cache.check_device_error()
        cache.check_device_error()  # read and cleared
        cache2, batch2 = U.handles(fcp, b, good)
        want_o, want_l, _ = attend(fcp, b, good, cache2, batch2)
        row = 0
        for i, n in enumerate(b.new):
            if i not in bad:
                assert torch.equal(o[:, row:row + n], want_o[:, row:row + n]), (what, i)
                assert torch.equal(lse[:, row:row + n], want_l[:, row:row + n])
            elif code == 0x50:
                assert torch.equal(o[:, row:row + n], before[0][:, row:row + n]), (what, i)
            row += n
        assert torch.equal(o[:, row:], before[0][:, row:])
        k = torch.full_like(t["k"], 3.0)
        fcp.cache_read(cache, batch, k, torch.empty_like(k))
        with pytest.raises(fcp.FcpError):
            if what in ("page", "low page"):  # only a needed entry counts: position 0 is not read back here
                batch4 = fcp.CacheBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                        torch.tensor([1], dtype=torch.int32).cuda(), t["table"][4:].contiguous(), 1,
                                        max_new=1)
                fcp.cache_read(cache, batch4, k[:, :1].contiguous(), k[:, :1].contiguous())
            cache.check_device_error()


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_captured_calls_follow_the_tensors(fcp, c):
    """write, attention and read captured into one graph on a side stream; replays see new rows, lengths
    and block tables in the same buffers, for few rows and for chunks."""
    for new, lens in (([1, 1, 1], [40, 7, 300]), ([45, 3, 0], [60, 200, 5])):
        b = Batch(new, lens, hq=4, hkv=2, d=128, page=32, cache=c, seed=1)
        t = U.make(b)
        cache, batch = U.handles(fcp, b, t)
        att = fcp.PagedAttention(cache, b.hq)
        o, lse = torch.zeros_like(t["q"]), torch.zeros(b.hq, b.total, device="cuda")
        k, v = torch.zeros_like(t["k"]), torch.zeros_like(t["v"])
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            fcp.cache_write(cache, batch, t["k"], t["v"])
            att.forward(batch, t["q"], o, lse)
            fcp.cache_read(cache, batch, k, v)
        for seed in (5, 6):
            lens2 = [max(n, x - seed) for n, x in zip(new, lens)]
            other = Batch(new, lens2, hq=4, hkv=2, d=128, page=32, cache=c, seed=seed)
            u = U.make(other)
            keep = min(t["table"].shape[1], u["table"].shape[1])
            order = torch.arange(t["table"].numel(), dtype=torch.int32).view_as(t["table"]).cuda() % cache.n_pages
            need = [-(-x // 32) for x in lens2]
            ids = torch.randperm(cache.n_pages, generator=torch.Generator().manual_seed(seed)).int()
            at = 0
            for i, x in enumerate(need):
                order[i, :x] = ids[at:at + x].cuda()
                at += x
            assert keep and at <= cache.n_pages
            t["table"].copy_(order)
            t["lens"].copy_(u["lens"])
            for x in ("q", "k", "v"):
                t[x].copy_(u[x])
            for x in ("k_pages", "v_pages"):  # what was behind a sequence's end before may be inside now
                p = torch.randn(t[x].shape, generator=torch.Generator().manual_seed(seed)).cuda()
                t[x].copy_(p.to(t[x].dtype) if c == "bf16" else p.to(torch.float8_e4m3fn))
                if c == "e4m3":
                    t[x[0] + "_scales"].view(torch.uint8).fill_(126)
            graph.replay()
            cache.check_device_error()
            now = Batch(new, lens2, hq=4, hkv=2, d=128, page=32, cache=c)
            U.check_attention(now, t, o, lse)
            stored = U.values(t["k_pages"], t["k_scales"])
            table = t["table"].cpu().numpy()
            for row, _, _, pg, off in R.places(new, lens2, table, 32):
                assert np.array_equal(k[:, row].double().cpu().numpy(), stored[pg, :, off])


def test_two_streams_with_a_workspace_each(fcp):
    """Two attentions over one cache at a time, each on its own stream with its own PagedAttention."""
    b1 = Batch([1, 1], [3000, 700], hq=8, hkv=2, d=128, seed=2)
    b2 = Batch([70, 9], [3000, 700], hq=8, hkv=2, d=128, seed=2)
    t = U.make(b1)
    u = U.make(b2)
    for x in ("k_pages", "v_pages", "table"):
        u[x] = t[x]
    cache, batch1 = U.handles(fcp, b1, t)
    _, batch2 = U.handles(fcp, b2, u)
    want1, want2 = attend(fcp, b1, t, cache, batch1)[0], attend(fcp, b2, u, cache, batch2)[0]
    atts = [fcp.PagedAttention(cache, 8) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((torch.empty_like(t["q"]), torch.empty_like(u["q"])))
        lses = [torch.empty(8, x["q"].shape[1], device="cuda") for x in (t, u)]
        torch.cuda.synchronize()
        atts[0].forward(batch1, t["q"], outs[-1][0], lses[0], stream=streams[0])
        atts[1].forward(batch2, u["q"], outs[-1][1], lses[1], stream=streams[1])
    torch.cuda.synchronize()
    cache.check_device_error()
    for o1, o2 in outs:
        assert torch.equal(o1, want1) and torch.equal(o2, want2)


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40], ids=["few", "chunk"])
def test_offsets_past_32_bits(fcp, c, new):
    """Pages whose elements and bytes lie past 2^32: write, read and attention at the far end."""
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 40  # over 2^32 elements in K and in V
    cache = fcp.PagedCache(n_pages, page, hkv, d, dtype=torch.bfloat16 if c == "bf16" else torch.float8_e4m3fn)
    length = 3 * page - 5
    table = torch.tensor([[n_pages - 1, n_pages - 17, n_pages - 3, -9]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(hkv, length, d, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    fcp.cache_write(cache, fcp.CacheBatch(ints([0, length]), ints([length]), table, length, max_new=length), k, v)
    back = torch.empty_like(k), torch.empty_like(v)
    fcp.cache_read(cache, fcp.CacheBatch(ints([0, length]), ints([length]), table, length, max_new=length), *back)
    cache.check_device_error()
    if c == "bf16":
        assert torch.equal(back[0], k) and torch.equal(back[1], v)
    else:
        for got, x in zip(back, (k, v)):  # a code is off by at most half a step: 2^-4 of itself, or of 2^-6 * scale
            top = x.float().abs().amax(-1, keepdim=True)
            assert ((got.float() - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -10 * 2.0 ** -6 * top).all()
    q = torch.randn(hkv, new, d, generator=g).to(torch.bfloat16).cuda()
    o, lse = fcp.PagedAttention(cache, hkv).forward(
        fcp.CacheBatch(ints([0, new]), ints([length]), table, new, max_new=new), q)
    cache.check_device_error()
    for h in (0, hkv - 1):
        ro, rl, spread, _, _ = R.attend(*(x[h].double().cpu().numpy() for x in (q, *back)), new, True)
        assert (np.abs(o[h].double().cpu().numpy() - ro) <= 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread).all()
        assert np.abs(lse[h].double().cpu().numpy() - rl).max() <= 1e-4


# ---------------------------------------------------------------- together, as a server uses them
@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_prompt_then_chunk_then_tokens(fcp, c):
    """Two conversations: the prompt's attention over the work list (FcpAttention) with its K and V written
    to the cache, then a chunk, then single tokens, each written and attended; every output is the causal
    attention of the whole conversation at its rows, over the rows that the cache holds. Then the whole
    conversation is read back and its attention over the work list is the same again."""
    hq, hkv, d, page = 8, 2, 128, 32
    prompts, chunks, steps = [300, 129], [70, 33], 3
    total = [p + m + steps for p, m in zip(prompts, chunks)]
    g = torch.Generator().manual_seed(8)
    q, k, v = ([torch.randn(h, n, d, generator=g).to(torch.bfloat16).cuda() for n in total] for h in (hq, hkv, hkv))
    pages = [-(-n // page) for n in total]
    cache = fcp.PagedCache(sum(pages) + 1, page, hkv, d, dtype=torch.bfloat16 if c == "bf16" else torch.float8_e4m3fn)
    ids = torch.randperm(sum(pages) + 1, generator=g).int()
    table = torch.full((2, max(pages)), -1, dtype=torch.int32)
    table[0, :pages[0]], table[1, :pages[1]] = ids[:pages[0]], ids[pages[0]:pages[0] + pages[1]]
    table = table.cuda()
    lens, cu = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    attention = fcp.PagedAttention(cache, hq)
    outs = [[], []]
    at = [0, 0]

    def pack(x, new):
        return torch.cat([x[i][:, at[i]:at[i] + new[i]] for i in range(2)], 1).contiguous()

    for part, new in enumerate([prompts, chunks] + [[1, 1]] * steps):
        lens.copy_(torch.tensor([a + n for a, n in zip(at, new)]))
        cu.copy_(torch.tensor([0, new[0], sum(new)]))
        batch = fcp.CacheBatch(cu, lens, table, sum(new), max_new=max(new))
        qn, kn, vn = (pack(x, new) for x in (q, k, v))
        fcp.cache_write(cache, batch, kn, vn)
        if part == 0 and c == "bf16":
            att = fcp.FcpAttention(new, 128, True, 2, hq, hkv, d, backward=False)
            o, _ = att.forward(qn, kn, vn)
            att.check_device_error()
        else:
            o, _ = attention.forward(batch, qn)
        for i in range(2):
            outs[i].append(o[:, int(cu[i]):int(cu[i + 1])])
            at[i] += new[i]
    cache.check_device_error()
    lens.copy_(torch.tensor(total))
    cu.copy_(torch.tensor([0, total[0], sum(total)]))
    whole = fcp.CacheBatch(cu, lens, table, sum(total), max_new=max(total))
    rk, rv = (torch.empty(hkv, sum(total), d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fcp.cache_read(cache, whole, rk, rv)
    cache.check_device_error()
    att = fcp.FcpAttention(total, 128, True, 2, hq, hkv, d, backward=False)
    o, _ = att.forward(torch.cat(q, 1), rk, rv)
    att.check_device_error()
    for i in range(2):
        got = torch.cat(outs[i], 1).double().cpu().numpy()
        a = sum(total[:i])
        again = o[:, a:a + total[i]].double().cpu().numpy()
        if c == "bf16":
            assert torch.equal(rk[:, a:a + total[i]], k[i]) and torch.equal(rv[:, a:a + total[i]], v[i])
        for h in range(hq):
            kk, vv = (x[h * hkv // hq, a:a + total[i]].double().cpu().numpy() for x in (rk, rv))
            ro, _, spread, _, _ = R.attend(q[i][h].double().cpu().numpy(), kk, vv, total[i], True)
            bound = 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread
            assert (np.abs(got[h] - ro) <= bound).all(), (i, h)
            assert (np.abs(again[h] - ro) <= bound).all(), (i, h)


def test_the_binding_refuses_what_does_not_fit(fcp):
    b = Batch([1, 2], [20, 30])
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    ok = (torch.empty_like(t["q"]), torch.empty(b.hq, b.total, device="cuda"))
    att = fcp.PagedAttention(cache, b.hq)
    for q in (t["q"].float(), t["q"][:, :-1], t["q"][:-1], t["q"].transpose(0, 1), t["q"][..., :32].contiguous(), t["q"].cpu()):
        with pytest.raises((TypeError, ValueError)):
            att.forward(batch, q, *ok)
    with pytest.raises((TypeError, ValueError)):
        att.forward(batch, t["q"], ok[0].float(), ok[1])
    with pytest.raises((TypeError, ValueError)):
        att.forward(batch, t["q"], ok[0], ok[1].double())
    with pytest.raises(ValueError):
        fcp.PagedAttention(cache, 3)
    for k in (t["k"].float(), t["k"][:, 1:], t["k"].transpose(1, 2), t["k"].cpu()):
        with pytest.raises((TypeError, ValueError)):
            fcp.cache_write(cache, batch, k, t["v"])
        with pytest.raises((TypeError, ValueError)):
            fcp.cache_read(cache, batch, t["k"], k)
    with pytest.raises(ValueError):
        fcp.CacheBatch(t["cu"][:-1], t["lens"], t["table"], 3, max_new=1)
    with pytest.raises(ValueError):
        fcp.CacheBatch(t["cu"], t["lens"], t["table"][:1], 3, max_new=1)
    with pytest.raises(TypeError):
        fcp.CacheBatch(t["cu"].long(), t["lens"], t["table"], 3, max_new=1)
    with pytest.raises(ValueError):
        fcp.CacheBatch(t["cu"], t["lens"], t["table"], -1, max_new=1)
    with pytest.raises(ValueError):
        fcp.PagedCache(2, 24, 1, 64)
    with pytest.raises(ValueError):
        fcp.PagedCache(2, 16, 1, 96)
    with pytest.raises(ValueError):
        fcp.PagedCache.wrap(t["k_pages"], t["v_pages"], torch.zeros(1, device="cuda"))
    with pytest.raises(fcp.FcpError):  # a workspace too small for the C call
        fcp.paged_attn(cache, batch, t["q"], *ok, att.workspace[:256])


def test_nothing_to_do(fcp):
    cache = fcp.PagedCache(2, 16, 1, 64, dtype=torch.float8_e4m3fn)
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    none = torch.empty(1, 0, 64, dtype=torch.bfloat16, device="cuda")
    for batch in (fcp.CacheBatch(ints([0]), torch.empty(0, dtype=torch.int32, device="cuda"),
                                 torch.empty(0, 1, dtype=torch.int32, device="cuda"), 0, max_new=0),
                  fcp.CacheBatch(ints([0, 0]), ints([5]), ints([[0]]), 0, max_new=0)):
        fcp.cache_write(cache, batch, none, none)
        fcp.cache_read(cache, batch, none, none)
        o, lse = fcp.PagedAttention(cache, 2).forward(batch, torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda"))
        assert o.shape == (2, 0, 64) and lse.shape == (2, 0)
    # rows of no sequence at all
    q = torch.ones(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(q, 4.0), torch.full((2, 3), 4.0, device="cuda")
    for max_new in (1, 100):
        batch = fcp.CacheBatch(ints([0, 0]), ints([5]), ints([[0]]), 3, max_new=max_new)
        fcp.PagedAttention(cache, 2).forward(batch, q, o, lse)
        assert (o == 4).all() and (lse == 4).all()
    cache.check_device_error()


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_outputs_allocated_for_another_stream_are_its_own(fcp, raw):
    """Memory that the current stream may still be using (freed, its kernels perhaps running) does
    not become the output of a call on another stream."""
    b = Batch([1, 2], [20, 30], hq=64, hkv=2, d=128)
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    att = fcp.PagedAttention(cache, b.hq)
    want = att.forward(batch, t["q"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(t["q"]) for _ in range(8)] + [torch.empty(b.hq, b.total, device="cuda") for _ in range(8)]
    addresses = {x.data_ptr() for x in freed}
    del freed
    got = att.forward(batch, t["q"], stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert not addresses & {x.data_ptr() for x in got}
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_workspace_of_another_kind_is_refused(fcp):
    b = Batch([1], [20])
    t = U.make(b)
    cache, batch = U.handles(fcp, b, t)
    out = torch.empty_like(t["q"]), torch.empty(b.hq, b.total, device="cuda")
    n = fcp.lib().fcp_paged_attn_workspace_bytes(b.d)
    for ws in (torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2], torch.empty(n, dtype=torch.uint8),
               torch.empty(n, dtype=torch.int8, device="cuda")):
        with pytest.raises((TypeError, ValueError)):
            fcp.paged_attn(cache, batch, t["q"], *out, ws)


def many(c, new):
    n = 2600
    return Batch([new[i % len(new)] for i in range(n)], [(i * 29) % 90 for i in range(n)], hq=2, hkv=1, cache=c, seed=9, pad=2)


@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_more_sequences_than_a_block_has_threads(fcp, c):
    """Offsets are searched in two steps and a thread has several sequences of the schedule, some of
    them with no new token."""
    b = many(c, [0, 1, 2])
    t = U.make(b)
    for max_new in (2, 200):  # both kernels
        b.max_new = max_new
        cache, batch = U.handles(fcp, b, t)
        o, lse, before = attend(fcp, b, t, cache, batch)
        cache.check_device_error()
        U.check_attention(b, t, o, lse, *before)
    # every new token's row: what is read back is what the pages hold
    k, v = (torch.full((1, b.total, b.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fcp.cache_write(cache, batch, t["k"], t["v"])
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    row = 0
    for n, length in zip(b.new, b.lens):
        for j in range(n):
            if length - n + j < 0:
                assert (k[0, row] == 7).all() and (v[0, row] == 7).all()
            elif c == "bf16":
                assert torch.equal(k[0, row], t["k"][0, row]) and torch.equal(v[0, row], t["v"][0, row])
            row += 1
    assert (k[:, row:] == 7).all() and row == b.total - 2
    if c == "e4m3":
        held = torch.tensor([length - n + j >= 0 for n, length in zip(b.new, b.lens) for j in range(n)], device="cuda")
        for got, x in ((k, t["k"]), (v, t["v"])):
            x, got = x[0, :row][held].double(), got[0, :row][held].double()
            # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale, which is at most amax / 224
            assert ((got - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, x.abs().amax(1, keepdim=True) / 224 * 2.0 ** -10)).all()


@pytest.mark.parametrize("new", [1, 40], ids=["few", "chunk"])
@pytest.mark.parametrize("c", ["bf16", "e4m3"])
def test_buffers_at_the_least_alignment(fcp, c, new):
    """Rows, pages and scales on 16-byte, lse and the batch's arrays on 4-byte boundaries."""
    b = Batch([new, 3], [300, 70], hq=6, hkv=2, d=128, page=32, cache=c, seed=4)
    t = U.make(b)

    def shifted(x):
        if x is None:
            return None
        step = 16 // x.element_size() if x.dtype not in (torch.int32, torch.float32) else 1
        flat = torch.zeros(x.numel() + step, dtype=torch.uint8 if x.element_size() == 1 else x.dtype, device="cuda")
        out = flat[step:].view(x.dtype).view(x.shape)
        out.copy_(x) if x.element_size() > 1 else out.view(torch.uint8).copy_(x.view(torch.uint8))
        return out

    u = {name: shifted(x) for name, x in t.items()}
    results = []
    for z in (t, u):
        cache, batch = U.handles(fcp, b, z)
        o, lse = shifted(torch.zeros_like(z["q"])), shifted(torch.zeros(b.hq, b.total, device="cuda"))
        fcp.cache_write(cache, batch, z["k"], z["v"])
        k, v = shifted(torch.zeros_like(z["k"])), shifted(torch.zeros_like(z["v"]))
        fcp.cache_read(cache, batch, k, v)
        fcp.PagedAttention(cache, b.hq).forward(batch, z["q"], o, lse)
        cache.check_device_error()
        results.append((o, lse, k, v))
        U.check_attention(b, z, o, lse)
    assert all(torch.equal(x, y) for x, y in zip(*results))


FIRST_CALL = """
import torch
import context_parallelism_fcp_gb300 as fcp
from tests import paged_util as U
for c in ("bf16", "e4m3"):
    for new in (1, 40):
        b = U.Batch([new], [100], hq=2, hkv=1, d=128, cache=c)
        t = U.make(b)
        cache, batch = U.handles(fcp, b, t)
        att = fcp.PagedAttention(cache, b.hq)
        o, lse = torch.zeros_like(t["q"]), torch.zeros(b.hq, b.total, device="cuda")
        k, v = torch.zeros_like(t["k"]), torch.zeros_like(t["v"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fcp.cache_write(cache, batch, t["k"], t["v"])
            att.forward(batch, t["q"], o, lse)
            fcp.cache_read(cache, batch, k, v)
        graph.replay()
        torch.cuda.synchronize()
        cache.check_device_error()
        U.check_attention(b, t, o, lse)
        assert k.abs().sum() > 0
print("captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """Nothing is set up by a first call that a capture would not allow."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
