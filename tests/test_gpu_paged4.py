"""A 4-bit paged cache against its float64 definition (oracle/paged4.py)."""
import numpy as np
import pytest
import torch

from oracle import paged as R
from oracle import paged4 as R4
from tests import paged4_util as U
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu

MOVES = [
    Batch([1], [1]),
    Batch([3, 0, 17, 1], [3, 40, 33, 64], pad=2),
    Batch([5, 2, 64], [4, 1, 64], hkv=3, hq=3, page=32, d=128),          # tokens before position 0 are left out
    Batch([1] * 70, list(range(1, 71)), hkv=1, hq=1, page=64, d=128),
    Batch([129, 1], [300, 1], hkv=5, hq=5, d=128, page=128, pad=1, std=30.0),
    Batch([0, 0, 7], [0, 3, 7], page=256, std=0.01),
]


def byte(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("b", MOVES, ids=str)
def test_write_stores_the_definition_and_nothing_else(fcp, b):
    t = U.make(b)
    before = {x: byte(t[x]).copy() for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    cache, batch = U.handles(fcp, b, t)
    fcp.cache_write(cache, batch, t["k"], t["v"])
    cache.check_device_error()
    table = t["table"].cpu().numpy()
    for x, unit in (("k", U.K_UNIT), ("v", U.V_UNIT)):
        codes, scales = R4.quantise(t[x].double().cpu().numpy(), unit)
        packed = (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
        pages, got = byte(t[x + "_pages"]), byte(t[x + "_scales"])
        for row, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
            before[x + "_pages"][pg, :, off], before[x + "_scales"][pg, :, off] = packed[:, row], scales[:, row]
        # the sign of a value that rounds to zero is not kept in particular
        zero = lambda p: np.where(R4.unpack(p) == 8, 0, R4.unpack(p))  # noqa: E731
        written = np.zeros(pages.shape[:3], bool)
        for _, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
            written[pg, :, off] = True
        assert np.array_equal(pages[~written], before[x + "_pages"][~written])
        assert np.array_equal(zero(pages[written]), zero(before[x + "_pages"][written]))
        assert np.array_equal(got, before[x + "_scales"])


@pytest.mark.parametrize("b", MOVES, ids=str)
def test_read_returns_the_stored_values(fcp, b):
    t = U.make(b, lo=1, hi=0x7F)
    cache, batch = U.handles(fcp, b, t)
    k, v = torch.full_like(t["k"], 7.0), torch.full_like(t["v"], -7.0)
    before = k.clone(), v.clone()
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    table = t["table"].cpu().numpy()
    for got, old, x, unit in ((k, before[0], "k", U.K_UNIT), (v, before[1], "v", U.V_UNIT)):
        want = old.double().cpu().numpy()
        stored = U.values(t[x + "_pages"], t[x + "_scales"], unit)
        for row, _, _, pg, off in R.places(b.new, b.lens, table, b.page):
            want[:, row] = stored[pg, :, off]
        assert np.array_equal(got.double().cpu().numpy(), want)  # exact: 6 significant bits


@pytest.mark.parametrize("unit", [2.0 ** -60, 0.25, 1.0, 2.0 ** 60])
def test_every_code_and_scale_reads_back_exactly(fcp, unit):
    """All 16 codes at all 127 scales and NaN."""
    codes = torch.arange(16).repeat(4)
    packed = (codes[::2] | (codes[1::2] << 4)).to(torch.uint8)
    pages = packed.expand(2, 1, 64, 32).contiguous().cuda()
    scales = torch.arange(128, dtype=torch.int32).clamp(max=127).to(torch.uint8).view(2, 1, 64, 1).expand(2, 1, 64, 4).contiguous().cuda()
    cache = fcp.PagedCache.wrap(*(pages.clone().view(torch.float4_e2m1fn_x2) for _ in "kv"),
                                *(scales.clone().view(torch.float8_e4m3fn) for _ in "kv"), k_unit=unit, v_unit=unit)
    batch = fcp.CacheBatch(*(torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 128], [128], [[0, 1]])), 128, max_new=128)
    k, v = (torch.empty(1, 128, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    want = R4.value(codes.numpy()[None].repeat(128, 0), scales.cpu().numpy().reshape(128, 4).astype(np.int64), unit)
    for got in (k, v):
        assert np.array_equal(got[0].double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -6, 2.0 ** 9])
def test_quantising_at_borders_and_extremes(fcp, d, unit):
    """Every border between two codes at every scale (and its neighbours), borders between scales, rows of
    zeros, one tiny or huge value, infinities and NaN."""
    g = torch.Generator().manual_seed(3)
    scale = torch.tensor(R4._SCALES[1:], dtype=torch.float64)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    edge = (border[None] * scale[:, None]).to(torch.bfloat16)  # exact: 7 significant bits
    around = torch.cat([edge, torch.nextafter(edge, edge * 2), torch.nextafter(edge, edge * 0)], 1)[:, :15]
    rows = [torch.cat([(6 * scale[:, None]).to(torch.bfloat16), around], 1)]  # the largest sets the scale
    mid = ((scale[:-1] + scale[1:]) / 2 * 6).to(torch.bfloat16)
    for top in (mid, torch.nextafter(mid, mid * 2), torch.nextafter(mid, mid * 0)):
        x = (torch.rand(len(top), 16, generator=g) * 2 - 1).to(torch.bfloat16) * top[:, None]
        x[:, 3] = -top
        rows.append(x)
    odd = torch.zeros(16, 16, dtype=torch.bfloat16)
    odd[1, 5] = 1e-38
    odd[2] = torch.finfo(torch.bfloat16).max
    odd[3, 0] = 2.0 ** -9 * 0.25
    odd[4] = 2.0 ** -9 * 0.75
    odd[5] = torch.randn(16, generator=g).to(torch.bfloat16)
    odd[5, 15] = float("inf")
    odd[6] = 1.0
    odd[6, 3] = float("nan")
    odd[7] = -0.0
    odd[8] = 9.2e-41
    odd[9] = torch.linspace(-5000, 5000, 16).to(torch.bfloat16)
    odd[10, 0] = float("-inf")
    odd[11, 2], odd[11, 3] = 2688.0, 2704.0
    x = torch.cat([*rows, odd]) * torch.tensor(unit, dtype=torch.bfloat16)  # a power of two: borders stay borders
    x = torch.cat([x, torch.zeros(-len(x) % (d // 16), 16, dtype=torch.bfloat16)]).reshape(-1, d)
    n = len(x)
    cache = fcp.PagedCache(-(-n // 16), 16, 1, d, torch.float4_e2m1fn_x2, k_unit=unit, v_unit=unit)
    batch = fcp.CacheBatch(*(torch.tensor(y, dtype=torch.int32).cuda() for y in ([0, n], [n], [list(range(-(-n // 16)))])),
                           n, max_new=n)
    x = x[None].cuda().contiguous()
    fcp.cache_write(cache, batch, x, -x)
    codes, scales = R4.quantise(x[0].double().cpu().numpy(), unit)
    for pages, sc, sign in ((cache.k_pages, cache.k_scales, 1), (cache.v_pages, cache.v_scales, -1)):
        got = R4.value(R4.unpack(byte(pages)).reshape(-1, d)[:n], byte(sc).reshape(-1, d // 16)[:n], unit)
        assert np.array_equal(byte(sc).reshape(-1, d // 16)[:n], scales)
        assert np.array_equal(sign * got, R4.value(codes, scales, unit), equal_nan=True)
    # writing what was read stores the same values again, where the scale is a normal e4m3 number
    k, v = torch.empty_like(x), torch.empty_like(x)
    fcp.cache_read(cache, batch, k, v)
    cache.check_device_error()
    kept = np.repeat(scales >= 8, 16, -1) & np.isfinite(k[0].double().cpu().numpy())
    fcp.cache_write(cache, batch, k, v)
    again = R4.value(R4.unpack(byte(cache.k_pages)).reshape(-1, d)[:n], byte(cache.k_scales).reshape(-1, d // 16)[:n], unit)
    assert np.array_equal(again[kept], R4.value(codes, scales, unit)[kept])


# ---------------------------------------------------------------- attention
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
    Batch([4, 3], [777, 5], hq=16, hkv=2),
    Batch([3, 2], [1, 0], hq=2, hkv=1, d=128),                                 # rows before position 0 see nothing
    Batch([2, 1], [0, 5], causal=False),                                       # a sequence with no cached rows
    Batch([1] * 300, [(i * 37) % 260 for i in range(300)], hq=2, hkv=1),
    Batch([9, 40, 1], [200, 41, 77], hq=8, hkv=2, max_new=1),                  # a wrong max_new is only slow
    Batch([1], [20000], hq=2, hkv=1, page=512, std=3.0),
]
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
    Batch([600, 300, 450], [700, 300, 451], hq=8, hkv=4, d=128),         # units of one and of two tiles in turn
]
ATTEND = [b.__class__(**{**b.__dict__, "seed": i}) for i, b in enumerate(FEW + CHUNK)]


def attend(fcp, b, t, cache, batch):
    o = torch.full((b.hq, b.total, b.d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.hq, b.total), 5.0, device="cuda")
    att = fcp.PagedAttention(cache, b.hq, causal=b.causal)
    att.workspace.fill_(255)  # NaN: nothing may be read that this call did not write
    before = o.clone(), lse.clone()
    att.forward(batch, t["q"], o, lse)
    cache.check_device_error()
    return o, lse, before


@pytest.mark.parametrize("b", ATTEND, ids=str)
def test_attention(fcp, b):
    t = U.make(b)
    o, lse, before = attend(fcp, b, t, *U.handles(fcp, b, t))
    U.check_attention(b, t, o, lse, *before)


# Sequences of one tile of rows at most, of whose key tiles two groups of warps take half the keys each: one key tile,
# two, an odd number, many over several blocks; beside them batches with longer sequences, and one that says it has none.
ONE_TILE = [
    Batch([5], [129], hq=8, hkv=1, d=128),
    Batch([5], [257], hq=8, hkv=1),
    Batch([16, 5, 12, 9, 7], [300, 128, 40, 1000, 513], hq=8, hkv=1, d=128, pad=1),
    Batch([40, 6, 17, 5, 100], [400, 800, 17, 300, 100], hq=8, hkv=2, d=128, page=32),
    Batch([40, 6, 17, 5, 100], [400, 800, 17, 300, 100], hq=8, hkv=2),
    Batch([6], [20000], hq=8, hkv=1, d=128, page=256, std=3.0),
    Batch([1, 1, 1], [700, 2000, 129], hq=48, hkv=1, d=128, page=64),
    Batch([1, 1], [640, 130], hq=100, hkv=2, page=64, causal=False),
    Batch([5] * 60, [100 + (i * 97) % 900 for i in range(60)], hq=32, hkv=4, d=128),
    Batch([5, 37] * 20, [37 + (i * 97) % 900 for i in range(40)], hq=16, hkv=2),
    Batch([150, 5], [140, 300], hq=8, hkv=1, d=128),                     # rows before position 0 see nothing
    Batch([70], [300], hq=1, hkv=1, d=128, causal=False),
    Batch([128, 100, 0, 33], [128, 500, 40, 300], hq=3, hkv=3, d=128),
    Batch([30, 17], [30, 1000], hq=8, hkv=2, pad=1, std=3.0),
    Batch([5, 12], [64, 65], hq=8, hkv=1, d=128, page=64),
    Batch([200, 5, 17], [900, 300, 100], hq=8, hkv=1, d=128, max_new=5),  # a wrong max_new is only slow
]
ONE_TILE = [b.__class__(**{**b.__dict__, "seed": 50 + i}) for i, b in enumerate(ONE_TILE)]


@pytest.mark.parametrize("b", ONE_TILE, ids=str)
def test_attention_of_one_tile(fcp, b):
    t = U.make(b)
    o, lse, before = attend(fcp, b, t, *U.handles(fcp, b, t))
    U.check_attention(b, t, o, lse, *before)


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_scale_in_either_half_of_a_key_tile(fcp, d):
    """As below, with the scale among the keys of either group of warps."""
    new, n, hq = 9, 400, 8
    for x in "kv":
        for pos in (19, 100, 150, 300, n - 5, n - 1):
            b = Batch([new, new], [n, n], hq=hq, hkv=1, d=d, page=16)
            t = U.make(b)
            page, group = int(t["table"][0, pos // 16]), (pos * 7) % (d // 16)
            t[x + "_scales"].view(torch.uint8)[page, 0, pos % 16, group] = 0x7F
            o, lse, _ = attend(fcp, b, t, *U.handles(fcp, b, t))
            sees = (torch.arange(new) + n - new >= pos)[None].expand(hq, -1)
            assert o[:, :new].isnan().cpu().any(-1).equal(sees), (x, pos)
            if x == "k":
                assert lse[:, :new].isnan().cpu().equal(sees)
            t[x + "_scales"].view(torch.uint8)[page, 0, pos % 16, group] = 0x20
            want, _, _ = attend(fcp, b, t, *U.handles(fcp, b, t))
            assert torch.equal(o[:, new:], want[:, new:])
            clear = ~sees.cuda()
            assert torch.equal(o[:, :new][clear], want[:, :new][clear])


@pytest.mark.parametrize("new", [1, 4, 8, 60], ids=["few8", "few16", "few32", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_with_scales_across_the_range(fcp, new, d):
    """Scales from the smallest to the largest, rows of V of 2^17 times one another's size among them, and q of
    any size: weights and sums must not over- or underflow on the way."""
    b = Batch([new, new], [200, 333], hq=4, hkv=1, d=d, page=32, seed=new)
    t = U.make(b, lo=1, hi=0x7F)
    ks = t["k_scales"].view(torch.uint8)
    ks.copy_(torch.where(ks == 0x7F, ks, ks // 4 + 1))  # up to 2^-3: scores that do not leave one key alone
    t["q"][0] *= 2.0 ** -40
    t["q"][1] *= 2.0 ** -3
    t["q"][2, 0] = 0
    o, lse, before = attend(fcp, b, t, *U.handles(fcp, b, t))
    U.check_attention(b, t, o, lse, *before)


@pytest.mark.parametrize("units", [(2.0 ** -40, 2.0 ** 30), (2.0 ** 20, 2.0 ** -50)])
@pytest.mark.parametrize("new", [1, 50], ids=["few", "chunk"])
def test_units(fcp, new, units):
    """A unit is a factor of the scores, or of the output, whether a group is split over blocks or not."""
    b = Batch([new, new], [3000, 70], hq=4, hkv=1, d=128, page=64, seed=new)
    t = U.make(b)
    t["q"] *= 1 / units[0]
    o, lse, before = attend(fcp, b, t, *U.handles(fcp, b, t, *units))
    U.check_attention(b, t, o, lse, *before, *units)


@pytest.mark.parametrize("unit", [2.0 ** -60, 1.0, 2.0 ** 60])
@pytest.mark.parametrize("new,hq", [(1, 4), (3, 4), (3, 16), (50, 4)], ids=["few8", "few16", "few32", "chunk"])
def test_rows_of_zeros_and_of_the_smallest_and_largest_numbers(fcp, new, hq, unit):
    """A q of zeros weighs all keys the same, whatever the unit; so do q and units whose products are below float32's
    range, beside rows that are masked."""
    b = Batch([new, new], [100, 2 * new], hq=hq, hkv=1, d=128, page=32, seed=new)
    t = U.make(b)
    t["q"][0] = 0
    t["q"][1] = torch.finfo(torch.bfloat16).tiny
    t["q"][2, :, ::2] = 0
    t["q"][2, :, 1::2] *= 2.0 ** -100 if unit >= 1 else 2.0 ** 50
    o, lse, before = attend(fcp, b, t, *U.handles(fcp, b, t, unit, 1.0))
    for h in (0, 1, 2):  # one head at a time, as a batch of its own
        one = Batch(b.new, b.lens, hq=1, hkv=1, d=128, page=32)
        U.check_attention(one, {**t, "q": t["q"][h:h + 1]}, o[h:h + 1], lse[h:h + 1], before[0][h:h + 1], before[1][h:h + 1], unit, 1.0)


@pytest.mark.parametrize("new,hq", [(1, 2), (4, 2), (4, 4), (4, 8), (50, 2)], ids=["few1", "few8", "few16", "few32", "chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_scale_reaches_its_readers_only(fcp, new, hq, d):
    """In K it makes every row that sees it NaN; in V the rows that see it, in its channels at least; and no row
    that comes before it, nor another sequence."""
    for x in "kv":
        for pos in (19, 100 - new, 99, 98 if new > 2 else 99):
            b = Batch([new, new], [100, 100], hq=hq, hkv=1, d=d, page=16)
            t = U.make(b)
            page, group = int(t["table"][0, pos // 16]), (pos * 7) % (d // 16)
            t[x + "_scales"].view(torch.uint8)[page, 0, pos % 16, group] = 0x7F if pos % 2 else 0xFF
            o, lse, _ = attend(fcp, b, t, *U.handles(fcp, b, t))
            sees = (torch.arange(new) + 100 - new >= pos)[None].expand(hq, -1)
            channels = slice(None) if x == "k" else slice(16 * group, 16 * group + 16)
            bad = o[:, :new].isnan().cpu()
            assert bad[..., channels].all(-1).equal(sees) and bad.any(-1).equal(sees), (x, pos)
            if x == "k":
                assert lse[:, :new].isnan().cpu().equal(sees)
            t[x + "_scales"].view(torch.uint8)[page, 0, pos % 16, group] = 0x20
            want, _, _ = attend(fcp, b, t, *U.handles(fcp, b, t))
            assert torch.equal(o[:, new:], want[:, new:])
            clear = ~sees.cuda()
            assert torch.equal(o[:, :new][clear], want[:, :new][clear])


@pytest.mark.parametrize("max_new", [1, 100], ids=["few", "chunk"])
def test_broken_batches_are_reported_and_harm_nothing(fcp, max_new):
    b = Batch([2, 3, 1, 2, 2], [40, 30, 20, 33, 50], hq=4, hkv=2, max_new=max_new, pad=4)
    for what, code in (("len", 0x50), ("negative", 0x50), ("page", 0x51), ("low page", 0x51)):
        t, good = U.make(b), U.make(b)
        if what == "len":
            t["lens"][4] = 16 * t["table"].shape[1] + 1
        elif what == "negative":
            t["lens"][4] = -1
        else:
            t["table"][4, 1] = 1 << 30 if what == "page" else -1
        cache, batch = U.handles(fcp, b, t)
        att = fcp.PagedAttention(cache, b.hq)
        o, lse = att.forward(batch, t["q"])
        with pytest.raises(fcp.FcpError, match=hex(code)):
            cache.check_device_error()
        want, _, _ = attend(fcp, b, good, *U.handles(fcp, b, good))
        assert torch.equal(o[:, :8], want[:, :8]), what
        if code == 0x51:  # a page's keys count as zeros
            assert o[:, 8:10].isfinite().all()


def test_attention_is_the_same_every_time_and_on_any_stream(fcp):
    for new in ([1, 4, 1], [300, 4, 70]):
        b = Batch(new, [5000, 700, 74], hq=8, hkv=2, d=128)
        t = U.make(b)
        cache, batch = U.handles(fcp, b, t)
        first = attend(fcp, b, t, cache, batch)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for stream in (None, side, side):
            with torch.cuda.stream(stream or torch.cuda.current_stream()):
                again = attend(fcp, b, t, cache, batch)
            torch.cuda.synchronize()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_calls_follow_the_tensors(fcp):
    """write, attention and read in one graph; replays see new rows, lengths and block tables."""
    for new, lens in (([1, 1, 1], [40, 7, 300]), ([45, 3, 0], [60, 200, 5])):
        b = Batch(new, lens, hq=4, hkv=2, d=128, page=32, seed=1)
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
        for seed in (5, 6):
            z = U.make(Batch(new, lens, hq=4, hkv=2, d=128, page=32, seed=seed))
            lens2 = [x - (seed == 6 and x > n) for x, n in zip(lens, new)]
            z["lens"] = torch.tensor(lens2, dtype=torch.int32)
            for x, y in z.items():
                small = x.endswith("pages") or x.endswith("scales")
                (t[x].view(torch.uint8) if small else t[x]).copy_(y.view(torch.uint8) if small else y)
            graph.replay()
            cache.check_device_error()
            b2 = Batch(new, lens2, hq=4, hkv=2, d=128, page=32)
            U.check_attention(b2, t, o, lse)
            codes, scales = R4.quantise(t["k"].double().cpu().numpy(), U.K_UNIT)
            assert np.array_equal(k.double().cpu().numpy(), R4.value(codes, scales, U.K_UNIT))


def test_pages_past_32_bits(fcp):
    """Codes whose bytes lie past 2^32: write, read and attention at the far end."""
    page, hkv, d = 4096, 8, 128
    n_pages = (1 << 32) // (page * hkv * d // 2) + 2
    cache = fcp.PagedCache(n_pages, page, hkv, d, torch.float4_e2m1fn_x2)
    g = torch.Generator(device="cuda").manual_seed(0)
    length = 300
    k, v = (torch.randn(hkv, length, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    q = torch.randn(hkv, length, d, generator=g, device="cuda", dtype=torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    table = ints([[n_pages - 1]])
    whole = fcp.CacheBatch(ints([0, length]), ints([length]), table, length, max_new=length)
    fcp.cache_write(cache, whole, k, v)
    back = torch.empty_like(k), torch.empty_like(v)
    fcp.cache_read(cache, whole, *back)
    for x, y in zip((k, v), back):
        codes, scales = R4.quantise(x.double().cpu().numpy(), 1.0)
        assert np.array_equal(y.double().cpu().numpy(), R4.value(codes, scales, 1.0))
    for new in (1, length):
        batch = fcp.CacheBatch(ints([0, new]), ints([length]), table, new, max_new=new)
        o, _ = fcp.PagedAttention(cache, hkv).forward(batch, q[:, length - new:].contiguous())
        for h in (0, 5):
            ro, _, spread, _, _ = R.attend(*(x[h].double().cpu().numpy() for x in (q[:, length - new:], *back)), new, True)
            assert (np.abs(o[h].double().cpu().numpy() - ro) <= 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread).all()
    cache.check_device_error()
