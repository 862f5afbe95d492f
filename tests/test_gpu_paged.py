"""The paged cache and its attention against the float64 definitions (oracle/paged.py)."""
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
