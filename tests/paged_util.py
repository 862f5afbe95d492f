"""Batches over a paged cache for the tests, and their comparison with the float64 definition.

Every page that a batch does not use, every row of its pages past a sequence's length and every
unused block-table entry hold what must never matter: NaN rows and page ids out of range.

Tolerances of the attention, from its arithmetic. P is rounded to bf16 before the product with
V, by at most 2^-8 of itself, and o is rounded to bf16 once, by at most 2^-8 of itself; float32
sums, products and exp2 add errors of the order 2^-20. So, with A = sum_j w_j |v_j| (at least
|o|), every element is off by at most 2^-8 A + 2^-8 |o| + 2^-12 A. The roundings are independent,
so on the average over all elements the error stays below 2^-8 (sqrt(sum_j w_j^2 v_j^2) + |o|),
plus the same 2^-12 A. Scores are float32 sums of D exact products: each is off by at most
D * 2^-24 times the sum of the products' magnitudes, and so is the lse (at most; plus 2^-20 of
its size and of 1 for exp2, log2 and the conversions between bases).
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import List

import numpy as np
import torch

from oracle import paged as R


@dataclass
class Batch:
    new: List[int]
    lens: List[int]
    hq: int = 4
    hkv: int = 2
    d: int = 64
    page: int = 16
    cache: str = "bf16"
    causal: bool = True
    pad: int = 0
    seed: int = 0
    max_new: int = -1
    std: float = 1.0
    extra_pages: int = 2
    tables: dict = field(default_factory=dict)

    @property
    def total(self):
        return sum(self.new) + self.pad

    def __str__(self):
        return f"{self.cache}-d{self.d}-h{self.hq}.{self.hkv}-p{self.page}-new{self.new}-len{self.lens}-" \
               f"{'causal' if self.causal else 'full'}".replace(" ", "")[:120]


def make(b: Batch, device="cuda"):
    """The batch's tensors: table, cu, lens, q, new rows k and v, and filled pages."""
    rng = np.random.default_rng(b.seed)
    need = [-(-x // b.page) for x in b.lens]
    n_pages = sum(need) + b.extra_pages
    ids = rng.permutation(n_pages)
    table = np.full((len(b.lens), max([1] + need) + 1), -7, np.int32)
    table[:, -1] = n_pages + 5
    at = 0
    for i, x in enumerate(need):
        table[i, :x] = ids[at:at + x]
        at += x
    g = torch.Generator().manual_seed(b.seed)

    def normal(*shape):
        return (torch.randn(*shape, generator=g) * b.std).to(torch.bfloat16)

    shape = (n_pages, b.hkv, b.page, b.d)
    held = np.zeros((n_pages, b.page), bool)
    for i, x in enumerate(b.lens):
        for p in range(x):
            held[table[i, p // b.page], p % b.page] = True
    held_t = torch.from_numpy(held)[:, None, :, None].expand(n_pages, b.hkv, b.page, 1)
    k_scales = v_scales = None
    if b.cache == "bf16":
        pages = [torch.where(held_t, normal(*shape), torch.tensor(float("nan"), dtype=torch.bfloat16)) for _ in "kv"]
    else:
        pages, scales = [], []
        for _ in "kv":
            code = torch.randint(0, 256, shape, generator=g, dtype=torch.int32)
            code = torch.where(code % 128 >= 0x7F, code - 1, code)  # 0x7f and 0xff are never written
            byte = torch.randint(127 - 10, 127 - 7, shape[:3], generator=g, dtype=torch.int32)
            pages.append(torch.where(held_t, code, torch.full_like(code, 0x7F)).to(torch.uint8).view(torch.float8_e4m3fn))
            scales.append(torch.where(held_t[..., 0], byte, torch.full_like(byte, 255)).to(torch.uint8))
        k_scales, v_scales = (x.view(torch.float8_e8m0fnu) for x in scales)
    t = dict(table=torch.from_numpy(table), lens=torch.tensor(b.lens, dtype=torch.int32),
             cu=torch.tensor(np.concatenate([[0], np.cumsum(b.new)]), dtype=torch.int32), q=normal(b.hq, b.total, b.d),
             k=normal(b.hkv, b.total, b.d), v=normal(b.hkv, b.total, b.d), k_pages=pages[0], v_pages=pages[1],
             k_scales=k_scales, v_scales=v_scales)
    return {x: (y.to(device) if y is not None else None) for x, y in t.items()}


def handles(fcp, b: Batch, t):
    cache = fcp.PagedCache.wrap(t["k_pages"], t["v_pages"], t["k_scales"], t["v_scales"])
    most = b.max_new if b.max_new >= 0 else max([0] + b.new)
    return cache, fcp.CacheBatch(t["cu"], t["lens"], t["table"], b.total, max_new=most)


def values(pages, scales):
    """The pages' values in float64, [n_pages, Hkv, page, D]."""
    if scales is None:
        return pages.double().cpu().numpy()
    codes, byte = pages.view(torch.uint8).cpu().numpy(), scales.view(torch.uint8).cpu().numpy().astype(np.int64)
    scale = np.where(byte == 255, np.nan, np.exp2(np.minimum(byte, 254) - 127.0))
    return R.e4m3_values()[codes] * scale[..., None]


def sequence_rows(pages, table, i, length, page, h):
    pos = np.arange(length)
    return pages[table[i, pos // page], h, pos % page]


def check_attention(b: Batch, t, o, lse, before_o=None, before_lse=None):
    kp, vp = values(t["k_pages"], t["k_scales"]), values(t["v_pages"], t["v_scales"])
    table, q = t["table"].cpu().numpy(), t["q"].double().cpu().numpy()
    got_o, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    err_sum = bound_sum = 0.0
    row = 0
    for i, (n, length) in enumerate(zip(b.new, b.lens)):
        for h in range(b.hkv if n else 0):
            k, v = (sequence_rows(x, table, i, length, b.page, h) for x in (kp, vp))
            for hh in range(h * b.hq // b.hkv, (h + 1) * b.hq // b.hkv):
                ro, rl, spread, rms, size = R.attend(q[hh, row:row + n], k, v, n, b.causal)
                go, gl = got_o[hh, row:row + n], got_l[hh, row:row + n]
                where = f"sequence {i} head {hh}"
                empty = np.isneginf(rl)
                assert np.array_equal(empty, np.isneginf(gl)), (where, rl, gl)
                assert not go[empty].any(), where
                err = np.abs(go - ro)
                assert np.isfinite(err).all(), where
                bound = 2.0 ** -8 * (spread + np.abs(ro)) + 2.0 ** -12 * spread + 1e-30
                assert (err <= bound).all(), (where, float((err / bound).max()), np.argwhere(err > bound)[:4])
                le = np.abs(gl[~empty] - rl[~empty])
                lb = b.d * 2.0 ** -24 * size[~empty] + 2.0 ** -20 * (1 + np.abs(rl[~empty]))
                assert (le <= lb).all(), (where, float((le / lb).max()))
                err_sum += err.sum()
                bound_sum += (2.0 ** -8 * (rms + np.abs(ro)) + 2.0 ** -12 * spread).sum()
        row += n
    assert err_sum <= bound_sum, (err_sum, bound_sum)
    if before_o is not None:
        assert torch.equal(o[:, row:], before_o[:, row:]) and torch.equal(lse[:, row:], before_lse[:, row:])
