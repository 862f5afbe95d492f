"""Batches over a 4-bit paged cache for the tests: those of paged_util with e2m1 pages, whose rows past
the sequences' ends and whose unused pages hold NaN scales.

Tolerances are paged_util's: code * scale is exact in f16, which the products run in, so the kernels
compute the attention over the stored values with P rounded to f16, by at most 2^-11 of itself or
2^-32 of the row's largest weight, where paged_util allows bf16's 2^-8 of itself. Q is scaled by a power
of two on its way to f16, which loses what is below 2^-28 of its row's largest element: less than
float32's sums do."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged4 as R4
from tests import paged_util as U
from tests.paged_util import Batch  # noqa: F401 (the tests' batches)

K_UNIT, V_UNIT = 0.5, 4.0


def make(b, device="cuda", lo=0x10, hi=0x40):
    """paged_util.make with e2m1 pages; scales are e4m3 bytes from lo to hi - 1 (2^-5 to 2 by default)."""
    plain = U.make(type(b)(**{**b.__dict__, "cache": "bf16"}), device="cpu")
    g = torch.Generator().manual_seed(b.seed + 1)
    held = ~plain["k_pages"][..., 0].isnan()  # [n_pages, Hkv, page]
    t = {x: (y.to(device) if y is not None else None) for x, y in plain.items()}
    for x in "kv":
        packed = torch.randint(0, 256, (*held.shape, b.d // 2), generator=g, dtype=torch.int32).to(torch.uint8)
        scale = torch.randint(lo, hi, (*held.shape, b.d // 16), generator=g, dtype=torch.int32)
        scale = torch.where(held[..., None], scale, torch.full_like(scale, 0x7F)).to(torch.uint8)
        t[x + "_pages"] = packed.to(device).view(torch.float4_e2m1fn_x2)
        t[x + "_scales"] = scale.to(device).view(torch.float8_e4m3fn)
    return t


def handles(fcp, b, t, k_unit=K_UNIT, v_unit=V_UNIT):
    cache = fcp.PagedCache.wrap(t["k_pages"], t["v_pages"], t["k_scales"], t["v_scales"], k_unit=k_unit, v_unit=v_unit)
    most = b.max_new if b.max_new >= 0 else max([0] + b.new)
    return cache, fcp.CacheBatch(t["cu"], t["lens"], t["table"], b.total, max_new=most)


def values(pages, scales, unit):
    """The pages' values in float64, [n_pages, Hkv, page, D]."""
    return R4.value(R4.unpack(pages.view(torch.uint8).cpu().numpy()), scales.view(torch.uint8).cpu().numpy(), unit)


def check_attention(b, t, o, lse, before_o=None, before_lse=None, k_unit=K_UNIT, v_unit=V_UNIT):
    full = {x: torch.from_numpy(values(t[x + "_pages"], t[x + "_scales"], u)) for x, u in (("k", k_unit), ("v", v_unit))}
    U.check_attention(b, {**t, "k_pages": full["k"], "v_pages": full["v"], "k_scales": None, "v_scales": None}, o, lse,
                      before_o, before_lse)
