"""A server's step around the paged key/value cache: pages for the new tokens, rotary positions, and a cache held in
4 bits with the attention that reads it. The cases that are measured, the operators in plain form, and the calls that a
user makes of them.

  pages   sequences are cut back to ``keep`` tokens (their last whole pages return to the stack of free ones) and
          get ``new`` tokens each: pages from the stack, entries of the block table, lengths, row offsets, and for every
          packed row its position and its slot (page * page_size + row of the page)
  rotary  pairs of channels of q [Hq, T, D] and k [Hkv, T, D] turned by position * frequency, or their gradients turned back
  place   the same for a batch's new tokens, with the turned k and v written to the pages of a bf16 or e4m3 cache
  store   new tokens' K and V into the pages of a 4-bit cache and read back as bf16
  read    the rows of whole sequences of a 4-bit cache as bf16
  attn    softmax(q K^T / sqrt(D)) V of the new tokens' queries over a 4-bit cache, and each row's log-sum-exp

A 4-bit cache holds e2m1 codes, two to a byte (the even channel in the low half), ``k_pages`` and ``v_pages``
[n_pages, Hkv, page_size, D / 2], and an e4m3 scale for every 16 channels, ``k_scales`` and ``v_scales``
[n_pages, Hkv, page_size, D / 16]; a code stands for code * scale * unit with a power of two ``unit`` for K and one for V.
Writing takes scale = e4m3(max|x| / (6 * unit)), 2^-9 at least, and the codes nearest to x / (scale * unit). Batches are
those of a paged cache: ``new[i]`` packed rows of sequence i, ``lens[i]`` its cached tokens with the new ones, position p
in row p % page_size of page ``table[i, p // page_size]``.
"""
import math

import numpy as np
import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
K_UNIT, V_UNIT = 1.0, 0.25


def listed():
    def pages(name, n, new, length, page, drop=0, pick=0):
        return dict(name=name, op="pages", n=n, new=new, len=length, page=page, drop=drop, pick=pick)

    def rotary(name, tokens, hq, hkv, d, part, pairs, far=0, back=False, scaling="none"):
        return dict(name=name, op="rotary", tokens=tokens, hq=hq, hkv=hkv, d=d, part=part, pairs=pairs, far=far, back=back,
                    scaling=scaling)

    def serve(name, op, n, new, length, hq, hkv, d, page, shape="ragged", causal=True, pad=0, pick=0, cache="e2m1", part=0):
        return dict(name=name, op=op, n=n, new=new, len=length, hq=hq, hkv=hkv, d=d, page=page, shape=shape, causal=causal,
                    pad=pad, pick=pick, cache=cache, part=part)

    return [
        # a busy server's step: one new token for each conversation
        pages("pages_step", 128, 1, 8192, 64, pick=1),
        # prompts of many lengths beside conversations whose last drafts were refused
        pages("pages_prompts", 300, 16384, 16384, 16, drop=5, pick=2),
        # a training batch of 32768 tokens before its attention
        rotary("rotary_train", 32768, 64, 8, 128, 128, "half"),
        # the gradients of a small model with turned pairs side by side in half of each head
        rotary("rotary_back_part", 3578, 4, 2, 64, 32, "adjacent", back=True),
        # a step of a busy server, far into long documents, into an e4m3 cache
        serve("place_step_e4m3", "place", 128, 1, 131072, 64, 8, 128, 64, pick=3, cache="e4m3", part=128),
        # prompts of many lengths into a bf16 cache
        serve("place_prompts_bf16", "place", 16, 16384, 16384, 64, 8, 128, 64, pick=4, pad=5, cache="bf16", part=64),
        # the same prompts kept in 4 bits
        serve("store_prompts", "store", 16, 16384, 16384, 8, 8, 128, 64, pick=5),
        # one token each for a few short conversations: latency
        serve("attn_step_few", "attn", 4, 1, 333, 4, 2, 64, 16, pick=6),
        # the step of a busy server: many conversations of very different lengths
        serve("attn_step_batch", "attn", 128, 1, 8192, 64, 8, 128, 64, pick=7),
        # drafted tokens checked in one pass, four for each sequence
        serve("attn_drafts", "attn", 32, 4, 4096, 32, 8, 128, 32, pick=8),
        # chunks of prompts behind what is cached already, of odd sizes, beside single tokens
        serve("attn_chunk_mixed", "attn", 9, 701, 6007, 32, 4, 128, 16, pad=3, pick=9),
        # one long chunk deep in a long document: the largest products
        serve("attn_chunk_long", "attn", 1, 2048, 32768, 64, 8, 128, 64, shape="equal"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["pages", "rotary", "place", "store", "read", "attn", "attn", "attn"])
    page, pick = rng.choice([16, 32, 64, 128, 256]), rng.randrange(1 << 16)
    if op == "pages":
        case = dict(op=op, n=log(1, 2000), new=rng.choice([1, log(2, 16384)]), len=log(16, 65536), page=page,
                    drop=rng.choice([0, 0, rng.randint(1, 40)]), pick=pick)
        case["len"] = max(case["len"], case["new"])
        while case["n"] * case["len"] > 1 << 22:
            case["n"] = max(1, case["n"] * 2 // 3)
        return case
    d = rng.choice([64, 128, 128])
    part = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
    if op == "rotary":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 3, 4, 8])
        return dict(op=op, tokens=log(1, 32768), hq=hq, hkv=hkv, d=d, part=part, pairs=rng.choice(["half", "adjacent"]),
                    far=rng.choice([0, log(1, 1 << 20)]), back=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]))
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 8]) if op in ("attn", "place") else 1
    case = dict(op=op, n=log(1, 128), new=1, len=log(16, 65536), hq=hkv * group, hkv=hkv, d=d, page=page,
                shape=rng.choice(["equal", "ragged", "ragged"]), causal=True, pad=rng.choice([0, 0, 1, 7]), pick=pick,
                cache=rng.choice(["bf16", "e4m3"]) if op == "place" else "e2m1", part=part if op == "place" else 0)
    if op == "attn":
        case["new"] = rng.choice([1, 1, rng.randint(2, 16), log(17, 2048)])
        case["causal"] = rng.random() < 0.8
    else:
        case["new"] = rng.choice([1, log(2, 16384)])
    # no drawn case costs more than the largest listed one, nor takes more memory in its plain form
    while True:
        case["len"] = max(case["len"], case["new"])
        rows = case["n"] * case["len"] * hkv * d
        pairs = case["n"] * case["new"] * case["len"] * case["hq"]
        moved = case["n"] * case["new"] * (case["hq"] + 2 * hkv) * d
        if rows <= 1 << 29 and (pairs <= 1 << 31 if op == "attn" else moved <= 1 << 29):
            return case
        if case["n"] > 1:
            case["n"] = max(1, case["n"] * 2 // 3)
        else:
            case["len"] = max(16, case["len"] * 2 // 3)
            case["new"] = min(case["new"], case["len"])


def _lengths(case):
    """(new, lens) of every sequence, lens with the new ones: a property of the case, not of the seed."""
    n, new, longest = case["n"], case["new"], case["len"]
    if case.get("shape") == "equal":
        return np.full(n, new, np.int64), np.full(n, longest, np.int64)
    r = np.random.RandomState(case["pick"])
    lens = np.clip(np.exp(r.normal(math.log(max(2.0, longest / 3.0)), 0.8, n)), 1, longest).astype(np.int64)
    lens[0] = longest
    fresh = np.maximum(1, np.round(np.exp(r.uniform(0, math.log(max(new, 1) + 0.5), n)))).astype(np.int64)
    fresh[r.randint(n)] = new
    fresh = np.minimum(np.minimum(fresh, new), lens)
    if n >= 4 and new > 1:
        fresh[1] = 0  # a conversation that waits
        lens[2] = fresh[2]  # one that begins with this batch
    if case["op"] == "read":
        fresh = lens.copy()  # whole sequences
    return fresh, lens


def work(case):
    op = case["op"]
    if op == "rotary":
        return {"bytes": 2 * 2 * case["tokens"] * (case["hq"] + case["hkv"]) * case["d"] + 4 * case["tokens"],
                "flops": 6 * case["tokens"] * (case["hq"] + case["hkv"]) * (case["part"] // 2)}
    new, lens = _lengths(case)
    T = int(new.sum())
    if op == "pages":
        n, page = case["n"], case["page"]
        back = int((-(-lens // page) - -(-(lens - new) // page)).sum())  # pages returned, and taken again
        return {"bytes": 4 * (6 * n + 1) + 4 * 4 * back + 12 * T, "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = {"bf16": 2 * d * 2, "e4m3": 2 * (d + 1), "e2m1": 2 * (d // 2 + d // 16)}[case["cache"]]  # K and V of a token and head
    if op == "place":
        return {"bytes": T * (hq * 2 * d * 2 + hkv * (2 * d * 2 + row)), "flops": 6 * T * (hq + hkv) * (case["part"] // 2)}
    if op == "store":
        return {"bytes": T * hkv * (2 * (2 * d * 2) + 2 * row), "flops": 0}
    if op == "read":
        return {"bytes": T * hkv * (2 * d * 2 + row), "flops": 0}
    pairs = sum(int(a) * int(b) - (int(a) * (int(a) - 1) // 2 if case["causal"] else 0) for a, b in zip(new, lens))
    cached = int(lens[new > 0].sum())
    return {"bytes": cached * hkv * row + T * hq * (2 * d * 2 + 4), "flops": 4 * hq * d * pairs}


def _frequencies(part, scaling, base=10000.0):
    """Radians a position of each pair, and the factor that the turned pairs get."""
    f = base ** (-2.0 * torch.arange(part // 2, dtype=torch.float64) / part)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "yarn":  # 16 times the 4096 positions of training; fast pairs stay, slow ones are stretched
        low, high = (part * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), part // 2 - 1)
        slow = ((torch.arange(part // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - slow) + f / 16 * slow, 0.1 * math.log(16.0) + 1
    return f, 1.0


_SCALING = {"none": None, "linear": dict(kind="linear", factor=8.0),
            "yarn": dict(kind="yarn", factor=16.0, original=4096)}


def _power(k):
    """2^k in float32 for whole k in [-126, 127]."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise8(x):
    """bf16 rows [..., D] as (e4m3 codes, e8m0 scales): the smallest 2^k, k >= -126, with amax <= 448 * 2^k."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m * 2^e with m in [0.5, 1)
    k = torch.where(m > 0.875, e - 8, e - 9).to(torch.int32).clamp(-126, 126)
    k = torch.where(m == 0, torch.zeros_like(k), k)
    codes = (x * _power(-k).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _quantise4(x, unit):
    """bf16 rows [..., D] as (packed e2m1 codes, e4m3 scales of 16 channels)."""
    x = x.float().unflatten(-1, (-1, 16)) / unit
    s = (x.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    y = x / s.unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
            + 8 * (y < 0).to(torch.uint8)).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), s.to(torch.float8_e4m3fn)


def _dequantise4(packed, scales, unit):
    """Float32 rows of packed codes (uint8)."""
    table = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float32, device=packed.device)
    x = torch.stack([table[(packed & 15).int()], table[(packed >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * (scales.float() * unit).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)

    if case["op"] == "rotary":
        s = {x: case[x] for x in ("op", "part", "pairs", "back", "scaling")}
        # packed sequences of the batch, each from its own first position on
        at = np.concatenate([[0], np.sort(r.choice(case["tokens"], min(7, case["tokens"]), replace=False))])
        first = np.maximum.accumulate(np.where(np.isin(np.arange(case["tokens"]), at), np.arange(case["tokens"]), 0))
        s["positions"] = ints(np.arange(case["tokens"]) - first + case["far"])
        s["q"], s["k"] = (normal(case[h], case["tokens"], case["d"]) for h in ("hq", "hkv"))
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        if own:
            import context_parallelism_fcp_gb300 as fcp

            s["rotary"] = fcp.Rotary(case["part"], interleaved=case["pairs"] == "adjacent", scaling=_SCALING[case["scaling"]])
        return s

    new, lens = _lengths(case)
    n, page = case["n"], case["page"]
    before = lens - new if case["op"] == "pages" else lens
    had = -(-before // page)  # pages that a sequence has
    need = -(-lens // page)
    n_pages = int(need.sum()) + 3
    table = np.full((n, max(1, int(need.max()))), -1, np.int32)
    ids = r.permutation(n_pages)
    ends = np.cumsum(had)
    for i in range(n):
        table[i, :had[i]] = ids[ends[i] - had[i]:ends[i]]
    s = dict(op=case["op"], page=page, table=ints(table), lens=ints(before))
    if case["op"] == "pages":
        T = int(new.sum()) + 7  # rows that no sequence gets, as in a batch of fixed size
        left = np.zeros(n_pages, np.int32)
        left[:n_pages - int(had.sum())] = ids[int(had.sum()):]
        keep = np.maximum(0, before - (r.randint(0, case["drop"] + 1, n) if case["drop"] else 0))
        s.update(free=ints(left), n_free=ints([n_pages - int(had.sum())]), keep=ints(keep), new=ints(new), T=T,
                 cu=torch.zeros(n + 1, dtype=torch.int32, device=dev), granted=torch.zeros(n, dtype=torch.int32, device=dev),
                 positions=torch.zeros(T, dtype=torch.int32, device=dev), slots=torch.zeros(T, dtype=torch.int64, device=dev))
        if own:
            import context_parallelism_fcp_gb300 as fcp

            s["pool"] = fcp.PagePool.wrap(s["free"], s["n_free"], s["lens"], s["table"], page, cu_new=s["cu"],
                                          granted=s["granted"])
        return s

    hkv, d, T = case["hkv"], case["d"], int(new.sum()) + case["pad"]
    s.update(causal=case["causal"], rows=int(new.sum()), longest=int(lens.max()), most_new=max(1, int(new.max())),
             part=case["part"], cu=ints(np.concatenate([[0], np.cumsum(new)])))
    shape, pages, scales = (n_pages, hkv, page, d), [], []
    for unit in (K_UNIT, V_UNIT):
        if case["cache"] != "e2m1":
            x = normal(*shape)
            x, z = (x, None) if case["cache"] == "bf16" else _quantise8(x)
        else:  # rows of different sizes, some channels far larger than others, as keys have them
            size = torch.exp2(torch.randint(-2, 3, (*shape[:3], 1), generator=g, device=dev).to(torch.bfloat16))
            wide = torch.where(torch.arange(d, device=dev) % 29 == 3, 4.0, 1.0).to(torch.bfloat16)
            x = torch.empty(*shape[:3], d // 2, dtype=torch.uint8, device=dev)
            z = torch.empty(*shape[:3], d // 16, dtype=torch.float8_e4m3fn, device=dev)
            step = max(1, (1 << 26) // (hkv * page * d))
            for p in range(0, n_pages, step):
                some = slice(p, p + step)
                rows = normal(*x[some].shape[:3], d) * size[some] * wide
                x[some], z[some] = _quantise4(rows, unit)
        pages.append(x)
        scales.append(z)
    s.update(k_pages=pages[0], v_pages=pages[1], k_scales=scales[0], v_scales=scales[1])
    if case["op"] in ("attn", "place"):
        s["q"] = normal(case["hq"], T, d)
        s["o"] = torch.zeros(case["hq"], T, d, dtype=torch.bfloat16, device=dev)
    if case["op"] == "attn":
        s["lse"] = torch.zeros(case["hq"], T, dtype=torch.float32, device=dev)
    else:
        s["k"], s["v"] = normal(hkv, T, d), normal(hkv, T, d)
        s["k_back"], s["v_back"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    if own:
        import context_parallelism_fcp_gb300 as fcp

        if case["cache"] == "e2m1":
            s["cache"] = fcp.PagedCache.wrap(*(s[x].view(torch.float4_e2m1fn_x2) for x in ("k_pages", "v_pages")),
                                             s["k_scales"], s["v_scales"], k_unit=K_UNIT, v_unit=V_UNIT)
        else:
            s["cache"] = fcp.PagedCache.wrap(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        s["batch"] = fcp.CacheBatch(s["cu"], s["lens"], s["table"], T, max_new=s["most_new"])
        if case["op"] == "attn":
            s["attention"] = fcp.PagedAttention(s["cache"], case["hq"], causal=case["causal"])
        if case["op"] == "place":
            s["rotary"] = fcp.Rotary(case["part"], scaling=_SCALING["yarn"])
    return s


def run(s):
    if own:
        import context_parallelism_fcp_gb300 as fcp

        if s["op"] == "pages":
            s["pool"].release(s["keep"])
            s["pool"].admit(s["new"], s["positions"], s["slots"])
            return _pages_state(s)
        if s["op"] == "rotary":
            if s["back"]:
                return fcp.rotary_backward(s["rotary"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
            return fcp.rotary_apply(s["rotary"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        if s["op"] == "attn":
            return s["attention"].forward(s["batch"], s["q"], s["o"], s["lse"])
        if s["op"] == "place":
            fcp.rotary_write(s["cache"], s["batch"], s["rotary"], s["q"], s["k"], s["v"], s["o"])
            return [s["o"], *_pool(s)]
        if s["op"] == "store":
            fcp.cache_write(s["cache"], s["batch"], s["k"], s["v"])
        fcp.cache_read(s["cache"], s["batch"], s["k_back"], s["v_back"])
        return s["k_back"], s["v_back"]
    return {"pages": _pages, "rotary": _rotary, "attn": _attn, "place": _place, "store": _store, "read": _read}[s["op"]](s)


def _pool(s):
    return [s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales") if s[x] is not None]


def _pages_state(s):
    return {x: s[x] for x in ("free", "n_free", "lens", "table", "cu", "granted", "positions", "slots")}


def _scatter(to, at, on, values):
    """to[at] = values where `on`; the others land behind the end and are dropped."""
    more = torch.cat([to.flatten(), to.new_zeros(1)])
    more[torch.where(on, at, to.numel()).flatten()] = values.to(to.dtype).flatten()
    to.copy_(more[:-1].view_as(to))


def _pages(s):
    page, table, free = s["page"], s["table"], s["free"]
    n, width = table.shape
    column = torch.arange(width, device=table.device)[None]
    row0 = torch.arange(n, device=table.device)[:, None] * width
    # back to `keep` tokens: pages behind them go to the stack, sequence by sequence
    lens = torch.minimum(s["lens"], torch.where(s["keep"] < 0, s["lens"], s["keep"])).long()
    old, left = (s["lens"].long() + page - 1) // page, (lens + page - 1) // page
    back = (column >= left[:, None]) & (column < old[:, None])
    place = back.flatten().long().cumsum(0).view_as(back) - 1 + s["n_free"].long()
    _scatter(free, place, back, table)
    table.masked_fill_(back, -1)
    n_free = s["n_free"].long() + back.sum()
    # `new` tokens each, first come first served: pages from the stack's top
    want = s["new"].long()
    whole = (lens + want + page - 1) // page
    fits = (want >= 0) & (whole <= width)
    want = torch.where(fits, want, 0)
    need = torch.where(fits, whole - left, 0)
    pages_to = need.cumsum(0)
    want = torch.where((need == 0) | (pages_to <= n_free), want, 0)
    want = torch.where(want.cumsum(0) <= s["T"], want, 0)
    need = torch.where(want > 0, need, 0)
    first = need.cumsum(0) - need
    k = column - left[:, None]
    mine = (k >= 0) & (k < need[:, None])
    at = n_free - 1 - (first[:, None] + k)
    _scatter(table, row0 + column, mine, free[at.clamp(0, free.numel() - 1)])
    s["n_free"].copy_(n_free - need.sum())
    s["cu"][1:] = want.cumsum(0)
    s["granted"].copy_(want)
    s["lens"].copy_(lens + want)
    # packed rows
    row = torch.arange(s["T"], device=table.device, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    on = seq < n
    seq = seq.clamp(max=n - 1)
    position = torch.where(on, lens[seq] + row - s["cu"][seq], -1)
    slot = table[seq, (position // page).clamp(min=0)].long() * page + position % page
    s["positions"].copy_(position)
    s["slots"].copy_(torch.where(on, slot, -1))
    return _pages_state(s)


def _turned(x, positions, part, pairs, scaling, back=False):
    f, size = _frequencies(part, scaling)
    angle = positions.double()[:, None] * f.to(x.device)
    c, z = (angle.cos() * size).float(), (angle.sin() * size).float()
    if back:
        z = -z
    y = x.float()
    if pairs == "half":
        a, b = y[..., :part // 2], y[..., part // 2:part]
        turned = torch.cat([a * c - b * z, b * c + a * z], -1)
    else:
        a, b = y[..., :part:2], y[..., 1:part:2]
        turned = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    return torch.cat([turned, y[..., part:]], -1).to(torch.bfloat16)


def _rotary(s):
    for x in ("q", "k"):
        s[x + "_out"].copy_(_turned(s[x], s["positions"], s["part"], s["pairs"], s["scaling"], s["back"]))
    return s["q_out"], s["k_out"]


def _rows(s):
    """Sequence, index among its new tokens, and position of each packed row."""
    row = torch.arange(s["rows"], device=s["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    tok = row - s["cu"][seq]
    return seq, tok, s["lens"][seq] - (s["cu"][seq + 1] - s["cu"][seq]) + tok


def _places(s):
    seq, _, pos = _rows(s)
    return s["table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()


def _place(s):
    page, off = _places(s)
    rows, positions = s["rows"], _rows(s)[2]
    s["o"][:, :rows] = _turned(s["q"][:, :rows], positions, s["part"], "half", "yarn")
    for x in ("k", "v"):
        y = s[x][:, :rows]
        y = (_turned(y, positions, s["part"], "half", "yarn") if x == "k" else y).transpose(0, 1)
        if s[x + "_scales"] is None:
            s[x + "_pages"][page, :, off] = y
        else:
            codes, scales = _quantise8(y)
            s[x + "_pages"].view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
            s[x + "_scales"].view(torch.uint8)[page, :, off] = scales.view(torch.uint8)
    return [s["o"], *_pool(s)]


def _store(s):
    page, off = _places(s)
    for x, unit in (("k", K_UNIT), ("v", V_UNIT)):
        codes, scales = _quantise4(s[x][:, :s["rows"]].transpose(0, 1), unit)
        s[x + "_pages"][page, :, off] = codes
        s[x + "_scales"].view(torch.uint8)[page, :, off] = scales.view(torch.uint8)
    return _read(s)


def _read(s):
    page, off = _places(s)
    for x, unit in (("k", K_UNIT), ("v", V_UNIT)):
        rows = _dequantise4(s[x + "_pages"][page, :, off], s[x + "_scales"].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn), unit)
        s[x + "_back"][:, :s["rows"]] = rows.transpose(0, 1).to(torch.bfloat16)
    return s["k_back"], s["v_back"]


def _attn(s):
    q, m, n = s["q"], s["most_new"], s["lens"].numel()
    hq, _, d = q.shape
    hkv = s["k_pages"].shape[1]
    seq, tok, _ = _rows(s)
    slot = seq * m + tok
    new = s["cu"][1:] - s["cu"][:-1]
    table = s["table"].clamp(min=0).long()

    def rows(x, unit):  # [n, Hkv, longest, D] in float32
        y = _dequantise4(s[x + "_pages"][table], s[x + "_scales"].view(torch.uint8)[table].view(torch.float8_e4m3fn), unit)
        return y.permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)[:, :, :s["longest"]]

    k, v = rows("k", K_UNIT), rows("v", V_UNIT)
    at = torch.arange(k.shape[2], device=q.device)
    held = at[None, :] < s["lens"][:, None]
    v = torch.where(held[:, None, :, None], v, 0.0)
    padded = torch.zeros(hq, n * m, d, device=q.device)
    padded[:, slot] = q[:, :s["rows"]].float()
    padded = padded.view(hkv, hq // hkv, n, m, d).permute(2, 0, 1, 3, 4).reshape(n, hkv, -1, d)
    seen = held[:, None, :]
    if s["causal"]:
        place = (s["lens"] - new)[:, None] + torch.arange(m, device=q.device)
        seen = seen & (at[None, None, :] <= place[:, :, None])
    seen = seen[:, None, None].expand(n, hkv, hq // hkv, m if s["causal"] else 1, at.numel())
    x = (padded @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(n, hkv, hq // hkv, m, -1)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(n, hkv, -1, at.numel()) @ v).view(n, hkv, hq // hkv, m, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    s["o"][:, :s["rows"]] = o.permute(1, 2, 0, 3, 4).reshape(hq, n * m, d)[:, slot].to(torch.bfloat16)
    s["lse"][:, :s["rows"]] = lse.permute(1, 2, 0, 3).reshape(hq, n * m)[:, slot]
    return s["o"], s["lse"]


def exact(case, seed):
    """The definitions in 64 bits. Pages are whole numbers, and have no such value."""
    op = case["op"]
    if op == "pages":
        return None
    s = prepare(case, seed)

    def turn(x, positions, part, adjacent, scaling, back):
        y = x.double()
        for i in range(part // 2):
            f, size = 10000.0 ** (-2.0 * i / part), 1.0
            if scaling == "linear":
                f /= 8.0
            elif scaling == "yarn":
                edge = [part * math.log(4096 / (2 * math.pi * turns)) / math.log(10000.0) / 2 for turns in (32, 1)]
                edge = [max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), part // 2 - 1)]
                slow = min(max((i - edge[0]) / max(edge[1] - edge[0], 0.001), 0.0), 1.0)
                f, size = f * (1 - slow) + f / 16 * slow, 0.1 * math.log(16) + 1
            pair = torch.complex(positions.double() * 0, positions.double() * f * (-1.0 if back else 1.0)).exp() * size
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + part // 2)
            z = torch.complex(x[..., a].double(), x[..., b].double()) * pair
            y[..., a], y[..., b] = z.real, z.imag
        return y

    if op == "rotary":
        return tuple(turn(s[x], s["positions"], case["part"], case["pairs"] == "adjacent", case["scaling"], case["back"])
                     for x in ("q", "k"))

    new, lens = _lengths(case)
    page, d, hkv, group = case["page"], case["d"], case["hkv"], case["hq"] // case["hkv"]
    table = s["table"].cpu().numpy()
    ends = np.cumsum(new)
    unit = {"k": K_UNIT, "v": V_UNIT}
    if op in ("attn", "store", "read") and (work(case)["flops"] > 3e12 or case["n"] * hkv > 4096):
        return None

    def two(k):  # 2^k for whole k, exactly
        return ((k.long() + 1023) << 52).view(torch.float64)

    def where(i, first):  # pages and rows of the positions first .. of sequence i
        pos = np.arange(first, int(lens[i]))
        return (torch.from_numpy(table[i, pos // page].astype(np.int64)).cuda(),
                torch.from_numpy((pos % page).astype(np.int64)).cuda())

    def stored(x, h, i, first=0):  # rows of a 4-bit cache
        pg, off = where(i, first)
        byte = s[x + "_pages"][:, h][pg, off]
        code = torch.stack([byte % 16, byte // 16], -1).reshape(len(pg), d).long()
        m, e = code % 2, code // 2 % 4
        value = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * two(e - 1)) * torch.where(code >= 8, -1.0, 1.0)
        scale = s[x + "_scales"][:, h].view(torch.uint8)[pg, off].view(torch.float8_e4m3fn).double() * unit[x]
        return value * scale.repeat_interleave(16, -1)

    def nearest(y, bits, least):  # to so many bits behind the leading one, ties to even, steps of 2^least at least
        e = torch.frexp(y.abs())[1] - 1
        step = two((e - bits).clamp(min=least))
        return torch.round(y / step) * step

    if op == "attn":
        o, lse = s["o"].double(), s["lse"].double()
        for i in range(case["n"]):
            if new[i] == 0:
                continue
            a, b, L, m = int(ends[i] - new[i]), int(ends[i]), int(lens[i]), int(new[i])
            mask = torch.arange(L, device=o.device)[None, :] > L - m + torch.arange(m, device=o.device)[:, None]
            for h in range(hkv):
                k, v = stored("k", h, i), stored("v", h, i)
                for j in range(h * group, (h + 1) * group):
                    z = s["q"][j, a:b].double() @ k.T / math.sqrt(d)
                    if case["causal"]:
                        z[mask] = -math.inf
                    lse[j, a:b] = torch.logsumexp(z, -1)
                    o[j, a:b] = torch.softmax(z, -1) @ v
        return o, lse
    if op in ("store", "read"):
        out = []
        for x in ("k", "v"):
            r = s[x + "_back"].double()
            for i in range(case["n"]):
                a, b = int(ends[i] - new[i]), int(ends[i])
                if op == "read":
                    for h in range(hkv):
                        r[h, a:b] = stored(x, h, i, int(lens[i] - new[i]))
                else:
                    y = s[x][:, a:b].double().reshape(hkv, b - a, d // 16, 16) / unit[x]
                    scale = nearest((y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0), 3, -9).clamp(min=2.0 ** -9)
                    y = nearest(y / scale, 1, -1).clamp(-6.0, 6.0)
                    r[:, a:b] = (y * scale * unit[x]).reshape(hkv, b - a, d)
            out.append(r)
        return tuple(out)

    # place: q turned; k turned, rounded to bf16, and v, in their pages
    positions = torch.from_numpy(np.concatenate([np.arange(b - a, b) for a, b in zip(new, lens)])).cuda()
    rows = int(new.sum())
    o = s["o"].double()
    o[:, :rows] = turn(s["q"][:, :rows], positions, case["part"], False, "yarn", False)
    out = {x: s[x].double() for x in ("k_pages", "v_pages", "k_scales", "v_scales") if s[x] is not None}
    for x in ("k", "v"):
        y = s[x][:, :rows].double()
        if x == "k":
            y = turn(s[x][:, :rows], positions, case["part"], False, "yarn", False).to(torch.bfloat16).double()
        for i in range(case["n"]):
            if new[i] == 0:
                continue
            pg, off = where(i, int(lens[i] - new[i]))
            z = y[:, int(ends[i] - new[i]):int(ends[i])].transpose(0, 1)
            if case["cache"] == "e4m3":
                top = z.abs().amax(-1, keepdim=True)
                top = torch.where(top == 0, 448.0, top)
                k = torch.ceil(torch.log2(top / 448.0))
                k = k + (top > 448.0 * two(k)).double() - (top <= 448.0 * two(k - 1)).double()
                out[x + "_scales"][pg, :, off] = two(k).squeeze(-1)
                z = nearest(z / two(k), 3, -9)
            out[x + "_pages"][pg, :, off] = z
    return [o, *out.values()]
