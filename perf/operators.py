"""The paged key/value cache and the attention that reads it: the cases that are measured, the operators in plain
form, and the calls that a user makes of them.

A cache holds K and V in pages: ``k_pages`` and ``v_pages`` are [n_pages, Hkv, page_size, D], bf16 or e4m3. An e4m3
cache has a power-of-two scale for each row (token and head) of K and of V, ``k_scales`` and ``v_scales``
[n_pages, Hkv, page_size] in e8m0: the smallest 2^k with amax <= 448 * 2^k. Position p of sequence i is row
p % page_size of page ``table[i, p // page_size]``. A batch brings ``new[i]`` tokens for sequence i, packed behind one
another over T rows; ``lens[i]`` counts the sequence's cached tokens with the new ones, so new token j is position
lens[i] - new[i] + j.

  write  the new tokens' K and V [Hkv, T, D] into their pages (quantised where the cache is e4m3)
  read   the same rows back as bf16 [Hkv, T, D]
  attn   softmax(q K^T / sqrt(D)) V of the new tokens' queries [Hq, T, D] over their sequences' cached keys up to and
         with their own position (or over all of them), and the log-sum-exp of each row
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


def listed():
    def attn(name, n, new, length, hq, hkv, d, page, cache, shape="ragged", causal=True, pad=0, pick=0):
        return dict(name=name, op="attn", n=n, new=new, len=length, hq=hq, hkv=hkv, d=d, page=page, cache=cache,
                    shape=shape, causal=causal, pad=pad, pick=pick)

    def move(name, op, n, new, length, hkv, d, page, cache, shape="ragged", pad=0, pick=0):
        return dict(name=name, op=op, n=n, new=new, len=length, hq=hkv, hkv=hkv, d=d, page=page, cache=cache,
                    shape=shape, causal=True, pad=pad, pick=pick)

    return [
        # one token each for a few short conversations: latency
        attn("attn_step_few", 4, 1, 333, 4, 2, 64, 16, "bf16", pick=1),
        # the step of a busy server: many conversations of very different lengths, a quantised cache
        attn("attn_step_batch_e4m3", 128, 1, 8192, 64, 8, 128, 64, "e4m3", pick=2),
        # two documents near the longest context: few rows, a long axis
        attn("attn_step_long", 2, 1, 131072, 64, 8, 128, 128, "bf16", shape="equal"),
        # drafted tokens checked in one pass, four for each sequence
        attn("attn_drafts", 32, 4, 4096, 32, 8, 128, 32, "bf16", pick=3),
        # prompts taken in chunks of 512 behind what is cached already
        attn("attn_chunk", 4, 512, 16384, 64, 8, 128, 128, "bf16", pad=9, pick=4),
        # chunks of odd sizes beside single tokens, a small model with a quantised cache
        attn("attn_chunk_mixed_e4m3", 9, 701, 6007, 8, 2, 64, 16, "e4m3", pad=3, pick=5),
        # one long chunk deep in a long document, a quantised cache: the largest products
        attn("attn_chunk_long_e4m3", 1, 2048, 32768, 64, 8, 128, 64, "e4m3", shape="equal"),
        # a server's step writes one token for each conversation
        move("write_step_e4m3", "write", 128, 1, 8192, 8, 128, 64, "e4m3", pick=6),
        # prompts of many lengths written whole
        move("write_prompts_e4m3", "write", 16, 16384, 16384, 8, 128, 64, "e4m3", pick=7),
        move("write_prompts_bf16", "write", 7, 5001, 9001, 2, 64, 16, "bf16", pad=5, pick=8),
        # a shared prefix read back for training-style attention, and a preempted conversation saved
        move("read_prefix_e4m3", "read", 16, 16384, 16384, 8, 128, 64, "e4m3", pick=9),
        move("read_saved_bf16", "read", 3, 777, 2100, 4, 128, 32, "bf16", pad=2, pick=10),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn", "attn", "attn", "write", "read"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 8]) if op == "attn" else 1
    case = dict(op=op, n=log(1, 128), new=1, len=log(16, 65536), hq=hkv * group, hkv=hkv, d=rng.choice([64, 128, 128]),
                page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["bf16", "e4m3"]),
                shape=rng.choice(["equal", "ragged", "ragged"]), causal=rng.random() < 0.8, pad=rng.choice([0, 0, 1, 7]),
                pick=rng.randrange(1 << 16))
    if op == "attn":
        case["new"] = rng.choice([1, 1, rng.randint(2, 16), log(17, 2048)])
    else:
        case["new"] = rng.choice([1, log(2, 16384)])
        case["causal"] = True
    # no drawn case costs more than the largest listed one, nor takes more memory in its plain form
    while True:
        case["len"] = max(case["len"], case["new"])
        rows = case["n"] * case["len"] * hkv * case["d"]
        pairs = case["n"] * case["new"] * case["len"] * case["hq"]
        if rows <= 1 << 29 and (op != "attn" or pairs <= 1 << 31):
            return case
        if case["n"] > 1:
            case["n"] = max(1, case["n"] * 2 // 3)
        else:
            case["len"] = max(16, case["len"] * 2 // 3)
            case["new"] = min(case["new"], case["len"])


def _lengths(case):
    """(new, lens) of every sequence: a property of the case, not of the seed."""
    n, new, longest = case["n"], case["new"], case["len"]
    if case["shape"] == "equal":
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
    return fresh, lens


def work(case):
    new, lens = _lengths(case)
    T, hq, hkv, d = int(new.sum()), case["hq"], case["hkv"], case["d"]
    row = 2 * d * 2 if case["cache"] == "bf16" else 2 * (d + 1)  # K and V of one token and head, with their scales
    if case["op"] != "attn":
        return {"bytes": T * hkv * (2 * d * 2 + row), "flops": 0}
    pairs = sum(int(a) * int(b) - (int(a) * (int(a) - 1) // 2 if case["causal"] else 0) for a, b in zip(new, lens))
    cached = int(lens[new > 0].sum())
    return {"bytes": cached * hkv * row + T * hq * (2 * d * 2 + 4), "flops": 4 * hq * d * pairs}


def _power(k):
    """2^k in float32 for whole k in [-126, 127]."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """bf16 rows [..., D] as (e4m3 codes, e8m0 scales): the smallest 2^k, k >= -126, with amax <= 448 * 2^k."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m * 2^e with m in [0.5, 1)
    k = torch.where(m > 0.875, e - 8, e - 9).to(torch.int32).clamp(-126, 126)
    k = torch.where(m == 0, torch.zeros_like(k), k)
    codes = (x * _power(-k).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantise(codes, scales):
    return codes.float() if scales is None else codes.float() * scales.float().unsqueeze(-1)


def prepare(case, seed):
    dev = torch.device("cuda")
    new, lens = _lengths(case)
    n, page, hkv, d, T = case["n"], case["page"], case["hkv"], case["d"], int(new.sum()) + case["pad"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    need = -(-lens // page)
    n_pages = int(need.sum()) + 3
    table = np.full((n, max(1, int(need.max()))), -1, np.int32)
    ids = r.permutation(n_pages)
    at = 0
    for i in range(n):
        table[i, :need[i]] = ids[at:at + need[i]]
        at += int(need[i])

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    pages = [normal(n_pages, hkv, page, d) for _ in range(2)]
    scales = [None, None]
    if case["cache"] == "e4m3":
        pages, scales = zip(*[_quantise(p * torch.exp2(torch.randint(-2, 3, p.shape[:-1], generator=g, device=dev)
                                                       .to(torch.bfloat16)).unsqueeze(-1)) for p in pages])
    s = dict(op=case["op"], causal=case["causal"], page=page, rows=int(new.sum()), longest=int(lens.max()),
             most_new=max(1, int(new.max())), k_pages=pages[0], v_pages=pages[1], k_scales=scales[0],
             v_scales=scales[1], table=torch.from_numpy(table).to(dev),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev),
             lens=torch.from_numpy(lens.astype(np.int32)).to(dev))
    if case["op"] == "attn":
        s["q"] = normal(case["hq"], T, d)
        s["o"] = torch.zeros(case["hq"], T, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(case["hq"], T, dtype=torch.float32, device=dev)
    elif case["op"] == "write":
        s["k"], s["v"] = normal(hkv, T, d), normal(hkv, T, d)
    else:
        s["k"], s["v"] = (torch.zeros(hkv, T, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if own:
        import context_parallelism_fcp_gb300 as fcp

        s["cache"] = fcp.PagedCache.wrap(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        s["batch"] = fcp.CacheBatch(s["cu"], s["lens"], s["table"], T, max_new=s["most_new"])
        if case["op"] == "attn":
            s["attention"] = fcp.PagedAttention(s["cache"], case["hq"], causal=case["causal"])
    return s


def run(s):
    if own:
        import context_parallelism_fcp_gb300 as fcp

        if s["op"] == "attn":
            return s["attention"].forward(s["batch"], s["q"], s["o"], s["lse"])
        if s["op"] == "read":
            fcp.cache_read(s["cache"], s["batch"], s["k"], s["v"])
            return s["k"], s["v"]
        fcp.cache_write(s["cache"], s["batch"], s["k"], s["v"])
        return _pool(s)
    return {"attn": _attn, "write": _write, "read": _read}[s["op"]](s)


def _pool(s):
    return [s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales") if s[x] is not None]


def _rows(s):
    """Sequence, index among its new tokens, and position of each packed row."""
    row = torch.arange(s["rows"], device=s["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    tok = row - s["cu"][seq]
    return seq, tok, s["lens"][seq] - (s["cu"][seq + 1] - s["cu"][seq]) + tok


def _attn(s):
    q, page, m, n = s["q"], s["page"], s["most_new"], s["lens"].numel()
    hq, _, d = q.shape
    hkv = s["k_pages"].shape[1]
    seq, tok, _ = _rows(s)
    slot = seq * m + tok
    new = s["cu"][1:] - s["cu"][:-1]
    table = s["table"].clamp(min=0).long()

    def rows(pages, scales):  # [n, Hkv, longest, D] in float32
        x = _dequantise(pages[table], None if scales is None else scales[table])
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)[:, :, :s["longest"]]

    k, v = rows(s["k_pages"], s["k_scales"]), rows(s["v_pages"], s["v_scales"])
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


def _places(s):
    seq, _, pos = _rows(s)
    return s["table"][seq, pos // s["page"]].long(), (pos % s["page"]).long()


def _write(s):
    page, off = _places(s)
    for x in ("k", "v"):
        rows = s[x][:, :s["rows"]].transpose(0, 1)
        if s[x + "_scales"] is None:
            s[x + "_pages"][page, :, off] = rows
        else:
            codes, scales = _quantise(rows)
            s[x + "_pages"].view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
            s[x + "_scales"].view(torch.uint8)[page, :, off] = scales.view(torch.uint8)
    return _pool(s)


def _read(s):
    page, off = _places(s)
    for x in ("k", "v"):
        scales = s[x + "_scales"]
        rows = _dequantise(s[x + "_pages"][page, :, off], None if scales is None else scales[page, :, off])
        s[x][:, :s["rows"]] = rows.transpose(0, 1).to(torch.bfloat16)
    return s["k"], s["v"]


def exact(case, seed):
    """The definitions in 64 bits, one sequence and head at a time."""
    s = prepare(case, seed)
    new, lens = _lengths(case)
    page, d, hkv, group = case["page"], case["d"], case["hkv"], case["hq"] // case["hkv"]
    table = s["table"].cpu().numpy()
    ends = np.cumsum(new)

    def two(k):  # 2^k for whole k, exactly
        return ((k.long() + 1023) << 52).view(torch.float64)

    def where(i, first):  # pages and rows of the positions first .. of sequence i
        pos = np.arange(first, int(lens[i]))
        return (torch.from_numpy(table[i, pos // page].astype(np.int64)).cuda(),
                torch.from_numpy((pos % page).astype(np.int64)).cuda())

    def stored(x, h, i, first=0):
        pg, off = where(i, first)
        rows = s[x + "_pages"][:, h].float()[pg, off].double() if lens[i] else torch.zeros(0, d).cuda().double()
        if s[x + "_scales"] is not None:
            e = s[x + "_scales"].view(torch.uint8)[:, h][pg, off].double()
            rows = rows * two(e - 127)[:, None]
        return rows

    if case["op"] == "attn":
        if work(case)["flops"] > 3e12 or case["n"] * hkv > 4096:
            return None
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
    if case["op"] == "read":
        out = []
        for x in ("k", "v"):
            r = s[x].double()
            for h in range(hkv):
                for i in range(case["n"]):
                    if new[i]:
                        r[h, int(ends[i] - new[i]):int(ends[i])] = stored(x, h, i, int(lens[i] - new[i]))
            out.append(r)
        return tuple(out)
    out = {x: s[x].double() for x in ("k_pages", "v_pages", "k_scales", "v_scales") if s[x] is not None}
    for x in ("k", "v"):
        for i in range(case["n"]):
            if new[i] == 0:
                continue
            pg, off = where(i, int(lens[i] - new[i]))
            rows = s[x][:, int(ends[i] - new[i]):int(ends[i])].double().transpose(0, 1)
            if case["cache"] == "e4m3":
                amax = rows.abs().amax(-1, keepdim=True)
                amax = torch.where(amax == 0, E4M3_MAX, amax)
                k = torch.ceil(torch.log2(amax / E4M3_MAX))
                k = k + (amax > E4M3_MAX * two(k)).double() - (amax <= E4M3_MAX * two(k - 1)).double()
                scale = two(k.clamp(min=-126))
                y = rows / scale
                m, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))
                step = two(e - 4)
                rows = torch.round(y / step) * step  # e4m3: three bits behind the leading one, ties to even
                out[x + "_scales"][pg, :, off] = scale.squeeze(-1)
            out[x + "_pages"][pg, :, off] = rows
    return list(out.values())
