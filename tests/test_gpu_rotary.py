"""Rotary positions on the GPU against their float64 definition (oracle/rotary.py).

Tolerance: the angle is right to 2^-32 of a turn (2^-29 radians), m cos and m sin to two units (2^-22.9 m at
most), and two products and a sum round to float32 (2^-24 of the pair's size each); together below
2^-21 m (|a| + |b|). The result is rounded to bf16 once:
2^-8 of itself."""
import numpy as np
import pytest
import torch

from oracle import rotary as R
from tests import paged4_util as U4
from tests import paged_util as U
from tests.paged_util import Batch

pytestmark = pytest.mark.gpu


def check(rot, x, y, positions, backward=False):
    x = x.double().cpu().numpy()
    want, size = R.turn(x, positions.cpu().numpy(), rot.radians, rot.magnitude, rot.interleaved, backward)
    err = np.abs(y.double().cpu().numpy() - want)
    turned = np.arange(x.shape[-1]) < rot.rotary_dim
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size)[..., turned].all(), float(err.max())
    assert (err[..., ~turned] == 0).all()


CASES = [(1, 1, 1, 64, 64), (33, 4, 2, 64, 32), (300, 3, 1, 128, 16), (31, 8, 8, 128, 128), (1000, 5, 1, 128, 112),
         (65, 64, 8, 64, 48), (7, 2, 2, 128, 64), (4099, 8, 2, 128, 128)]


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hkv,d,part", CASES, ids=str)
def test_against_the_definition(fcp, T, hq, hkv, d, part, interleaved, backward):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k = (torch.randn(h, T, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv))
    positions = torch.randint(-(1 << 31), (1 << 31) - 1, (T,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    positions[:T // 2] = positions[:T // 2] % 5000
    rot = fcp.Rotary(part, base=500000.0, interleaved=interleaved, scaling=dict(kind="yarn", factor=4.0, original=4096))
    call = fcp.rotary_backward if backward else fcp.rotary_apply
    oq, ok = call(rot, q, k, positions)
    check(rot, q, oq, positions, backward)
    check(rot, k, ok, positions, backward)
    # in place, and each alone, is the same
    q2, k2 = q.clone(), k.clone()
    assert call(rot, q2, k2, positions, q2, k2)[0] is q2
    assert torch.equal(q2, oq) and torch.equal(k2, ok)
    assert torch.equal(call(rot, q, None, positions)[0], oq) and torch.equal(call(rot, None, k, positions)[1], ok)


def test_values_that_are_not_finite_stay_in_their_pair(fcp):
    q = torch.ones(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 1, 5], q[1, 2, 40], q[0, 0, 63] = float("inf"), float("nan"), float("-inf")
    positions = torch.tensor([0, 3, 9], dtype=torch.int32).cuda()
    for interleaved in (False, True):
        rot = fcp.Rotary(48, interleaved=interleaved)
        out = fcp.rotary_apply(rot, q, None, positions)[0].isfinite().cpu()
        pair = lambda c: {c, c ^ 1} if interleaved else {c, (c + 24) % 48}  # noqa: E731
        want = torch.ones(2, 3, 64, dtype=torch.bool)
        want[0, 1, sorted(pair(5))] = want[1, 2, sorted(pair(40))] = False
        want[0, 0, 63] = False
        assert torch.equal(out, want)


def test_far_positions_keep_the_differences(fcp):
    """q . k depends on the difference of the positions alone: at 2^30 as at 0."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(1, 1, 128, generator=g, device="cuda", dtype=torch.bfloat16).expand(1, 64, 128).contiguous() for _ in "qk")
    rot = fcp.Rotary(128)
    near = torch.arange(64, dtype=torch.int32, device="cuda")
    a, b = fcp.rotary_apply(rot, q, k, near)
    c, e = fcp.rotary_apply(rot, q, k, near + (1 << 30))
    s, t = (x[0].double() @ y[0].double().T for x, y in ((a, b), (c, e)))
    # each turned channel is off by 2^-8 of itself and 2^-21 of its pair: so is each product, twice
    size = a[0].double().abs() @ b[0].double().abs().T + c[0].double().abs() @ e[0].double().abs().T
    assert ((s - t).abs() <= 2.0 ** -6.9 * size).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("part,interleaved", [(128, False), (64, True), (48, False), (16, False), (112, True), (96, False)])
@pytest.mark.parametrize("new,lens,hq,hkv,d", [([1, 1, 1, 1], [40, 7, 300, 17], 8, 2, 128), ([3, 0, 17, 1], [3, 40, 33, 64], 4, 2, 64),
                                               ([5, 2, 64], [4, 1, 64], 3, 3, 128), ([129, 1, 200], [300, 1, 200], 5, 5, 128)])
def test_write_is_turn_then_write(fcp, cache, part, interleaved, new, lens, hq, hkv, d):
    """Bit for bit what rotary_apply and cache_write do; rows of no sequence and rows before position 0 (the third
    batch has some) are left as they were."""
    part = min(part, d)
    b = Batch(new, lens, hq=hq, hkv=hkv, d=d, page=32, pad=3, cache=cache, seed=part)
    util = U4 if cache == "e2m1" else U
    t, z = util.make(b), util.make(b)
    handle, batch = util.handles(fcp, b, t)
    other, batch2 = util.handles(fcp, b, z)
    rot = fcp.Rotary(part, interleaved=interleaved, scaling=dict(kind="linear", factor=2.0))
    positions = torch.full((b.total,), -1, dtype=torch.int32)
    row = 0
    for n, length in zip(new, lens):
        positions[row:row + n] = torch.arange(length - n, length, dtype=torch.int32)
        row += n
    on = (positions >= 0).cuda()
    q, k = fcp.rotary_apply(rot, t["q"], t["k"], positions.cuda())
    fcp.cache_write(other, batch2, k, z["v"])
    out = torch.full_like(t["q"], 7.0)
    kept = t["k"].clone(), t["v"].clone(), t["q"].clone()
    assert fcp.rotary_write(handle, batch, rot, t["q"], t["k"], t["v"], out) is out
    handle.check_device_error()
    other.check_device_error()
    assert torch.equal(out[:, on], q[:, on]) and (out[:, ~on] == 7.0).all()
    for x, y in zip(kept, (t["k"], t["v"], t["q"])):
        assert torch.equal(x, y)
    for x in ("k_pages", "v_pages", "k_scales", "v_scales"):
        if t[x] is not None:
            assert torch.equal(t[x].view(torch.uint8), z[x].view(torch.uint8)), x
    # in place, and without q
    fcp.rotary_write(handle, batch, rot, t["q"], t["k"], t["v"], t["q"])
    assert torch.equal(t["q"][:, on], q[:, on]) and torch.equal(t["q"][:, ~on], kept[2][:, ~on])
    assert fcp.rotary_write(handle, batch, rot, None, t["k"], t["v"]) is None
    assert torch.equal(t["k_pages"].view(torch.uint8), z["k_pages"].view(torch.uint8))


def test_broken_batches(fcp):
    """A bad page leaves its k and v out (q is turned all the same); a bad length leaves out the sequence."""
    for what, code in (("page", 0x51), ("len", 0x50)):
        b = Batch([2, 3, 2], [40, 30, 33], hq=4, hkv=2, cache="e2m1")
        t = U4.make(b)
        if what == "page":
            t["table"][1, 1] = 1 << 30  # positions 16 and on: all three of its rows
        else:
            t["lens"][1] = -3
        before = t["k_pages"].view(torch.uint8).clone()
        cache, batch = U4.handles(fcp, b, t)
        rot = fcp.Rotary(64)
        out = torch.full_like(t["q"], 7.0)
        fcp.rotary_write(cache, batch, rot, t["q"], t["k"], t["v"], out)
        with pytest.raises(fcp.FcpError, match=hex(code)):
            cache.check_device_error()
        assert (out[:, 2:5] == 7.0).all().item() == (what == "len")
        after = t["k_pages"].view(torch.uint8)
        rows = (after != before).any(-1).any(1).sum().item()
        assert rows == 4  # of the other two sequences
        assert not (out[:, :2] == 7.0).all() and not (out[:, 5:] == 7.0).all()


def test_streams_and_capture(fcp):
    """On a stream that nothing was made on, and in a graph that replays with new positions and lengths."""
    b = Batch([5, 1, 40], [50, 7, 300], hq=4, hkv=2, d=128, page=32)
    t = U4.make(b)
    cache, batch = U4.handles(fcp, b, t)
    rot = fcp.Rotary(128)
    positions = torch.arange(b.total, dtype=torch.int32, device="cuda")
    q, k, w = torch.empty_like(t["q"]), torch.empty_like(t["k"]), torch.empty_like(t["q"])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        fcp.rotary_apply(rot, t["q"], t["k"], positions, q, k)
        fcp.rotary_write(cache, batch, rot, t["q"], t["k"], t["v"], w)
    for far in (0, 100000):
        positions.copy_(torch.arange(b.total, device="cuda") * 3 + far)
        t["lens"].copy_(torch.tensor([x - (far > 0) for x in b.lens]))
        graph.replay()
        check(rot, t["q"], q, positions)
        check(rot, t["k"], k, positions)
        rows = np.concatenate([np.arange(l - n, l) - (far > 0) for n, l in zip(b.new, b.lens)])
        check(rot, t["q"], w, torch.from_numpy(rows))
    with torch.cuda.stream(side):
        again = fcp.rotary_apply(rot, t["q"], t["k"], positions, stream=side)
    handle = fcp.rotary_apply(rot, t["q"], t["k"], positions, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for x in (again, handle):
        assert torch.equal(x[0], q) and torch.equal(x[1], k)
    cache.check_device_error()


def test_offsets_past_32_bits(fcp):
    """Rows whose elements lie past 2^31: the last head's last rows."""
    T, hq, d = 1 << 19, 33, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(hq, T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    rot = fcp.Rotary(d)
    out, _ = fcp.rotary_apply(rot, q, None, positions)
    check(rot, q[-1:, -500:], out[-1:, -500:], positions[-500:])
    check(rot, q[:1, :500], out[:1, :500], positions[:500])


@pytest.mark.parametrize("pipeline", [None, 2])
def test_the_attention_with_rotary(fcp, pipeline):
    """FcpAttention(rotary=...): the attention over turned q and k, and its gradients turned back; dq and dk are
    bf16 before they are turned, so twice the rounding."""
    seqlens, hq, hkv, d = [300, 77, 1024], 4, 2, 64
    T = sum(seqlens)
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, do = (torch.randn(h, T, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv, hkv, hq))
    rot = fcp.Rotary(d)
    att = fcp.FcpAttention(seqlens, 512, True, 4, hq, hkv, d, rotary=rot, pipeline=pipeline)
    plain = fcp.FcpAttention(seqlens, 512, True, 4, hq, hkv, d, pipeline=pipeline)
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in seqlens]).cuda()
    assert torch.equal(att.positions, positions)
    keep = q.clone(), k.clone()
    o, lse = att.forward(q, k, v)
    tq, tk = fcp.rotary_apply(rot, q, k, positions)
    o2, lse2 = plain.forward(tq, tk, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dq, dk, dv = att.backward(q, k, v, o, lse, do)
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    gq, gk, gv = plain.backward(tq, tk, v, o, lse, do)
    # the sums of dq are added in an order that varies: a unit of bf16 more here and there
    for got, raw in ((dq, gq), (dk, gk)):
        want, size = R.turn(raw.double().cpu().numpy(), positions.cpu().numpy(), rot.radians, 1.0, False, backward=True)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -7 + 2.0 ** -20) * size + 1e-4).all()
    # on another stream, by its handle, the same
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, lse3 = torch.zeros_like(o), torch.zeros_like(lse)
    att.forward(q, k, v, o3, lse3, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o3, o) and torch.equal(lse3, lse)
    if pipeline is None:
        att.replan([77, 300, 1024])
        assert att.positions[76].item() == 76 and att.positions[77].item() == 0
    with pytest.raises(ValueError, match="rotary_dim"):
        fcp.FcpAttention(seqlens, 512, True, 4, hq, hkv, d, rotary=fcp.Rotary(128))


def test_refusals(fcp):
    rot = fcp.Rotary(64)
    q = torch.zeros(2, 5, 64, dtype=torch.bfloat16, device="cuda")
    positions = torch.zeros(5, dtype=torch.int32, device="cuda")
    for bad in (lambda: fcp.rotary_apply(rot, None, None, positions), lambda: fcp.rotary_apply(rot, q, None, positions[:4]),
                lambda: fcp.rotary_apply(rot, q, q[:, :4].contiguous(), positions),
                lambda: fcp.rotary_apply(rot, q, None, positions, k_out=q), lambda: fcp.rotary_apply(rot, q[0], None, positions),
                lambda: fcp.rotary_apply(rot, q.transpose(0, 1), None, positions),
                lambda: fcp.rotary_apply(rot, q, None, positions.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fcp.rotary_apply(rot, q.float(), None, positions)
    with pytest.raises(TypeError):
        fcp.rotary_apply(rot, q, None, positions.long())
    with pytest.raises(fcp.FcpError):
        fcp.rotary_apply(rot, q[..., :32].contiguous(), None, positions)
    empty = torch.zeros(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    assert fcp.rotary_apply(rot, empty, empty, positions[:0])[0].shape == (2, 0, 64)
