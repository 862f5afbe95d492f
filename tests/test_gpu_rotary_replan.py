"""FcpAttention(rotary=...) with another batch in the same buffers (replan): its rows' new positions in every call that
is enqueued behind it and in none before, and no wait for the stream."""
import numpy as np
import pytest
import torch

from oracle import rotary as R

pytestmark = pytest.mark.gpu


def positions_of(seqlens):
    return torch.cat([torch.arange(n, dtype=torch.int32) for n in seqlens]).cuda()


def rows(seqlens, hq, hkv, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(h, sum(seqlens), d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (hq, hkv, hkv, hq)]


BATCHES = [[1401], [77, 1024, 300], [1, 1, 1399], [300, 77, 1024], [700, 0, 701]]  # the first needs most partial rows


@pytest.mark.parametrize("stream", ["current", "stream", "handle"])
def test_forward_and_backward_follow_the_new_batch(fcp, stream):
    """Against the attention of a plain plan over freshly turned q and k, with work still queued in front; dq and dk are
    bf16 before they are turned back, so twice the rounding."""
    hq, hkv, d = 4, 2, 64
    rot = fcp.Rotary(d)
    att = fcp.FcpAttention(BATCHES[0], 512, True, 4, hq, hkv, d, rotary=rot)
    side = torch.cuda.current_stream() if stream == "current" else torch.cuda.Stream()
    arg = {"current": None, "stream": side, "handle": side.cuda_stream}[stream]
    outs, wants = [], []
    sets = [rows(b, hq, hkv, d, i) for i, b in enumerate(BATCHES)]
    for seqlens, (q, k, v, do) in zip(BATCHES, sets):
        plain = fcp.FcpAttention(seqlens, 512, True, 4, hq, hkv, d)
        positions = positions_of(seqlens)
        tq, tk = fcp.rotary_apply(rot, q, k, positions)
        o, lse = plain.forward(tq, tk, v)
        wants.append((o, lse, positions, plain.backward(tq, tk, v, o, lse, do)))
    buffers = [[torch.full_like(x, 7.0) for x in (q, q[..., 0].float(), q, k, v)] for q, k, v, _ in sets]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e8))
    for i, (seqlens, (q, k, v, do), (o, lse, dq, dk, dv)) in enumerate(zip(BATCHES, sets, buffers)):
        if i:
            att.replan(seqlens, stream=arg)
        att.forward(q, k, v, o, lse, stream=arg)
        att.backward(q, k, v, o, lse, do, dq, dk, dv, stream=arg)
    torch.cuda.synchronize()
    att.check_device_error()
    for (o, lse, dq, dk, dv), (wo, wl, positions, (gq, gk, gv)) in zip(buffers, wants):
        assert torch.equal(o, wo) and torch.equal(lse, wl)
        # the sums of dq are added in an order that varies: a unit of bf16 more here and there
        assert ((dv.float() - gv.float()).abs() <= 2.0 ** -7 * gv.float().abs() + 1e-4).all()
        for got, raw in ((dq, gq), (dk, gk)):
            want, size = R.turn(raw.double().cpu().numpy(), positions.cpu().numpy(), rot.radians, 1.0, False, backward=True)
            err = np.abs(got.double().cpu().numpy() - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -7 + 2.0 ** -20) * size + 1e-4).all()
    assert torch.equal(att.positions, wants[-1][2])


def test_the_host_does_not_wait(fcp):
    """replan returns while the stream still works on what came before it, with rotary positions as without. (The
    plan's image is below 64 KB, up to which the copy of ordinary host memory does not wait either.)"""
    hq, hkv, d, seqlens = 2, 1, 64, [1000, 600, 400]
    for rotary in (None, fcp.Rotary(d)):
        att = fcp.FcpAttention(seqlens, 512, True, 4, hq, hkv, d, rotary=rotary, backward=False)
        assert att.plan.device_bytes() < 60000
        att.replan(seqlens[::-1])
        torch.cuda.synchronize()
        torch.cuda._sleep(int(1e9))  # half a second
        done = torch.cuda.Event()
        done.record()
        att.replan(seqlens)
        waited = done.query()
        torch.cuda.synchronize()
        assert not waited, "with rotary" if rotary else "without"
        if rotary:
            assert torch.equal(att.positions, positions_of(seqlens))
