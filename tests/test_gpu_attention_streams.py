"""What an FcpAttention allocates, on other streams than the one that it was made on: with rotary positions and without."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SEQLENS, HQ, HKV, D = [300, 77, 1024], 4, 2, 64


def rows(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(h, sum(SEQLENS), D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (HQ, HKV, HKV, HQ)]


def make(fcp, turned):
    return fcp.FcpAttention(SEQLENS, 512, True, 4, HQ, HKV, D, rotary=fcp.Rotary(D) if turned else None)


def near(got, ref):
    # the sums of dq are added in an order that varies: a unit of bf16 more here and there, 2^-7 of itself and of the
    # gradients' size of about 1
    return ((got.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs() + 2.0 ** -7).all()


@pytest.mark.parametrize("turned", [False, True], ids=["plain", "rotary"])
@pytest.mark.parametrize("kind", ["stream", "current", "handle"])
def test_dropped_while_another_stream_works(fcp, kind, turned):
    """An attention used on another stream and dropped at once: its plan, its workspaces, its positions and turned q
    and k are not handed out while the work is under way."""
    q, k, v, do = rows(0)
    first = make(fcp, turned)
    want = first.forward(q, k, v)
    grads = first.backward(q, k, v, *want, do)
    att = make(fcp, turned)
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(1e8))
    if kind == "current":
        with torch.cuda.stream(side):
            att.forward(q, k, v, o, lse)
            att.backward(q, k, v, o, lse, do, dq, dk, dv)
    else:
        arg = side.cuda_stream if kind == "handle" else side
        att.forward(q, k, v, o, lse, stream=arg)
        att.backward(q, k, v, o, lse, do, dq, dk, dv, stream=arg)
    mine = [att.d_plan, att.part_o, att.part_lse, att.workspace] + ([att.positions, *att._turned] if turned else [])
    sizes, places = [x.numel() * x.element_size() for x in mine], {x.data_ptr() for x in mine}
    del att, mine
    over = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    if side.query():  # an object used on a stream of unknown life waits for the device when it is dropped
        assert kind == "handle"
    else:
        taken = places & {x.data_ptr() for x in over}
        torch.cuda.synchronize()
        assert not taken
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert all(near(*x) for x in zip((dq, dk, dv), grads))


@pytest.mark.parametrize("turned", [False, True], ids=["plain", "rotary"])
def test_made_on_a_busy_stream(fcp, turned):
    """An attention is whole when its constructor returns: another stream may use it at once, though the one that was
    current then is still at work."""
    q, k, v, do = rows(1)
    want = make(fcp, turned).forward(q, k, v)
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(int(1e8))
    att = make(fcp, turned)
    done = torch.cuda.current_stream().query()  # read here: nothing is launched on a plan that is not there yet
    assert done
    att.forward(q, k, v, o, lse, stream=side)
    torch.cuda.synchronize()
    att.check_device_error()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
