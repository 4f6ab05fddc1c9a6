"""``stream=``: the call's own tensors (workspace, offsets, flat copies,
results) belong to the stream that it is given, so neither a busy current
stream nor what is allocated there behind the call reaches them."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

LATE = 100_000_000  # cycles, some 50 ms


def calls():
    """name -> what takes further arguments and gives the call, whose result is all that it writes."""
    c = ref.make([300, 300], 4, 64, 2, 128, seed=51)
    g = c.to("cuda")
    par = dict(D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    x, dt, B, C, dy = (t.unflatten(0, (2, 300)) for t in (g.x, g.dt, g.B, g.C, g.dy))
    gen = torch.Generator().manual_seed(52)
    conv, pool = torch.randn(2, 768, 4, generator=gen).bfloat16().cuda(), torch.randn(2, 2, 4, 64, 128, generator=gen).cuda()
    weight, token = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((768, 4), (2, 2, 768)))
    dt1, slots = torch.randn(2, 2, 4, generator=gen).cuda(), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    y, z, w = (torch.randn(*s, generator=gen).bfloat16().cuda() for s in ((2, 300, 256), (2, 300, 256), (256,)))

    def step(**kw):
        a, b = conv.clone(), pool.clone()
        torch.cuda.synchronize()
        return lambda: (ccc.ssm_update(token, weight, a, dt1, g.A, b, slots, n_groups=2, **par, **kw), a, b)
    return {
        "scan": lambda **kw: lambda: (ccc.selective_scan_fn(x, dt, g.A, B, C, **par, **kw),),
        "scan backward": lambda **kw: lambda: tuple(t for t in ccc.selective_scan_bwd(x, dt, g.A, B, C, dy, **par, **kw) if t is not None),
        "step": step,
        "norm": lambda **kw: lambda: (ccc.gated_rms_norm_fn(y, z, w, **kw),),
        "norm backward": lambda **kw: lambda: ccc.gated_rms_norm_bwd(y, z, w, y, **kw),
    }


NAMES = ["scan", "scan backward", "step", "norm", "norm backward"]


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_is_busy(name):
    """The call neither waits for the current stream nor reads what that one would have made late."""
    made = calls()[name]
    want = [t.clone() for t in made()()]
    side = torch.cuda.Stream()
    run = made(stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    busy = torch.cuda.Event()
    busy.record()
    got = run()
    side.synchronize()
    assert not busy.query(), "the call waited for the current stream"
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_given_stream_is_late(name, as_handle):
    """While the given stream has yet to run the call, the current one allocates and fills whatever it is given."""
    made = calls()[name]
    want = [t.clone() for t in made()()]
    side = torch.cuda.Stream()
    run = made(stream=side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    got = run()
    trash = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 19, 1 << 20, 3 << 20, 1 << 25) for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del trash
