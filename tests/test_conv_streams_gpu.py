"""``stream=`` of the convolution's allocating helpers: what they make belongs
to the stream that they are given (the mixer's: test_mixer_streams_gpu.py)."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests.test_mixer_streams_gpu import LATE

pytestmark = pytest.mark.gpu


def calls():
    g = torch.Generator().manual_seed(53)
    x, dy = (torch.randn(3, 200, 256, generator=g).bfloat16().cuda() for _ in range(2))
    w, b = torch.randn(256, 4, generator=g).cuda(), torch.randn(256, generator=g).cuda()
    slots, pool = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"), torch.randn(3, 256, 3, generator=g).bfloat16().cuda()
    hist = torch.randn(3, 3, 256, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 200, 400, 600], dtype=torch.int32, device="cuda")

    def update(**kw):
        p, out = pool.clone(), torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
        return lambda: (ccc.causal_conv1d_update(x[:, 0], w, p, slots, bias=b, out=out, **kw), p)
    return {
        "forward": lambda **kw: lambda: (ccc.causal_conv1d_fn(x, w, bias=b, **kw),),
        "backward": lambda **kw: lambda: ccc.causal_conv1d_bwd(x, w, dy, bias=b, **kw)[:3],
        "update": update,
        "recompute": lambda **kw: lambda: (ccc.recompute_fwd(x.flatten(0, 1), w, hist, cu, bias=b, **kw),),
        "check": lambda **kw: lambda: (ccc.ccc_check(600, cu, slots, 3, **kw)[:1],),
    }


NAMES = ["forward", "backward", "update", "recompute", "check"]


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_is_busy(name):
    made = calls()[name]
    want = [t.clone() for t in made()()]
    side = torch.cuda.Stream()
    run = made(stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_given_stream_is_late(name):
    made = calls()[name]
    want = [t.clone() for t in made()()]
    side = torch.cuda.Stream()
    run = made(stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    got = run()
    trash = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 19, 1 << 20, 3 << 20) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del trash
