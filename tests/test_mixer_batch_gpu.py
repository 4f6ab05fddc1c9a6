"""[B, T, ...] calls of the scan that write into the caller's tensors: the
packed call's bits, in place."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


def test_given_outputs_are_written():
    """out, dx, dB and dC as slices of wider [B, T, ...] rows."""
    c = ref.make([60, 60, 60], 4, 64, 2, 128, seed=41)
    g = c.to("cuda")
    par = dict(D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    y = ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, g.cu, **par)
    d = ccc.selective_scan_bwd(g.x, g.dt, g.A, g.B, g.C, g.dy, g.cu, **par)
    x, dt, B, C, dy = (t.unflatten(0, (3, 60)) for t in (g.x, g.dt, g.B, g.C, g.dy))
    wide = torch.full((3, 60, 4 * 64 + 2 * 256 + 8), 7.0, dtype=torch.bfloat16, device="cuda")

    def part(first, heads, size):
        return wide[..., first:first + heads * size].unflatten(2, (heads, size))
    out = part(0, 4, 64)
    assert ccc.selective_scan_fn(x, dt, g.A, B, C, out=out, **par) is out
    assert torch.equal(out.flatten(0, 1), y) and bool((wide[..., 256:] == 7.0).all())
    dx, dB, dC = part(0, 4, 64), part(256, 2, 128), part(512, 2, 128)
    got = ccc.selective_scan_bwd(x, dt, g.A, B, C, dy, dx=dx, dB=dB, dC=dC, **par)
    assert got.dx is dx and got.dB is dB and got.dC is dC
    for a, b in ((dx, d.dx), (dB, d.dB), (dC, d.dC), (got.ddt, d.ddt)):
        assert torch.equal(a.flatten(0, 1), b)
    assert bool((wide[..., 768:] == 7.0).all())
