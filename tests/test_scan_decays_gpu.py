"""States of heads that forget within a few tokens (steps of some units, A down
to -16).  What a token gives to the state at its chunk's end is decayed by the
sum of the steps behind it; taken as a difference of two running sums of
thousands, that exponent would be off by 2^-14 or more.

Bounds as in test_mixer_gpu: states and state gradients within 2^-14 of their
magnitude without cancellation.  A term of 2^-24 of the largest or more has an
exponent below 24, whose sum over at most 128 tokens (seven additions deep) is off
by 24 * 9 * 2^-24 < 2^-16; terms below that do not count."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,H,P,G,N", [([128, 100, 31, 700], 8, 64, 2, 128), ([2000, 333], 4, 64, 1, 64), ([64, 200, 33], 8, 24, 4, 136), ([90, 500], 4, 72, 2, 32)])
def test_states_of_heads_that_forget(lengths, H, P, G, N):
    c = ref.make(lengths, H, P, G, N, seed=95, initial=True, d_final=True, bias=False)
    c.dt = c.dt + 4
    c.A = -torch.linspace(0.25, 16, H)
    want, mag = ref.scan(c, grad=True), ref.scan(c, grad=True, mag=True)
    g = c.to("cuda")
    final = torch.empty_like(g.initial)
    ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, g.cu, D=g.D, dt_softplus=True, initial_state=g.initial, final_state=final)
    d = ccc.selective_scan_bwd(g.x, g.dt, g.A, g.B, g.C, g.dy, g.cu, D=g.D, dt_softplus=True, initial_state=g.initial, d_final_state=g.d_final,
                               want_d_initial=True)
    for got, name in ((final, "final"), (d.d_initial, "d_initial")):
        off = (got.double().cpu() - want[name]).abs() / (mag[name] + 1e-30)
        assert float(off.max()) <= 2 ** -14, (name, float(off.max()) * 2 ** 14)
