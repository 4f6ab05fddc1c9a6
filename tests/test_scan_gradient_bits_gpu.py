"""dx's term from behind a chunk keeps the state gradient's bits.

With dy = 0 and one value in each token's B, dx_s = dt_s 2^(a_end - a_s) G_pn B_sn
is one product, G the gradient of the final state in 32 bits.  It is rounded to
BF16 once: by at most 2^-8 of the value.  Everything before that (G as BF16
parts of 16 bits or more, 2^-16; decays and steps in 32 bits, a running sum of
128 of them, under 2^-14 as in test_mixer_gpu) stays under 2^-13 of it.  G
rounded to one BF16 would be off by 2^-8 more."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,H,P,G,N", [([100], 4, 64, 2, 128), ([128, 7], 2, 64, 1, 64), ([90, 128], 2, 128, 1, 128), ([60], 2, 24, 1, 40), ([64], 1, 16, 1, 256)])
def test_state_term_of_dx(lengths, H, P, G, N):
    c = ref.make(lengths, H, P, G, N, seed=91, d_final=True)
    gen = torch.Generator().manual_seed(92)
    rows = sum(lengths)
    c.dy.zero_()
    c.d_final.copy_(torch.randn(c.d_final.shape, generator=gen))
    c.B.copy_(torch.zeros(rows, G, N).scatter_(2, torch.randint(0, N, (rows, G, 1), generator=gen), (1 + torch.rand(rows, G, 1, generator=gen))).bfloat16())
    want = ref.scan(c, grad=True)["dx"]
    g = c.to("cuda")
    got = ccc.selective_scan_bwd(g.x, g.dt, g.A, g.B, g.C, g.dy, g.cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=c.softplus, d_final_state=g.d_final).dx
    off = (got.double().cpu() - want).abs() - (2 ** -8 + 2 ** -13) * want.abs() - 1e-30
    assert bool((off <= 0).all()), f"{int((off > 0).sum())} of {off.numel()} values"
