"""Accepted counts past the positions that a decode step's pools hold: both
pools start from the same token, the last one that both have.  [B, k, C] calls
against the packed call, bit for bit.

Tolerances as in test_mixer_gpu.test_step: y is rounded to BF16 once (2^-8),
states are FP32 (2^-14 of the magnitude without cancellation)."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

H, P, G, N, SEQS = 4, 64, 2, 128, 3


def inputs(W, L, held, draft, seed):
    g = torch.Generator().manual_seed(seed)
    C, rows = H * P + 2 * G * N, sum(draft)

    def normal(*shape):
        return torch.randn(shape, generator=g)
    return dict(xbc=normal(rows, C).bfloat16(), w=torch.rand(C, W, generator=g) - 0.5, b=normal(C).bfloat16(), conv=normal(5, C, L).bfloat16(), dt=normal(rows, H),
                A=-(1 + 15 * torch.rand(H, generator=g)), D=normal(H), dt_bias=normal(H) - 3, pool=normal(5, held, H, P, N),
                cu=torch.tensor([0, *torch.tensor(draft).cumsum(0)], dtype=torch.int32), cache=torch.tensor([3, 0, 4], dtype=torch.int32))


def step(t, accepted, out=None, **kw):
    conv, pool = t["conv"].cuda(), t["pool"].cuda()
    d = {k: v.cuda() for k, v in t.items()}
    y = ccc.ssm_update(kw.pop("xbc", d["xbc"]), d["w"], conv, kw.pop("dt", d["dt"]), d["A"], pool, d["cache"], n_groups=G,
                       num_accepted=accepted.cuda(), bias=d["b"], D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True, out=out, **kw)
    return y, conv, pool


@pytest.mark.parametrize("W,L,held,draft", [(4, 8, 2, [1, 2, 1]), (4, 4, 5, [1, 1, 2]), (2, 6, 3, [3, 1, 2]), (3, 2, 1, [1, 1, 1])])
def test_accepted_past_the_positions(W, L, held, draft):
    t = inputs(W, L, held, draft, seed=71)
    most = min(held, L - W + 2)
    for accepted in ([most + 1, 1, 1000], [most, -3, most + 2], [0, most + 1, 1]):
        given = torch.tensor(accepted, dtype=torch.int32)
        args = (t["xbc"], t["w"], t["b"], True, t["conv"], t["dt"], t["A"], t["D"], t["dt_bias"], True, t["pool"], t["cu"], t["cache"],
                given.clamp(1, most), H, P, G, N)
        y, conv, pool = ref.step(*args)
        ym, _, pm = ref.step(*args, mag=True)
        got = step(t, given, cu_seqlens=t["cu"].cuda())
        assert bool(((got[0].double().cpu() - y).abs() <= 2 ** -8 * ym + 1e-5).all())
        assert torch.equal(got[1].cpu().view(torch.int16), conv.view(torch.int16))
        assert bool(((got[2].double().cpu() - pool).abs() <= 2 ** -14 * pm + 1e-6).all())


@pytest.mark.parametrize("k,held,L", [(1, 1, 3), (2, 2, 4), (5, 5, 7)])
def test_batch_form(k, held, L):
    """[B, k, C] with dt [B, k, H] and out [B, k, H, P]."""
    t = inputs(4, L, held, [k] * SEQS, seed=72)
    accepted = torch.tensor([1, held, (held + 1) // 2], dtype=torch.int32)
    want = step(t, accepted, cu_seqlens=t["cu"].cuda())
    three = dict(xbc=t["xbc"].cuda().unflatten(0, (SEQS, k)), dt=t["dt"].cuda().unflatten(0, (SEQS, k)))
    out = torch.empty(SEQS, k, H, P, dtype=torch.bfloat16, device="cuda")
    for given in (None, out):
        got = step(t, accepted, out=given, **three)
        assert got[0].shape == out.shape and (given is None or got[0] is out)
        assert torch.equal(got[0].flatten(0, 1), want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
