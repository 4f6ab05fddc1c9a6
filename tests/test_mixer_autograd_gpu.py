"""What the mixer's autograd wrappers refuse: a second derivative, whose terms
would be lost without a word (the backwards' results are constants to
autograd)."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


def penalty(out, leaf):
    """Adds a function of the gradient to the loss, and differentiates again."""
    grad, = torch.autograd.grad(out.float().square().sum(), leaf, create_graph=True)
    (grad.float().square().sum() + leaf.float().sum()).backward()


def test_second_derivative_is_refused():
    g = ref.make([40, 9], 2, 64, 1, 128, seed=61).to("cuda")
    x = g.x.clone().requires_grad_()
    y, _ = ccc.selective_scan(x, g.dt, g.A, g.B, g.C, g.cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        penalty(y, x)
    y, z, w = (torch.randn(*s, device="cuda").bfloat16().requires_grad_() for s in ((7, 64), (7, 64), (64,)))
    with pytest.raises(RuntimeError, match="once_differentiable"):
        penalty(ccc.gated_rms_norm(y, z, w), y)


def test_gradients_with_a_graph_kept():
    """create_graph alone changes nothing."""
    g = ref.make([40, 9], 2, 64, 1, 128, seed=62).to("cuda")
    grads = []
    for keep in (False, True):
        x = g.x.clone().requires_grad_()
        y, _ = ccc.selective_scan(x, g.dt, g.A, g.B, g.C, g.cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
        grads.append(torch.autograd.grad(y, x, g.dy, create_graph=keep)[0].detach())
    assert torch.equal(*grads)
