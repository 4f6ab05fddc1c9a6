"""What the mixer's binding checks before the library is called (no GPU
needed): tensors on the CPU pass the checks of shape, type and layout and are
refused for their device last, so every other refusal comes from the check
that is meant."""
import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


# Two sequences of five tokens, four heads of 64 in two groups of 128 states.
def batch():
    return dict(x=b16(2, 5, 4, 64), dt=torch.zeros(2, 5, 4), A=torch.zeros(4), B=b16(2, 5, 2, 128), C=b16(2, 5, 2, 128))


@pytest.mark.parametrize("name", ["out", "dx", "dB", "dC"])
def test_written_in_place_or_refused(name):
    """A [B, T, ...] tensor to write that has no flat view is refused (a flat copy would be written in its place); one that
    has a view, also as a slice of wider rows, is taken."""
    args = batch()
    heads, per = (2, 128) if name in ("dB", "dC") else (4, 64)
    if name == "out":
        def call(t):
            ccc.selective_scan_fn(**args, out=t)
    else:
        def call(t):
            ccc.selective_scan_bwd(**args, dy=b16(2, 5, 4, 64), **{name: t})
    with pytest.raises(ValueError, match=f"{name} .*view"):
        call(b16(2, 9, heads, per)[:, :5])
    with pytest.raises(ValueError, match=f"{name} .*view"):
        call(b16(5, 2, heads, per).transpose(0, 1))
    for good in (b16(2, 5, heads, per), b16(2, 5, heads * per + 16)[..., :heads * per].unflatten(2, (heads, per))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call(good)
