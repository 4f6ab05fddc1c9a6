"""The example's mixer with head counts that are not a multiple of eight: the
projection's rows hold z, x, B, C and dt side by side, and their stride has to
be a multiple of eight all the same."""
import pytest

from examples import ssm_mixer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,P,G,N", [(3, 64, 1, 64), (6, 32, 2, 128), (2, 128, 2, 16), (1, 8, 1, 8)])
def test_any_number_of_heads(H, P, G, N):
    mixer = ssm_mixer.Mixer(64, H, P, G, N).cuda()
    losses = ssm_mixer.train(mixer, [60, 1, 90], 4)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    # as in test_mixer_gpu.test_example: the roundings of the convolution's three results and of y, and as much again
    assert ssm_mixer.serve(mixer, [70, 1], 2) < 8 * 2 ** -8
