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


def packed(**kw):
    """The same as three packed sequences of ten rows."""
    a = dict(x=b16(10, 4, 64), dt=torch.zeros(10, 4), A=torch.zeros(4), B=b16(10, 2, 128), C=b16(10, 2, 128), cu_seqlens=ints(4))
    a.update(kw)
    return a


def ints(n, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def step(**kw):
    a = dict(xBC=b16(3, 768), weight=torch.zeros(768, 4), conv_state=b16(8, 768, 5), dt=torch.zeros(3, 4), A=torch.zeros(4), ssm_state=torch.zeros(8, 2, 4, 64, 128),
             cache_indices=ints(3), n_groups=2, cu_seqlens=ints(4), num_accepted=ints(3), bias=b16(768))
    a.update(kw)
    return a


NOT_INT32 = [ints(3, torch.int64), ints(6)[::2], ints(2)]  # another type, a stride, too short


@pytest.mark.parametrize("bad", [ints(4, torch.int64), ints(8)[::2], ints(0)])
def test_cu_seqlens_type_and_layout(bad):
    for call in (lambda: ccc.selective_scan_fn(**packed(cu_seqlens=bad)), lambda: ccc.selective_scan_bwd(**packed(cu_seqlens=bad), dy=b16(10, 4, 64)),
                 lambda: ccc.ssm_update(**step(cu_seqlens=bad))):
        with pytest.raises(ValueError, match="cu_seqlens must"):
            call()


@pytest.mark.parametrize("bad", NOT_INT32)
def test_slots_and_counts_type_and_length(bad):
    for call in (lambda: ccc.selective_scan_fn(**packed(), cache_indices=bad), lambda: ccc.selective_scan_bwd(**packed(), dy=b16(10, 4, 64), cache_indices=bad),
                 lambda: ccc.ssm_update(**step(cache_indices=bad))):
        with pytest.raises(ValueError, match="cache_indices must"):
            call()
    with pytest.raises(ValueError, match="num_accepted must"):
        ccc.ssm_update(**step(num_accepted=bad))


@pytest.mark.parametrize("bad", [ints(3), torch.zeros(3), ints(2, torch.bool), ints(6, torch.bool)[::2]])
def test_flags_type_and_length(bad):
    with pytest.raises(ValueError, match="has_initial_state must"):
        ccc.selective_scan_fn(**packed(), has_initial_state=bad)


def test_metadata_that_fits_is_taken():
    """Flags as bool or bytes, and arrays longer than the batch, as a padded batch has them."""
    for flags in (ints(3, torch.bool), ints(5, torch.uint8)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            ccc.selective_scan_fn(**packed(), cache_indices=ints(5), has_initial_state=flags)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ccc.ssm_update(**step(cache_indices=ints(5), num_accepted=ints(5)))


@pytest.mark.parametrize("bad", [dict(weight=torch.zeros(4, 768).t()), dict(weight=torch.zeros(768, 8)[:, ::2]), dict(bias=b16(700)), dict(bias=b16(1)),
                                 dict(bias=b16(1536)[::2])])
def test_convolution_parameters_of_a_step(bad):
    """The taps are read as [C, W] and the bias as [C], whatever their strides and sizes say."""
    with pytest.raises(ValueError, match="must be contiguous"):
        ccc.ssm_update(**step(**bad))


def test_backward_options_are_checked():
    """ccc_scan_bwd_ex knows one bit; what it does not know is refused before anything else, and the array form agrees."""
    import struct

    from ssm_depthwise_causal_gb300 import _build, _lib
    from tests.test_host import E_NULL, E_SHAPE
    from tests.test_mixer_host import BWD
    _build.build()
    for bits, want in ((1, E_SHAPE), (4, E_SHAPE), (3, E_SHAPE), (_lib.OPT_CARRY_EMPTY, E_NULL), (0, E_NULL)):
        args = [*dict(BWD, dA=0).values()]
        args.insert(-1, bits)
        assert _lib.lib().ccc_scan_bwd_ex(*args) == want
        assert _lib.lib().ccc_scan_bwd_ex_v(struct.pack("42q", *args)) == want


def test_several_tokens_need_positions():
    """A pool without positions would keep the state after a request's first token alone."""
    flat = torch.zeros(8, 4, 64, 128)
    for call in (lambda: ccc.ssm_update(**step(ssm_state=flat, xBC=b16(6, 768), dt=torch.zeros(6, 4))),
                 lambda: ccc.ssm_update(**step(ssm_state=flat, xBC=b16(3, 2, 768), dt=torch.zeros(3, 2, 4), cu_seqlens=None))):
        with pytest.raises(ValueError, match="room for the state after one token"):
            call()
    for good in (step(ssm_state=flat), step(ssm_state=flat, xBC=b16(2, 768), dt=torch.zeros(2, 4)), step(ssm_state=flat, cu_seqlens=None),
                 step(ssm_state=flat[:, None], xBC=b16(6, 768), dt=torch.zeros(6, 4)), step(xBC=b16(3, 2, 768), dt=torch.zeros(3, 2, 4), cu_seqlens=None)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            ccc.ssm_update(**good)


def test_wait_limit_and_status_refuse():
    from ssm_depthwise_causal_gb300 import _build, _lib
    from tests.test_host import E_ALIGN, E_NULL, E_SHAPE
    _build.build()
    assert _lib.lib().ccc_set_wait_limit(-1) == E_SHAPE and _lib.lib().ccc_set_wait_limit(0) == 0
    ccc.set_wait_limit()  # the default again
    assert _lib.lib().ccc_wait_status(None, None) == E_NULL and _lib.lib().ccc_wait_status(4098, None) == E_ALIGN
    with pytest.raises(ccc.CCCError):
        ccc.set_wait_limit(-5)
    for bad in (ints(0), ints(1, torch.int64)):
        with pytest.raises(ValueError, match="status must"):
            ccc.ccc_wait_status(bad)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ccc.ccc_wait_status(ints(1))
