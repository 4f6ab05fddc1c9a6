"""The gradient of an empty sequence's initial state.  Its final state is its
initial one, so selective_scan hands d_final on as it is; a padded (-1)
request's final state is zeros, and so is that gradient.

Tolerances: where nothing is computed the bits have to be equal.  Against
central differences of the 64-bit loss (step 1e-5, whose own error is 1e-9 of
the third derivative's size and 1e-11 / 1e-5 of rounding): the gradient keeps
2^-14 of its magnitude without cancellation in every value, so its product
with a direction v is off by at most 2^-14 sum |mag v|.
"""
import dataclasses

import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu

CASES = [
    dict(lengths=[5, 0, 130], H=2, P=64, G=1, N=128),                                # one CTA a pair, tensor cores
    dict(lengths=[0, 2000, 0, 0, 1500, 0], H=2, P=64, G=1, N=128),                   # cut sequences
    dict(lengths=[7, 0, 40], H=2, P=24, G=2, N=40),
    dict(lengths=[7, 0, 40, 0], H=2, P=16, G=1, N=256, padded=(1,)),                 # FP32 kernels, a padded request without rows
    dict(lengths=[30, 0, 200, 0], H=4, P=64, G=2, N=64, padded=(1, 2)),
]


def gradients(c):
    """Of the initial state, by autograd through y and the final state."""
    g = c.to("cuda")
    first = g.initial.clone().requires_grad_()
    y, final = ccc.selective_scan(g.x, g.dt, g.A, g.B, g.C, g.cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=c.softplus, initial_state=first,
                                  cache_indices=g.cache)
    torch.autograd.backward([y, final], [g.dy, g.d_final])
    return first.grad


def is_padded(c, n):
    return c.cache is not None and int(c.cache[n]) == -1


@pytest.mark.parametrize("kw", CASES)
def test_empty_sequences_hand_the_gradient_on(kw):
    c = ref.make(seed=31, initial=True, d_final=True, **kw)
    got = gradients(c).cpu()
    for n, length in enumerate(c.lengths):
        if is_padded(c, n):
            assert bool((got[n] == 0).all()), n
        elif length == 0:
            assert torch.equal(got[n], c.d_final[n]), n


@pytest.mark.parametrize("kw", [CASES[0], CASES[2], CASES[4]])
def test_initial_gradient_against_differences(kw):
    c = ref.make(seed=32, initial=True, d_final=True, **kw)
    got, mag = gradients(c).double().cpu(), ref.scan(c, grad=True, mag=True)["d_initial"]
    gen = torch.Generator().manual_seed(33)

    def loss(initial):
        r = ref.scan(dataclasses.replace(c, initial=initial))
        return float((r["y"] * c.dy.double()).sum() + (r["final"] * c.d_final.double()).sum())
    first, eps = c.initial.double(), 1e-5
    for n in range(len(c.lengths)):  # a direction inside each sequence's state
        v = torch.zeros_like(first)
        v[n] = torch.randn(first[n].shape, generator=gen, dtype=torch.float64)
        diff = (loss(first + eps * v) - loss(first - eps * v)) / (2 * eps)
        assert abs(float((got * v).sum()) - diff) <= 2 ** -14 * float((mag * v).abs().sum()) + 1e-5 * (1 + abs(diff)), n


def test_without_rows():
    """No token at all: every gradient is zero but the initial states', which are the final ones'."""
    e = torch.empty
    x, dt, B = e(0, 2, 64, dtype=torch.bfloat16, device="cuda"), e(0, 2, device="cuda"), e(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    A, cu = (-torch.ones(2, device="cuda")).requires_grad_(), torch.zeros(4, dtype=torch.int32, device="cuda")
    cache = torch.tensor([0, -1, 1], dtype=torch.int32, device="cuda")
    first, d_final = torch.randn(3, 2, 64, 128, device="cuda", requires_grad=True), torch.randn(3, 2, 64, 128, device="cuda")
    y, final = ccc.selective_scan(x, dt, A, B, B, cu, initial_state=first, cache_indices=cache)
    torch.autograd.backward([y, final], [torch.zeros_like(y), d_final])
    assert torch.equal(first.grad[[0, 2]], d_final[[0, 2]]) and bool((first.grad[1] == 0).all()) and bool((A.grad == 0).all())


def test_a_chain_of_fragments_with_an_empty_one():
    """Three fragments, the middle one without rows, against the whole sequence: the state's gradient crosses it."""
    c = ref.make([150], 2, 64, 1, 128, seed=34, initial=True)
    want, mag = ref.scan(c, grad=True), ref.scan(c, grad=True, mag=True)
    g = c.to("cuda")
    first, cuts = g.initial.clone().requires_grad_(), [0, 70, 70, 150]
    state, ys = first, []
    for a, b in zip(cuts, cuts[1:]):
        y, state = ccc.selective_scan(g.x[a:b], g.dt[a:b], g.A, g.B[a:b], g.C[a:b], D=g.D, dt_bias=g.dt_bias, dt_softplus=True, initial_state=state)
        ys.append(y)
    torch.cat(ys).backward(g.dy)
    off = (first.grad.double().cpu() - want["d_initial"]).abs() - 2 ** -14 * mag["d_initial"] - 1e-30
    assert bool((off <= 0).all())


def with_empty_runs(c, runs):
    """The same batch with `runs[i]` empty sequences before sequence i, and the last count behind all."""
    lengths = [0] * runs[0]
    for n, more in zip(c.lengths, runs[1:]):
        lengths += [n] + [0] * more
    cu = torch.zeros(len(lengths) + 1, dtype=torch.int64)
    cu[1:] = torch.tensor(lengths).cumsum(0)
    return cu.to(torch.int32).cuda()


@pytest.mark.parametrize("runs", [[3, 0, 40, 1, 2], [300, 1000, 33, 2000, 700]])
def test_runs_of_empty_sequences(runs):
    """They change nothing, forward or backward, in either direction of the walks."""
    c = ref.make([20, 1800, 128, 700], 2, 64, 1, 128, seed=35)
    g, want, mag = c.to("cuda"), ref.scan(c, grad=True), ref.scan(c, grad=True, mag=True)
    cu = with_empty_runs(c, runs)
    par = dict(D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    y = ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, cu, **par)
    d = ccc.selective_scan_bwd(g.x, g.dt, g.A, g.B, g.C, g.dy, cu, **par)
    for got, name, eps in ((y, "y", 2 ** -7), (d.dx, "dx", 2 ** -6), (d.dB, "dB", 2 ** -6), (d.dC, "dC", 2 ** -6)):  # as in test_mixer_gpu
        off = (got.double().cpu() - want[name]).abs() - eps * mag[name] - 1e-30
        assert bool((off <= 0).all()), name
    assert float((d.dA.double().cpu() - want["dA"]).norm()) <= 2 ** -13 * float(mag["dA"].norm())


def test_a_million_empty_sequences():
    """A walk steps over a run of them at once: one by one would take as long as its other warps wait at most."""
    c = ref.make([40, 1500, 30], 2, 64, 1, 128, seed=36)
    g, want, mag = c.to("cuda"), ref.scan(c)["y"], ref.scan(c, mag=True)["y"]
    cu = with_empty_runs(c, [1_000_000, 0, 1_000_000, 5])
    y = ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, cu, D=g.D, dt_bias=g.dt_bias, dt_softplus=True)
    end.record()
    torch.cuda.synchronize()
    assert bool(((y.double().cpu() - want).abs() <= 2 ** -7 * mag + 1e-30).all())
    assert begin.elapsed_time(end) < 50.0  # ms; a step of one at a time is some 0.5 us, two million of them a second
