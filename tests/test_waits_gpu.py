"""Bounded waits of the scan's and the decode step's kernels: none is given up
in ordinary calls, and a caller can ask."""
import os
import subprocess
import sys

import pytest
import torch

import ssm_depthwise_causal_gb300 as ccc
from tests import mixer_reference as ref

pytestmark = pytest.mark.gpu


class Calls:
    """A cut batch through the scan, forward and backward, and a decode step of many requests."""

    def __init__(self, seed=81, seqs=64):
        self.c = ref.make([2300, 0, 40, 1400], 4, 64, 2, 128, seed=seed, initial=True, d_final=True)
        self.g = self.c.to("cuda")
        self.par = dict(D=self.g.D, dt_bias=self.g.dt_bias, dt_softplus=True)
        gen = torch.Generator().manual_seed(seed)
        self.conv, self.pool = torch.randn(seqs, 768, 3, generator=gen).bfloat16().cuda(), torch.randn(seqs, 4, 64, 128, generator=gen).cuda()
        self.weight, self.token = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((768, 4), (seqs, 768)))
        self.dt, self.slots = torch.randn(seqs, 4, generator=gen).cuda(), torch.randperm(seqs, generator=gen).to(torch.int32).cuda()

    def forward(self, **kw):
        g = self.g
        final = torch.empty_like(g.initial)
        return ccc.selective_scan_fn(g.x, g.dt, g.A, g.B, g.C, None, g.cu, initial_state=g.initial, final_state=final, **self.par, **kw), final

    def backward(self, **kw):
        g = self.g
        return tuple(ccc.selective_scan_bwd(g.x, g.dt, g.A, g.B, g.C, g.dy, g.cu, initial_state=g.initial, d_final_state=g.d_final, want_d_initial=True,
                                            **self.par, **kw))

    def step(self, conv=None, pool=None):
        conv, pool = self.conv.clone() if conv is None else conv, self.pool.clone() if pool is None else pool
        return ccc.ssm_update(self.token, self.weight, conv, self.dt, self.g.A, pool, self.slots, n_groups=2, **self.par), conv, pool

    def all(self):
        return [*self.forward(), *self.backward(), *self.step()]


def test_none_is_given_up():
    calls = Calls()
    before = ccc.given_up_waits()
    words = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    calls.all()
    calls.forward(workspace=words)
    calls.backward(workspace=words)
    assert ccc.given_up_waits() == before and int(words[:4].view(torch.int32)) == 0
    status = torch.full((3,), 77, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert ccc.ccc_wait_status(status, stream=side) is status
    side.synchronize()
    assert status.tolist() == [before, 77, 77]


def test_first_call_inside_a_capture():
    """A process whose first scan and step are captured: the replay gives what the calls give."""
    code = """
import torch
import ssm_depthwise_causal_gb300 as ccc
from tests.test_waits_gpu import Calls
calls, graph = Calls(), torch.cuda.CUDAGraph()
conv, pool = calls.conv.clone(), calls.pool.clone()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    made = [*calls.forward(), *calls.backward(), calls.step(conv, pool)[0]]
graph.replay()
torch.cuda.synchronize()
want = [*calls.forward(), *calls.backward(), calls.step()[0]]
assert all(torch.equal(a, b) for a, b in zip(made, want))
assert ccc.given_up_waits() == 0
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.fixture
def no_patience():
    """Waits are given up at the first look that finds them unfinished."""
    ccc.set_wait_limit(0)
    yield
    ccc.set_wait_limit()


@pytest.mark.parametrize("name", ["forward", "backward"])
def test_scan_waits_run_out(name, no_patience):
    """The kernels end, soon, and say so; the device, and the next call with patience, are as before."""
    calls = Calls(seed=82)
    ccc.set_wait_limit()
    run = getattr(calls, name)
    want = [t.clone() for t in run()]
    words = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    before = ccc.given_up_waits()
    for _ in range(3):
        ccc.set_wait_limit(0)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        run(workspace=words)
        end.record()
        ccc.set_wait_limit()
        count = ccc.given_up_waits()
        assert count > before and int(words[:4].view(torch.int32)) == 1
        # a drain that waits for what was never started takes a second
        assert begin.elapsed_time(end) < 100.0
        before = count
        assert all(torch.equal(a, b) for a, b in zip(want, run()))
        assert ccc.given_up_waits() == before


def test_step_waits_run_out(no_patience):
    """A warp that has no state stores none: every row of the pool has its old or its right value.  Many
    heads a group, whose states come in pieces one behind another, so that some are looked for before they are there."""
    ccc.set_wait_limit()
    H, P, G, N, seqs = 48, 64, 4, 128, 200
    gen = torch.Generator(device="cuda").manual_seed(83)
    C = H * P + 2 * G * N

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    pool, conv = normal(seqs, H, P, N), normal(seqs, C, 3).bfloat16()
    token, weight, dt, A = normal(seqs, C).bfloat16(), normal(C, 4).bfloat16(), normal(seqs, H), -normal(H).abs()
    slots = torch.randperm(seqs, generator=gen, device="cuda").to(torch.int32)

    def step():
        a, b = conv.clone(), pool.clone()
        return ccc.ssm_update(token, weight, a, dt, A, b, slots, n_groups=G, dt_softplus=True), a, b
    y, conv_after, after = step()
    before = ccc.given_up_waits()
    for _ in range(3):
        ccc.set_wait_limit(0)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        got = step()[2]
        end.record()
        ccc.set_wait_limit()
        count = ccc.given_up_waits()
        assert count > before
        # a drain that waits for what was never started takes a second
        assert begin.elapsed_time(end) < 100.0
        before = count
        left, right = (got == pool).all(-1), (got == after).all(-1)
        assert bool((left | right).all()) and not bool(right.all())
        assert all(torch.equal(a, b) for a, b in zip((y, conv_after, after), step())) and ccc.given_up_waits() == before
