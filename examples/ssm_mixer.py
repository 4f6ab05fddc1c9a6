"""An SSM mixer from the package's operators: convolution, selective scan and
gated norm for packed training and prompts, and one launch per decode step
before the norm.

    python examples/ssm_mixer.py

trains a small mixer on packed sequences for a few steps, reads a ragged batch
of prompts into the two state pools, continues every request token by token,
and compares the continuation with the scan of the whole sequence.
"""
from __future__ import annotations

import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ssm_depthwise_causal_gb300 as ccc  # noqa: E402


class Mixer(nn.Module):
    """hidden [rows, width] -> [rows, width]; H heads of P channels share B and C in G groups of N states."""

    def __init__(self, width, H, P, G, N, seed=0):
        super().__init__()
        self.sizes = H, P, G, N
        self.inner, self.channels = H * P, H * P + 2 * G * N
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return nn.Parameter((torch.randn(shape, generator=g) * shape[-1] ** -0.5).bfloat16())
        # z | x B C | dt, and unused columns up to a multiple of eight: z and x are read with the projection's row stride
        self.parts = [self.inner, self.channels, H, -H % 8]
        self.w_in = weight(sum(self.parts), width)
        self.w_out = weight(width, self.inner)
        self.conv_w = nn.Parameter(torch.rand(self.channels, 4, generator=g) - 0.5)
        self.conv_b = nn.Parameter(torch.zeros(self.channels))
        self.A_log = nn.Parameter(torch.log(1 + 15 * torch.rand(H, generator=g)))
        self.D = nn.Parameter(torch.ones(H))
        self.dt_bias = nn.Parameter(torch.full((H,), -3.0))
        self.norm_w = nn.Parameter(torch.ones(self.inner))

    def project(self, hidden):
        return (hidden @ self.w_in.t()).split(self.parts, dim=1)[:3]

    def heads(self, xbc):
        H, P, G, N = self.sizes
        x, B, C = xbc.split([H * P, G * N, G * N], dim=1)
        return x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N))

    def finish(self, y, z):
        return ccc.gated_rms_norm(y.flatten(1), z, self.norm_w, group_size=self.inner // self.sizes[2]) @ self.w_out.t()

    def forward(self, hidden, cu_seqlens):
        """Differentiable, over packed sequences that start from nothing."""
        z, xbc, dt = self.project(hidden)
        x, B, C = self.heads(ccc.causal_conv1d(xbc, self.conv_w, self.conv_b, cu_seqlens))
        y, _ = ccc.selective_scan(x, dt, -torch.exp(self.A_log), B, C, cu_seqlens, D=self.D, dt_bias=self.dt_bias, dt_softplus=True)
        return self.finish(y, z)

    def pools(self, slots):
        """Convolution histories and scan states of `slots` requests, updated in place by the calls below."""
        H, P, _, N = self.sizes
        dev = self.D.device
        return torch.zeros(slots, self.channels, 3, dtype=torch.bfloat16, device=dev), torch.zeros(slots, H, P, N, device=dev)

    @torch.no_grad()
    def prompt(self, hidden, cu_seqlens, pools, slots, continues):
        """Packed prompts (or pieces of them: `continues`) of the requests in `slots`."""
        conv, states = pools
        z, xbc, dt = self.project(hidden)
        x, B, C = self.heads(ccc.causal_conv1d_fn(xbc, self.conv_w, conv, cu_seqlens, slots, continues, bias=self.conv_b))
        y = ccc.selective_scan_fn(x, dt, -torch.exp(self.A_log), B, C, states, cu_seqlens, slots, continues, D=self.D, dt_bias=self.dt_bias,
                                  dt_softplus=True)
        return self.finish(y, z)

    @torch.no_grad()
    def step(self, hidden, pools, slots):
        """One token of each request in `slots`: convolution and scan in one launch."""
        conv, states = pools
        z, xbc, dt = self.project(hidden)
        y = ccc.ssm_update(xbc, self.conv_w, conv, dt, -torch.exp(self.A_log), states, slots, n_groups=self.sizes[2], bias=self.conv_b,
                           D=self.D, dt_bias=self.dt_bias, dt_softplus=True)
        return self.finish(y, z)


def offsets(lengths, device):
    return torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32, device=device)


def train(mixer, lengths, steps, lr=0.1):
    """Gradient steps toward a fixed random target; the losses."""
    dev = mixer.D.device
    g = torch.Generator().manual_seed(1)
    hidden, target = (torch.randn(sum(lengths), mixer.w_in.shape[1], generator=g).bfloat16().to(dev) for _ in range(2))
    cu, losses = offsets(lengths, dev), []
    for _ in range(steps):
        loss = (mixer(hidden, cu).float() - target.float()).square().mean()
        losses.append(float(loss.detach()))
        grads = torch.autograd.grad(loss, list(mixer.parameters()))
        with torch.no_grad():
            for p, d in zip(mixer.parameters(), grads):
                p -= (lr * d.float()).to(p.dtype)
    return losses


def serve(mixer, lengths, more):
    """Prompts, the first one in two pieces, then `more` tokens a request; the largest relative error of a step against the whole."""
    dev = mixer.D.device
    width, n = mixer.w_in.shape[1], len(lengths)
    g = torch.Generator().manual_seed(2)
    text = [torch.randn(k + more, width, generator=g).bfloat16().to(dev) for k in lengths]
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=dev)
    pools, new = mixer.pools(n + 1), torch.zeros(n, dtype=torch.bool, device=dev)
    cut = lengths[0] // 2
    mixer.prompt(text[0][:cut], offsets([cut], dev), pools, slots[:1], new[:1])
    rest = [lengths[0] - cut, *lengths[1:]]
    continues = new.clone()
    continues[0] = True
    mixer.prompt(torch.cat([t[k - r:k] for t, k, r in zip(text, lengths, rest)]), offsets(rest, dev), pools, slots, continues)
    made = [mixer.step(torch.stack([t[k + j] for t, k in zip(text, lengths)]), pools, slots) for j in range(more)]
    with torch.no_grad():
        whole = mixer(torch.cat(text), offsets([k + more for k in lengths], dev)).split([k + more for k in lengths])
    want = torch.stack([w[-more:] for w in whole], dim=1).float()
    return float(((torch.stack(made).float() - want).norm(dim=-1) / want.norm(dim=-1)).max())


def main(device="cuda"):
    mixer = Mixer(256, 8, 64, 2, 128).to(device)
    losses = train(mixer, [200, 1, 333, 64], 5)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    off = serve(mixer, [70, 1, 300], 4)
    print(f"continued prompts against the whole sequences: {off:.4f}")
    return losses, off


if __name__ == "__main__":
    main()
