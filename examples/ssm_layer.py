"""One state-space layer, prompts and tokens, from the library's operators.

The layer's in-projection gives a row z | x B C | dt per token; x, B and C go through the short
causal convolution, then through the selective scan, gated by z, and the out-projection brings
the result back. Its weights are held in 4 bits. A serving loop keeps, for every sequence, a slot
of convolution state and a slot of scan state:

* ``prompt``: packed prompts of any lengths, into their slots (w4_matmul, causal_conv1d_packed,
  selective_scan, w4_matmul);
* ``token``: one token per row, in place on the slots (w4_matmul, selective_state_update, w4_matmul).

Run it: three prompts are taken in, continued token by token, and compared with the same
sequences taken in as whole prompts.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import depthwise_causal_conv1d_gb300 as ccu  # noqa: E402


class Layer:
    """Random weights of a layer of ``width`` channels: ``heads`` of ``head`` inner channels, ``states`` states a
    channel, B and C shared by the heads of each of ``groups``; ``group`` inputs share a scale of the 4-bit weights."""

    def __init__(self, width, heads, head, states, groups, taps=4, group=128, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.heads, self.head, self.states, self.groups = heads, head, states, groups
        self.inner, self.bc = heads * head, groups * states
        self.mixed = self.inner + 2 * self.bc                       # channels of the convolution
        rows = self.inner + self.mixed + heads
        rows += -rows % 8                                           # whole 16-byte vectors a row

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

        self.w_in = ccu.w4_quantize(normal(rows, width, scale=width ** -0.5), group)
        self.w_out = ccu.w4_quantize(normal(width, self.inner, scale=self.inner ** -0.5), group)
        self.conv_weight, self.conv_bias = normal(self.mixed, taps, scale=0.5), normal(self.mixed, scale=0.1)
        step = torch.exp(torch.rand(heads, generator=g, device=device) * math.log(100) + math.log(1e-3))
        self.dt_bias = step + torch.log(-torch.expm1(-step))        # softplus(dt_bias) in 0.001..0.1
        self.A = -1 - 15 * torch.rand(heads, generator=g, device=device)
        self.D = torch.ones(heads, device=device)

    def slots(self, count):
        """Zeroed states of `count` sequences: the convolution's (channel-last) and the scan's."""
        taps = self.conv_weight.shape[1]
        conv = torch.zeros(count, taps - 1, self.mixed, dtype=torch.bfloat16, device=self.A.device).permute(0, 2, 1)
        return conv, torch.zeros(count, self.heads, self.head, self.states, device=self.A.device)

    def _split(self, u):
        """z, the convolution's channels, and dt: slices of the in-projection's rows."""
        row = ccu.w4_matmul(u, *self.w_in)
        z, mixed, dt = row[:, :self.inner], row[:, self.inner:self.inner + self.mixed], row[:, self.inner + self.mixed:]
        return z.unflatten(1, (self.heads, self.head)), mixed, dt[:, :self.heads]

    def prompt(self, u, cu_seqlens, slots, conv_state, state, has_initial=None):
        """``u`` [T, width]: packed prompts; returns [T, width] and leaves the states in the slots."""
        z, mixed, dt = self._split(u)
        mixed = ccu.causal_conv1d_packed(mixed, self.conv_weight, self.conv_bias, "silu", cu_seqlens=cu_seqlens,
                                         conv_state=conv_state, conv_state_indices=slots, has_initial_state=has_initial)
        x, B, C = mixed.split([self.inner, self.bc, self.bc], 1)
        y = ccu.selective_scan(x.unflatten(1, (self.heads, self.head)), dt, self.A, B.unflatten(1, (self.groups, self.states)),
                               C.unflatten(1, (self.groups, self.states)), D=self.D, z=z, dt_bias=self.dt_bias,
                               cu_seqlens=cu_seqlens, ssm_state=state, state_indices=slots, has_initial_state=has_initial)
        return ccu.w4_matmul(y.flatten(1), *self.w_out)

    def token(self, u, slots, conv_state, state):
        """``u`` [N, width]: one token for each slot of ``slots`` (-1: a padding row); returns [N, width]."""
        z, mixed, dt = self._split(u)
        y = ccu.selective_state_update(mixed, dt, self.A, state, conv_state, self.conv_weight, self.conv_bias, "silu",
                                       D=self.D, z=z, dt_bias=self.dt_bias, groups=self.groups, state_indices=slots)
        return ccu.w4_matmul(y.flatten(1), *self.w_out)


def main(width=1024, heads=32, head=64, states=128, groups=1, lens=(200, 1, 77), tokens=8, group=128, device="cuda"):
    """The largest difference of the two ways through the layer, relative to the outputs' size."""
    layer = Layer(width, heads, head, states, groups, group=group, device=device)
    i32 = dict(dtype=torch.int32, device=device)
    g = torch.Generator(device=device)
    g.manual_seed(1)
    seqs = [torch.randn(n + tokens, width, generator=g, device=device).to(torch.bfloat16) for n in lens]
    slots = torch.tensor([4, 0, 2], **i32)[:len(lens)]

    def offsets(ns):
        return torch.tensor([0, *torch.tensor(ns).cumsum(0).tolist()], **i32)

    conv, state = layer.slots(6)
    whole = layer.prompt(torch.cat(seqs), offsets([n + tokens for n in lens]), slots, conv, state)
    last = torch.stack([s[-tokens:] for s in whole.split([n + tokens for n in lens])], 1)      # [tokens, sequences, width]

    conv2, state2 = layer.slots(6)
    layer.prompt(torch.cat([s[:n] for s, n in zip(seqs, lens)]), offsets(list(lens)), slots, conv2, state2)
    steps = [layer.token(torch.stack([s[n + t] for s, n in zip(seqs, lens)]), slots, conv2, state2) for t in range(tokens)]
    off = (torch.stack(steps).float() - last.float()).abs().max() / last.float().abs().max()
    off_state = (state - state2).abs().max() / state.abs().max()
    return float(off), float(off_state)


if __name__ == "__main__":
    print("outputs of the two ways differ by %.2g of their size, states by %.2g" % main())
