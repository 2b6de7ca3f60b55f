"""Two recurrent layers as a model runs them, on random weights: a KDA layer and a selective scan layer.

KDA layer:   x -> one projection -> short convolution of q, k and v -> unit q and k rows with the position
             rotation -> the mixer -> output projection
scan layer:  x -> one projection -> short convolution -> selective scan with its gate -> output projection

Packed prompts of several lengths leave their states in pools of slots; single tokens go on from there. At the end every
token's output is compared with one prompt over prompt and tokens together, and one training step is taken.

    python examples/layers.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_56_gb300 as kda  # noqa: E402

WIDTH = 4  # taps of the short convolutions
GATE_BOUND = 5.0


def _weight(gen, out_features, in_features, dtype, device):
    return (torch.randn(out_features, in_features, generator=gen, device=device) / in_features ** 0.5).to(dtype)


class KDALayer:
    """q, k, v, the gate logits and beta come out of one projection; each slot of the pools is one sequence's state."""

    def __init__(self, model, heads, head, slots, positions, dtype, device, gen):
        self.heads, self.head, self.inner = heads, head, heads * head
        self.proj = _weight(gen, 4 * self.inner + heads, model, dtype, device)
        self.out = _weight(gen, model, self.inner, dtype, device)
        self.conv = torch.randn(3 * self.inner, WIDTH, generator=gen, device=device).div(WIDTH ** 0.5).to(dtype)
        freq = 10000.0 ** (-torch.arange(0, head // 2, 2, device=device, dtype=torch.float64) / (head // 2))
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq  # half of each head turns
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.conv_states = torch.zeros(slots, WIDTH - 1, 3 * self.inner, dtype=dtype, device=device)
        self.states = torch.zeros(slots, heads, head, head, device=device)

    def _split(self, p):
        lead = p.shape[:-1]
        g = p[..., 3 * self.inner:4 * self.inner].reshape(*lead, self.heads, self.head)
        return p[..., :3 * self.inner], g.contiguous(), torch.sigmoid(p[..., 4 * self.inner:]).contiguous()

    def _qkv(self, y, positions):
        q, k, v = (t.unflatten(-1, (self.heads, self.head)) for t in y.split(self.inner, -1))  # slices of one tensor
        q, k = kda.qk_norm_rotary(q, k, self.cos, self.sin, positions, norm="l2")
        return q, k, v.contiguous()

    def prompt(self, x, cu_seqlens, positions, slots):
        qkv, g, beta = self._split(x @ self.proj.t())
        first = torch.full_like(slots, -1)  # new sequences start from nothing
        y, _ = kda.conv_prefill(qkv, self.conv, cu_seqlens=cu_seqlens, initial_state=self.conv_states, final_state=self.conv_states,
                                initial_state_indices=first, final_state_indices=slots)
        q, k, v = self._qkv(y, positions)
        o, _ = kda.prefill(q, k, v, g, beta, cu_seqlens=cu_seqlens, initial_state=self.states, final_state=self.states,
                           initial_state_indices=first, final_state_indices=slots, gate_bound=GATE_BOUND)
        return o.flatten(-2) @ self.out.t()

    def token(self, x, positions, slots):
        qkv, g, beta = self._split(x @ self.proj.t())
        y = kda.conv_decode_step(qkv, self.conv, self.conv_states, state_indices=slots)
        q, k, v = self._qkv(y, positions)
        o = kda.decode_step(q, k, v, g, beta, self.states, state_indices=slots, gate_bound=GATE_BOUND)
        return o.flatten(-2) @ self.out.t()


class ScanLayer:
    """x and its gate come out of one projection, the time steps, B and C out of a second one behind the convolution."""

    def __init__(self, model, channels, n, slots, dtype, device, gen):
        self.channels, self.n = channels, n
        self.proj, self.out = _weight(gen, 2 * channels, model, dtype, device), _weight(gen, model, channels, dtype, device)
        self.second = _weight(gen, channels + 2 * n, channels, dtype, device)
        self.conv = torch.randn(channels, WIDTH, generator=gen, device=device).div(WIDTH ** 0.5).to(dtype)
        self.conv_bias = torch.zeros(channels, dtype=dtype, device=device)
        self.A = -torch.arange(1, n + 1, device=device).float().repeat(channels, 1)
        self.D, self.dt_bias = torch.ones(channels, device=device), torch.full((channels,), -4.0, device=device)
        self.conv_states = torch.zeros(slots, WIDTH - 1, channels, dtype=dtype, device=device)
        self.states = torch.zeros(slots, channels, n, device=device)

    def _second(self, y):
        p = y @ self.second.t()
        B, C = (t.unsqueeze(-2) for t in p[..., self.channels:].split(self.n, -1))  # one group
        return p[..., :self.channels], B, C

    def prompt(self, x, cu_seqlens, slots):
        p = x @ self.proj.t()
        first = torch.full_like(slots, -1)
        y, _ = kda.conv_prefill(p[..., :self.channels], self.conv, self.conv_bias, cu_seqlens=cu_seqlens, initial_state=self.conv_states,
                                final_state=self.conv_states, initial_state_indices=first, final_state_indices=slots)
        dt, B, C = self._second(y)
        o, _ = kda.scan_prefill(y, dt, self.A, B, C, D=self.D, z=p[..., self.channels:], dt_bias=self.dt_bias, cu_seqlens=cu_seqlens,
                                initial_state=self.states, final_state=self.states, initial_state_indices=first,
                                final_state_indices=slots)
        return o @ self.out.t()

    def token(self, x, slots):
        p = x @ self.proj.t()
        y = kda.conv_decode_step(p[..., :self.channels], self.conv, self.conv_states, self.conv_bias, state_indices=slots)
        dt, B, C = self._second(y)
        o = kda.scan_decode_step(y, dt, self.A, B, C, self.states, D=self.D, z=p[..., self.channels:], dt_bias=self.dt_bias,
                                 state_indices=slots)
        return o @ self.out.t()

    def train_step(self, x, target, rate):
        """One step of plain gradient descent on mean((layer(x) - target)^2): the new loss and the old one."""

        def forward():
            p = x @ self.proj.t()
            y, _ = kda.conv_prefill(p[..., :self.channels], self.conv, self.conv_bias, output_final_state=False)
            dt, B, C = self._second(y)
            o, _ = kda.scan_prefill(y, dt, self.A, B, C, D=self.D, z=p[..., self.channels:], dt_bias=self.dt_bias,
                                    output_final_state=False)
            return p, y, dt, B, C, o, o @ self.out.t() - target

        p, y, dt, B, C, o, off = forward()
        loss = off.float().square().mean()
        d = (off * (2.0 / off.numel())).to(x.dtype)
        d_out = d.flatten(0, -2).t().float() @ o.flatten(0, -2).float()
        g = kda.scan_backward(y, dt, self.A, B, C, d @ self.out, D=self.D, z=p[..., self.channels:], dt_bias=self.dt_bias,
                              want_d_initial_state=False)
        d_p2 = torch.cat([g["ddt"], g["dB"].squeeze(-2), g["dC"].squeeze(-2)], -1)
        d_second = d_p2.flatten(0, -2).t() @ y.flatten(0, -2).float()
        dy = g["dx"] + d_p2 @ self.second.float()
        c = kda.conv_backward(p[..., :self.channels], self.conv, dy.to(x.dtype), self.conv_bias, want_d_initial_state=False)
        d_p = torch.cat([c["dx"], g["dz"]], -1)
        d_proj = d_p.flatten(0, -2).t() @ x.flatten(0, -2).float()
        for weight, grad in ((self.proj, d_proj), (self.second, d_second), (self.out, d_out), (self.conv, c["dweight"]),
                             (self.conv_bias, c["dbias"]), (self.A, g["dA"]), (self.D, g["dD"]), (self.dt_bias, g["ddt_bias"])):
            weight -= (rate * grad).to(weight.dtype)
        return float(forward()[-1].float().square().mean()), float(loss)


def main(model=256, heads=4, head=64, channels=512, n=16, lengths=(70, 1, 133, 40), tokens=5, device="cuda:0"):
    """Prints and returns the largest differences (KDA, scan) between tokens and prompts, and (loss after, loss before)."""
    gen = torch.Generator(device=device)
    gen.manual_seed(0)
    dtype, count = torch.bfloat16, len(lengths)
    layers = KDALayer(model, heads, head, 2 * count, 4096, dtype, device, gen), ScanLayer(model, channels, n, 2 * count, dtype, device, gen)
    x = [torch.randn(t + tokens, model, generator=gen, device=device).to(dtype) for t in lengths]

    def packed(parts):
        cu = torch.tensor([0] + [len(p) for p in parts], device=device).cumsum(0).to(torch.int32)
        pos = torch.cat([torch.arange(len(p), device=device) for p in parts]).to(torch.int32)[None]
        return torch.cat(parts)[None], cu, pos

    slots = torch.arange(count, dtype=torch.int32, device=device)
    off = []
    for kind, layer in zip(("kda", "scan"), layers):
        more = (lambda pos: (pos,)) if kind == "kda" else (lambda pos: ())
        rows, cu, pos = packed([p[:t] for p, t in zip(x, lengths)])
        layer.prompt(rows, cu, *more(pos), slots)
        steps = []
        for i in range(tokens):
            at = torch.tensor([t + i for t in lengths], dtype=torch.int32, device=device)
            steps.append(layer.token(torch.stack([p[t + i] for p, t in zip(x, lengths)]), *more(at), slots))
        rows, cu, pos = packed(x)  # prompt and tokens as one prompt, in other slots
        whole = layer.prompt(rows, cu, *more(pos), slots + count)[0].float()
        want = torch.stack([whole[int(cu[s + 1]) - tokens:int(cu[s + 1])] for s in range(count)], 1)
        got = torch.stack(steps).float()
        off.append(float((got - want).norm() / want.norm()))
        print(f"{kind} layer: {tokens} tokens of {count} sequences against one prompt: {off[-1]:.2e} relative")
    rows = torch.randn(2, 128, model, generator=gen, device=device).to(dtype)
    losses = layers[1].train_step(rows, torch.randn(2, 128, model, generator=gen, device=device).to(dtype), 2.0)
    print(f"scan layer, one training step: loss {losses[1]:.4f} -> {losses[0]:.4f}")
    kda.check_status(device)
    return (*off, losses)


if __name__ == "__main__":
    main()
