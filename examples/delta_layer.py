"""A layer with the delta rule of one decay per value head as a model runs it, on random weights.

residual sum and RMS norm -> one projection -> short convolution of q, k and v -> unit q and k rows -> the mixer, value heads sharing key
heads -> RMS norm per head with its gate -> output projection

Packed prompts of several lengths leave their states in pools of slots; single tokens go on from there. At the end every token's
output is compared with one prompt over prompt and tokens together, and the gradients of one training step are taken.

    python examples/delta_layer.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_56_gb300 as kda  # noqa: E402

WIDTH = 4  # taps of the short convolution
EPS = 1e-6


class DeltaLayer:
    """q, k, v, the gate and the logits of decay and beta come out of one projection; each slot of the pools is one sequence's state."""

    def __init__(self, model, k_heads, v_heads, head, slots, dtype, device, gen):
        self.k_heads, self.v_heads, self.head = k_heads, v_heads, head
        self.keys, self.values = k_heads * head, v_heads * head
        self.mixed = 2 * self.keys + self.values  # channels of the convolution

        def rand(*shape):
            return torch.randn(*shape, generator=gen, device=device)

        self.weights = dict(
            norm=(1 + 0.1 * rand(model)).to(dtype), proj=(rand(self.mixed + self.values + 2 * v_heads, model) / model ** 0.5).to(dtype),
            conv=(rand(self.mixed, WIDTH) / WIDTH ** 0.5).to(dtype), rate=torch.exp(rand(v_heads)), dt_bias=rand(v_heads) - 3,
            head_norm=(1 + 0.1 * rand(head)).to(dtype), out=(rand(model, self.values) / self.values ** 0.5).to(dtype))
        self.conv_states = torch.zeros(slots, WIDTH - 1, self.mixed, dtype=dtype, device=device)
        self.states = torch.zeros(slots, v_heads, head, head, device=device)

    def _enter(self, x, residual):
        """The projection's parts behind the norm, and the sum."""
        w = self.weights
        h, total = kda.layer_norm(x, w["norm"], residual=residual, norm="rms", eps=EPS)
        p = h @ w["proj"].t()
        z = p[..., self.mixed:self.mixed + self.values].unflatten(-1, (self.v_heads, self.head))  # a slice: its rows lie apart
        logits = p[..., self.mixed + self.values:].float()
        return h, total, p, z, logits

    def _decay(self, logits):
        w = self.weights
        g = -w["rate"] * torch.nn.functional.softplus(logits[..., :self.v_heads] + w["dt_bias"])
        return g, torch.sigmoid(logits[..., self.v_heads:])

    def _heads(self, y):
        q, k = (t.unflatten(-1, (self.k_heads, self.head)) for t in (y[..., :self.keys], y[..., self.keys:2 * self.keys]))
        return q, k, y[..., 2 * self.keys:].unflatten(-1, (self.v_heads, self.head))

    def _leave(self, o, z):
        n, _ = kda.layer_norm(o, self.weights["head_norm"], gate=z, norm="rms", eps=EPS)
        return n, n.flatten(-2) @ self.weights["out"].t()

    def prompt(self, x, residual, cu_seqlens, slots):
        _, total, p, z, logits = self._enter(x, residual)
        first = torch.full_like(slots, -1)  # new sequences start from nothing
        y, _ = kda.conv_prefill(p[..., :self.mixed], self.weights["conv"], cu_seqlens=cu_seqlens, initial_state=self.conv_states,
                                final_state=self.conv_states, initial_state_indices=first, final_state_indices=slots)
        q, k, v = self._heads(y)
        q, k = kda.qk_norm_rotary(q, k, norm="l2", eps=EPS)
        g, beta = self._decay(logits)
        o, _ = kda.delta_prefill(q, k, v, g, beta, cu_seqlens=cu_seqlens, initial_state=self.states, final_state=self.states,
                                 initial_state_indices=first, final_state_indices=slots)
        return self._leave(o, z)[1], total

    def token(self, x, residual, slots):
        _, total, p, z, logits = self._enter(x, residual)
        y = kda.conv_decode_step(p[..., :self.mixed], self.weights["conv"], self.conv_states, state_indices=slots)
        q, k, v = self._heads(y)
        q, k = kda.qk_norm_rotary(q, k, norm="l2", eps=EPS)
        g, beta = self._decay(logits)
        o = kda.delta_decode_step(q, k, v, g, beta, self.states, state_indices=slots)
        return self._leave(o, z)[1], total

    def gradients(self, x, residual, d_out, d_total):
        """Gradients of sum(d_out * output) + sum(d_total * sum), fp32: of the weights by name, and of x (which is the residual's too)."""
        w, kind = self.weights, x.dtype
        h, total, p, z, logits = self._enter(x, residual)
        y, _ = kda.conv_prefill(p[..., :self.mixed], w["conv"], output_final_state=False)
        q0, k0, v = self._heads(y)
        q, k = kda.qk_norm_rotary(q0, k0, norm="l2", eps=EPS)
        raw = logits[..., :self.v_heads] + w["dt_bias"]
        g, beta = self._decay(logits)
        o, _ = kda.delta_prefill(q, k, v, g, beta, output_final_state=False)
        n, _ = self._leave(o, z)
        grads = dict(out=d_out.flatten(0, -2).t().float() @ n.flatten(-2).flatten(0, -2).float())
        d_n = (d_out @ w["out"]).unflatten(-1, (self.v_heads, self.head))
        norm = kda.layer_norm_backward(o, w["head_norm"], d_n, gate=z, norm="rms", eps=EPS)
        grads["head_norm"] = norm["dweight"]
        m = kda.delta_backward(q, k, v, g, beta, norm["dx"].to(kind), want_d_initial_state=False)
        unit = kda.qk_norm_rotary_backward(q0, k0, None, None, None, m["dq"].to(kind), m["dk"].to(kind), norm="l2", eps=EPS)
        d_y = torch.cat([unit["dq"].flatten(-2), unit["dk"].flatten(-2), m["dv"].flatten(-2)], -1)
        c = kda.conv_backward(p[..., :self.mixed], w["conv"], d_y.to(kind), want_d_initial_state=False)
        grads["conv"] = c["dweight"]
        step = torch.nn.functional.softplus(raw)
        d_raw = -m["dg"] * w["rate"] * torch.sigmoid(raw)
        grads["rate"], grads["dt_bias"] = -(m["dg"] * step).flatten(0, -2).sum(0), d_raw.flatten(0, -2).sum(0)
        d_p = torch.cat([c["dx"], norm["dgate"].flatten(-2), d_raw, m["dbeta"] * beta * (1 - beta)], -1)
        grads["proj"] = d_p.flatten(0, -2).t() @ h.flatten(0, -2).float()
        first = kda.layer_norm_backward(total, w["norm"], (d_p @ w["proj"].float()).to(kind), norm="rms", eps=EPS, d_sum=d_total)
        grads["norm"] = first["dweight"]
        return grads, first["dx"]


def main(model=256, k_heads=2, v_heads=4, head=64, lengths=(70, 1, 133, 40), tokens=5, device="cuda:0"):
    """Prints and returns the largest difference between tokens and prompts."""
    gen = torch.Generator(device=device)
    gen.manual_seed(0)
    dtype, count = torch.bfloat16, len(lengths)
    layer = DeltaLayer(model, k_heads, v_heads, head, 2 * count, dtype, device, gen)
    x, res = ([torch.randn(t + tokens, model, generator=gen, device=device).to(dtype) for t in lengths] for _ in range(2))

    def packed(parts):
        cu = torch.tensor([0] + [len(p) for p in parts], device=device).cumsum(0).to(torch.int32)
        return torch.cat(parts)[None], cu

    slots = torch.arange(count, dtype=torch.int32, device=device)
    rows, cu = packed([p[:t] for p, t in zip(x, lengths)])
    layer.prompt(rows, packed([p[:t] for p, t in zip(res, lengths)])[0], cu, slots)
    steps = [layer.token(*(torch.stack([p[t + i] for p, t in zip(parts, lengths)]) for parts in (x, res)), slots)[0] for i in range(tokens)]
    rows, cu = packed(x)  # prompt and tokens as one prompt, in other slots
    whole = layer.prompt(rows, packed(res)[0], cu, slots + count)[0][0].float()
    want = torch.stack([whole[int(cu[s + 1]) - tokens:int(cu[s + 1])] for s in range(count)], 1)
    off = float((torch.stack(steps).float() - want).norm() / want.norm())
    print(f"delta layer: {tokens} tokens of {count} sequences against one prompt: {off:.2e} relative")
    rows, more, d = (torch.randn(2, 128, model, generator=gen, device=device).to(dtype) for _ in range(3))
    grads, dx = layer.gradients(rows, more, d, None)
    print("gradients: " + ", ".join(f"{name} {float(g.norm()):.3g}" for name, g in grads.items()) + f", x {float(dx.norm()):.3g}")
    kda.check_status(device)
    return off


if __name__ == "__main__":
    main()
