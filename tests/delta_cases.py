"""Inputs, calls and comparisons that the GPU tests of the delta rule with one decay per value head share."""

import torch

import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from layers_cases import DEV, HALF, ULP32, cu_of, d64, gen, near

GRADS = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")


class Case:
    def __init__(self, dtype, B, T, hk, hv, dk, dv, lengths=None, seed=0, states=True, decay=1.0):
        r = gen(seed)
        self.dtype, self.lengths, self.heads, self.sizes = dtype, lengths, (hk, hv), (dk, dv)
        if lengths is not None:
            B, T = 1, sum(lengths)
        self.shape = (B, T)
        self.cu = None if lengths is None else cu_of(lengths)
        n = B if lengths is None else len(lengths)

        def unit(x):
            return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

        self.q, self.k = (unit(r(B, T, hk, dk)).to(dtype) for _ in range(2))
        self.v = r(B, T, hv, dv).to(dtype)
        self.g = -decay * torch.rand(B, T, hv, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed + 100)) ** 3
        self.beta = torch.sigmoid(r(B, T, hv))
        self.state = 0.3 * r(n, hv, dk, dv) if states else None
        self.d_o = r(B, T, hv, dv).to(dtype)
        self.d_final = 0.3 * r(n, hv, dk, dv) if states else None

    def inputs(self):
        return self.q, self.k, self.v, self.g, self.beta

    def prefill(self, **more):
        return kda.delta_prefill(*self.inputs(), **{**dict(cu_seqlens=self.cu, initial_state=self.state), **more})

    def backward(self, **more):
        return kda.delta_backward(*self.inputs(), self.d_o, **{**dict(cu_seqlens=self.cu, initial_state=self.state,
                                                                      d_final_state=self.d_final), **more})

    def sequences(self):
        """Each sequence's inputs in 64 bits, key heads repeated, with d_o and d_final."""
        (B, T), (hk, hv), (dk, dv) = self.shape, self.heads, self.sizes
        lens = self.lengths if self.lengths is not None else [T] * B
        at = 0
        for n, m in enumerate(lens):
            rows = slice(at, at + m)
            at += m
            q, k, v, g, b, do = (d64(t.flatten(0, 1)[rows]) for t in (*self.inputs(), self.d_o))
            q, k = (t.repeat_interleave(hv // hk, 1) for t in (q, k))
            S = torch.zeros(hv, dk, dv, dtype=torch.float64) if self.state is None else d64(self.state[n])
            df = torch.zeros(hv, dk, dv, dtype=torch.float64) if self.d_final is None else d64(self.d_final[n])
            yield (q, k, v, g, b, S), do, df

    def longest(self):
        return max(self.lengths) if self.lengths else self.shape[1]

    def tolerance(self):
        # A token's update loses to rounding: the decayed state and the sum (1 half step each), the read k^T S (a sum of up to 128 terms in
        # chains of 8 pairs and 4 levels: 12), u and the decay's exponential (4 together): under 24 half steps of the state's norm, of random signs,
        # so sqrt(tokens) of them meet; the reading adds one more read. The tensor-core form holds operands in two bf16 values, which is
        # 2^-17 at most of an operand's size, three operands to a product's chain (state, U, T), instead of the read's share.
        m = max(1, self.longest())
        return ULP32 * (32 + 24 * m ** 0.5) + (3 * 2.0 ** -17 if self.dtype == torch.bfloat16 else 0)

    def check_prefill(self, o, fin):
        hv, (dk, dv) = self.heads[1], self.sizes
        want = [ref.delta(*s) for s, _, _ in self.sequences()]
        tol = self.tolerance()
        half = HALF[self.dtype] if self.dtype == torch.bfloat16 else 0
        near("o", o.reshape(-1, hv, dv), torch.cat([w[0] for w in want]), tol + half)
        if fin is not None:
            near("final_state", fin, torch.stack([w[1] for w in want]), tol)

    def check_backward(self, g=None):
        g = g or self.backward()
        (hk, hv), (dk, dv) = self.heads, self.sizes
        want = [ref.delta_backward(*s, do, df) for s, do, df in self.sequences()]
        # The states and their gradients both carry the error of a pass; the gradients of g are differences of sums of both signs.
        tol = 4 * self.tolerance()
        shared = lambda i: torch.cat([w[i].unflatten(1, (hk, hv // hk)).sum(2) for w in want])  # noqa: E731
        plain = lambda i: torch.cat([w[i] for w in want])  # noqa: E731
        near("dq", g["dq"].flatten(0, 1), shared(0), tol)
        near("dk", g["dk"].flatten(0, 1), shared(1), tol)
        near("dv", g["dv"].flatten(0, 1), plain(2), tol)
        near("dg", g["dg"].flatten(0, 1), plain(3), 4 * tol)
        near("dbeta", g["dbeta"].flatten(0, 1), plain(4), tol)
        if g["d_initial_state"] is not None:
            near("d_initial_state", g["d_initial_state"], torch.stack([w[5] for w in want]), tol)
