"""The delta rule with one decay per value head, and the layer norm with residual and gate, in 64 bits from their definitions: one
sequence at a time, row by row."""

import torch


def delta(q, k, v, g, beta, S):
    """q, k [T, H, dk], v [T, H, dv], g, beta [T, H], S [H, dk, dv] (key heads already repeated): o [T, H, dv] and the last state."""
    o = torch.zeros(v.shape, dtype=torch.float64)
    for t in range(q.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        read = torch.einsum("hkv,hk->hv", S, k[t])
        S = S + torch.einsum("hk,hv->hkv", k[t], beta[t][:, None] * (v[t] - read))
        o[t] = torch.einsum("hkv,hk->hv", S, q[t])
    return o, S


def delta_backward(q, k, v, g, beta, S, d_o, d_final):
    """Gradients of sum(d_o * o) + sum(d_final * last state): dq, dk, dv, dg, dbeta, dS."""
    states, T = [S], q.shape[0]
    for t in range(T):
        S = torch.exp(g[t])[:, None, None] * S
        read = torch.einsum("hkv,hk->hv", S, k[t])
        S = S + torch.einsum("hk,hv->hkv", k[t], beta[t][:, None] * (v[t] - read))
        states.append(S)
    dq, dk, dv, dg, db = (torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v, g, beta))
    dS = d_final.clone()
    for t in reversed(range(T)):
        a = torch.exp(g[t])[:, None, None]
        old = a * states[t]
        miss = v[t] - torch.einsum("hkv,hk->hv", old, k[t])
        dq[t] = torch.einsum("hkv,hv->hk", states[t + 1], d_o[t])
        dS = dS + torch.einsum("hk,hv->hkv", q[t], d_o[t])
        du = torch.einsum("hkv,hk->hv", dS, k[t])
        db[t] = (du * miss).sum(-1)
        dv[t] = beta[t][:, None] * du
        dk[t] = torch.einsum("hkv,hv->hk", dS, beta[t][:, None] * miss) - torch.einsum("hkv,hv->hk", old, dv[t])
        dold = dS - torch.einsum("hk,hv->hkv", k[t], dv[t])
        dg[t] = (dold * old).sum((-1, -2))
        dS = a * dold
    return dq, dk, dv, dg, db, dS


def act(z, kind):
    e = 1 / (1 + torch.exp(-z))
    return z * e if kind == "silu" else e


def layer_norm(x, w, b, res, z, kind, rms, eps):
    s = x if res is None else x + res
    h = s if rms else s - s.mean(-1, keepdim=True)
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = n if w is None else n * w
    n = n if b is None else n + b
    return (n if z is None else n * act(z, kind)), s


def layer_norm_backward(x, w, b, z, kind, rms, eps, dy, d_sum):
    """dx, dweight, dbias, dz of sum(dy * y) + sum(d_sum * x), x the sum."""
    h = x if rms else x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * r if w is None else h * r * w
    n = n if b is None else n + b
    d, dz = dy, None
    if z is not None:
        e = 1 / (1 + torch.exp(-z))
        slope = e + z * e * (1 - e) if kind == "silu" else e * (1 - e)
        d, dz = dy * act(z, kind), dy * n * slope
    dw, db = ((d * y).reshape(-1, x.shape[-1]).sum(0) for y in (h * r, torch.ones_like(x)))
    t = d if w is None else d * w
    dx = t - h * r * (t * h * r).mean(-1, keepdim=True)
    dx = r * (dx if rms else dx - t.mean(-1, keepdim=True))
    return dx if d_sum is None else dx + d_sum, None if w is None else dw, None if b is None else db, dz
