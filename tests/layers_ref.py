"""64-bit references of the operators around the mixer, one sequence at a time, from their definitions."""

import torch


def spans(batch, tokens, cu=None):
    """(first row, end row) of every sequence over the flattened rows."""
    if cu is None:
        return [(n * tokens, (n + 1) * tokens) for n in range(batch)]
    cu = cu.tolist()
    return list(zip(cu[:-1], cu[1:]))


def silu(p):
    return p * torch.sigmoid(p)


def d_silu(p):
    s = torch.sigmoid(p)
    return s + p * s * (1 - s)


def conv(x, weight, bias, act, init):
    """One sequence: x [T, C], init [W-1, C] -> y, final state, all fp64."""
    W = weight.shape[1]
    line = torch.cat([init, x])
    p = torch.zeros_like(x) if bias is None else bias.expand_as(x).clone()
    for t in range(x.shape[0]):
        for j in range(W):
            p[t] = p[t] + weight[:, j] * line[t + j]
    return (silu(p) if act else p), line[line.shape[0] - (W - 1):]


def conv_backward(x, weight, bias, act, init, dy, d_final):
    """One sequence -> dx, dweight, dbias, d_init."""
    W, T = weight.shape[1], x.shape[0]
    line = torch.cat([init, x])
    dline, dw = torch.zeros_like(line), torch.zeros_like(weight)
    db = torch.zeros_like(weight[:, 0])
    for t in range(T):
        p = sum(weight[:, j] * line[t + j] for j in range(W)) + (0 if bias is None else bias)
        d = dy[t] * (d_silu(p) if act else 1)
        for j in range(W):
            dline[t + j] += weight[:, j] * d
            dw[:, j] += d * line[t + j]
        db += d
    dline[line.shape[0] - (W - 1):] += d_final
    return dline[W - 1:], dw, db, dline[:W - 1]


def time_step(raw, softplus):
    return torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw


def scan(x, dt, A, B, C, D, z, softplus, init):
    """One sequence: x, dt (with its bias) [T, D], B, C [T, D, N] (each channel's group's) -> y, final state."""
    h, ys = init.clone(), torch.zeros_like(x)
    for t in range(x.shape[0]):
        step = time_step(dt[t], softplus)
        h = torch.exp(step[:, None] * A) * h + (step * x[t])[:, None] * B[t]
        ys[t] = (C[t] * h).sum(-1) + (0 if D is None else D * x[t])
    return (ys if z is None else ys * silu(z)), h


def scan_backward(x, dt, A, B, C, D, z, softplus, init, dy, d_final):
    """One sequence -> dict of gradients (dB, dC per channel: [T, D, N])."""
    T = x.shape[0]
    hs, step = [init.clone()], time_step(dt, softplus)
    for t in range(T):
        hs.append(torch.exp(step[t][:, None] * A) * hs[-1] + (step[t] * x[t])[:, None] * B[t])
    out = {k: torch.zeros_like(v) for k, v in (("dx", x), ("ddt", x), ("dA", A), ("dB", B), ("dC", C), ("dD", x[:0].sum(0)),
                                               ("dz", x))}
    g = d_final.clone()
    for t in reversed(range(T)):
        y = (C[t] * hs[t + 1]).sum(-1) + (0 if D is None else D * x[t])
        d = dy[t]
        if z is not None:
            out["dz"][t] = dy[t] * y * d_silu(z[t])
            d = dy[t] * silu(z[t])
        g = g + C[t] * d[:, None]
        out["dC"][t] = d[:, None] * hs[t + 1]
        out["dB"][t] = g * (step[t] * x[t])[:, None]
        a = torch.exp(step[t][:, None] * A)
        gb, kept = (g * B[t]).sum(-1), g * a * hs[t]
        out["dx"][t] = gb * step[t] + (0 if D is None else D * d)
        ds = gb * x[t] + (kept * A).sum(-1)
        out["ddt"][t] = ds * torch.sigmoid(dt[t]) if softplus else ds
        out["dA"] += kept * step[t][:, None]
        out["dD"] += d * x[t]
        g = g * a
    out["d_init"] = g
    return out


def norm_rotary(x, weight, cos, sin, rms, eps, interleaved):
    """x [rows, heads, d]; cos, sin [rows, half] -> the output."""
    u = x / torch.sqrt((x.square().mean(-1, keepdim=True) if rms else x.square().sum(-1, keepdim=True)) + eps)
    u = u if weight is None else u * weight
    return turn(u, cos, sin, interleaved)


def turn(u, cos, sin, interleaved):
    half = cos.shape[-1]
    out = u.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = cos[:, None, i], sin[:, None, i]
        out[..., a], out[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    return out


def norm_rotary_backward(x, weight, cos, sin, rms, eps, interleaved, d):
    """-> dx, dweight."""
    d = turn(d, cos, -sin, interleaved)
    size = x.shape[-1] if rms else 1
    r = 1 / torch.sqrt(x.square().sum(-1, keepdim=True) / size + eps)
    dw = (d * x * r).sum((0, 1))
    d = d if weight is None else d * weight
    return r * d - x * r ** 3 * (d * x).sum(-1, keepdim=True) / size, dw
