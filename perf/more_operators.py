"""Workloads of the gated delta rule with one decay per value head (prompts, single tokens, gradients) and of the layer norm with the
residual sum before it and the gate behind it (forward and gradients).

Every operator is written here in a plain form (elementary torch operations in 32 bits, rounded once at the end) and once more,
apart from it, in 64 bits (``exact``). With ``own`` true, ``run`` makes the calls of ``gated_delta_rule_56_gb300`` instead."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"


def _kda():
    import gated_delta_rule_56_gb300 as kda
    return kda


# ------------------------------------------------------------------------------- cases ---


def listed():
    return [
        # The headline prompt batch: 32 value heads that share 16 key heads.
        dict(name="delta prompt", op="delta", form="prompt", dtype="bf16", batch=4, tokens=8192, seqs=0, k_heads=16, v_heads=32,
             dk=128, dv=128, states=False),
        # Packed prompts of ragged lengths that go on from cached states, as a server runs them.
        dict(name="delta prompt packed", op="delta", form="prompt", dtype="bf16", batch=1, tokens=20011, seqs=37, k_heads=8,
             v_heads=16, dk=128, dv=128, states=True),
        # The smallest prompt: a short one in fp32 over 4 heads of 64, where latency counts.
        dict(name="delta prompt short", op="delta", form="prompt", dtype="fp32", batch=1, tokens=257, seqs=0, k_heads=2,
             v_heads=4, dk=64, dv=64, states=True),
        # One token for each of 256 sequences, the states updated in place.
        dict(name="delta token", op="delta", form="token", dtype="bf16", batch=256, tokens=1, seqs=0, k_heads=16, v_heads=32,
             dk=128, dv=128, states=True),
        # One token of one sequence: the smallest call there is.
        dict(name="delta token single", op="delta", form="token", dtype="bf16", batch=1, tokens=1, seqs=0, k_heads=16,
             v_heads=32, dk=128, dv=128, states=True),
        # A training step's gradients.
        dict(name="delta backward", op="delta", form="backward", dtype="bf16", batch=2, tokens=2048, seqs=0, k_heads=16,
             v_heads=32, dk=128, dv=128, states=False),
        # Gradients of packed sequences in fp32, through states before and behind them, smaller heads.
        dict(name="delta backward packed", op="delta", form="backward", dtype="fp32", batch=1, tokens=1501, seqs=9, k_heads=4,
             v_heads=8, dk=64, dv=64, states=True),
        # The mixer's output, head by head, with its gate: the headline prompt batch's 32 heads of 128.
        dict(name="norm prompt gated", op="norm", form="prompt", dtype="bf16", batch=4, tokens=8192, heads=32, width=128, rms=True,
             bias=False, residual=False, gate="silu"),
        # A layer's entry: the sum with the residual and its norm, as wide as 32 heads of 128.
        dict(name="norm prompt residual", op="norm", form="prompt", dtype="bf16", batch=4, tokens=2048, heads=1, width=4096,
             rms=False, bias=True, residual=True, gate=""),
        # The same for one token of 16 sequences.
        dict(name="norm token", op="norm", form="token", dtype="bf16", batch=16, tokens=1, heads=1, width=4096, rms=True,
             bias=False, residual=True, gate=""),
        # A training step's gradients through the gated norm of the mixer's output.
        dict(name="norm backward gated", op="norm", form="backward", dtype="bf16", batch=2, tokens=4096, heads=32, width=128,
             rms=True, bias=False, residual=False, gate="silu"),
        # Gradients through a layer norm with weight and bias at an odd width, fp32, with the residual's own gradient added.
        dict(name="norm backward odd", op="norm", form="backward", dtype="fp32", batch=3, tokens=1367, heads=1, width=1531, rms=False,
             bias=True, residual=True, gate=""),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "norm"])
    form = rng.choice(["prompt", "prompt", "backward", "token"])
    case = dict(op=op, form=form, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "norm":
        if rng.random() < 0.4:
            heads, width = rng.choice([4, 8, 16, 32]), rng.choice([32, 64, 128, 128, 256])
        else:
            heads, width = 1, rng.choice([_log(rng, 64, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192) // 8 * 8])
        most = (1 << 27) // (heads * width) // (4 if form == "backward" else 1)
        rows = _log(rng, 1, 256) if form == "token" else _log(rng, 64, max(65, min(32768, most)))
        batch = rows if form == "token" else rng.choice([1, 1, 2, 3])
        rms = rng.random() < 0.5
        return dict(case, batch=batch, tokens=1 if form == "token" else max(1, rows // batch), heads=heads, width=width, rms=rms,
                    bias=not rms and rng.random() < 0.7, residual=heads == 1 and rng.random() < 0.5,
                    gate=rng.choice(["silu", "sigmoid"]) if heads > 1 else "")
    k_heads, per = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4])
    v_heads = k_heads * per
    dk, dv = rng.choice([32, 64, 128, 128, 128]), rng.choice([32, 64, 128, 128, 128])
    case.update(k_heads=k_heads, v_heads=v_heads, dk=dk, dv=dv)
    if form == "token":
        return dict(case, batch=_log(rng, 1, max(2, min(512, (1 << 27) // (v_heads * dk * dv)))), tokens=1, seqs=0, states=True)
    most = (1 << (31 if form == "backward" else 33)) // (v_heads * dk * dv)
    tokens = _log(rng, 1, max(2, min(8192, most)))
    packed = rng.random() < 0.5
    batch = 1 if packed else rng.choice([1, 1, 2, 3, 5])
    return dict(case, batch=batch, tokens=tokens if packed else max(1, tokens // batch),
                seqs=rng.randint(1, max(1, min(64, tokens // 16))) if packed else 0, states=rng.random() < 0.5)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows, back = case["batch"] * case["tokens"], case["form"] == "backward"
    if case["op"] == "norm":
        n = rows * case["heads"] * case["width"]
        more = 1 if case["gate"] else 0
        if back:
            # x, dy (z, the sum's gradient) read; dx (dz) written in 32 bits.
            return {"bytes": n * (e * (2 + more + (1 if case["residual"] else 0)) + 4 * (1 + more)) + case["width"] * (e + 4) * 2,
                    "flops": n * (12 + 10 * more)}
        return {"bytes": n * e * (2 + more + (2 if case["residual"] else 0)) + case["width"] * e, "flops": n * (8 + 6 * more)}
    hk, hv, dk, dv = case["k_heads"], case["v_heads"], case["dk"], case["dv"]
    seqs, one = case["seqs"] or case["batch"], hv * dk * dv * 4
    reads = rows * (e * (2 * hk * dk + hv * dv) + 8 * hv)
    if back:
        states = seqs * one * (3 if case["states"] else 1)
        return {"bytes": reads + rows * (hv * dv * (e + 4) + 8 * hk * dk + 8 * hv) + states, "flops": rows * hv * dk * dv * 16}
    states = seqs * one * (2 if case["states"] else 1)
    return {"bytes": reads + rows * hv * dv * e + states, "flops": rows * hv * dk * dv * 6}


# ------------------------------------------------------------------------------ inputs ---


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _lengths(case, seed):
    """Ragged lengths of packed sequences (some of one token, now and then an empty one), summing to the tokens."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 7 + 3)
    n, total = case["seqs"], case["tokens"]
    cuts = torch.sort(torch.randint(0, total + 1, (n - 1,), generator=g)).values
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([total])]).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    B, T, form = case["batch"], case["tokens"], case["form"]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(case=case)
    lead = (B,) if form == "token" else (B, T)
    if case["op"] == "norm":
        D, shape = case["width"], (*lead, case["heads"], case["width"]) if case["heads"] > 1 else (*lead, case["width"])
        s["x"] = (rand(*shape) * 1.5 + 0.25).to(dt)
        s["residual"] = (2 * rand(*shape)).to(dt) if case["residual"] else None
        if case["gate"]:  # the gate comes out of a wider projection
            s["wide"] = rand(*lead, 2 * case["heads"] * D).to(dt)
        s["weight"] = (1 + 0.2 * rand(D)).to(dt)
        s["bias"] = (0.2 * rand(D)).to(dt) if case["bias"] else None
        if form == "backward":
            s["dy"] = rand(*shape).to(dt)
            s["d_sum"] = rand(*shape).to(dt) if case["residual"] else None
        return s
    hk, hv, dk, dv, n_seqs = case["k_heads"], case["v_heads"], case["dk"], case["dv"], case["seqs"] or B
    if case["seqs"]:
        s["cu_seqlens"] = _lengths(case, seed).to(DEV)

    def silu(x):  # what the convolution's SiLU leaves
        return x * torch.sigmoid(x)

    def unit(x):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

    s["q"] = unit(silu(rand(*lead, hk, dk))).to(dt)
    s["k"] = unit(silu(rand(*lead, hk, dk))).to(dt)
    s["conv"] = silu(rand(*lead, 2 * hk * dk + hv * dv)).to(dt)  # v lies behind what q and k were made from
    # g = -A dt: time steps of 1e-3 to 1e-1 that the input moves, rates of 1 to 16 per head
    first = torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(100.0)) * 1e-3
    raw = 0.5 * rand(*lead, hv) + first + torch.log(-torch.expm1(-first))
    rate = torch.exp(torch.rand(hv, generator=g, device=DEV) * math.log(16.0))
    s["g"] = -rate * (torch.clamp(raw, min=0) + torch.log1p(torch.exp(-torch.abs(raw))))
    s["beta"] = torch.sigmoid(rand(*lead, hv))
    s["state"] = 0.1 * rand(n_seqs, hv, dk, dv) if case["states"] else None
    if form == "backward":
        s["d_o"] = rand(*lead, hv, dv).to(dt)
        s["d_final"] = 0.1 * rand(n_seqs, hv, dk, dv) if case["states"] else None
    return s


def _value(s):
    """The values' slice of the convolution's output."""
    c = s["case"]
    return s["conv"][..., 2 * c["k_heads"] * c["dk"]:].unflatten(-1, (c["v_heads"], c["dv"]))


def _gate(s):
    """The gate's slice of the projection."""
    c = s["case"]
    z = s["wide"][..., c["heads"] * c["width"]:]
    return z.unflatten(-1, (c["heads"], c["width"])) if c["heads"] > 1 else z


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c["form"])


# --------------------------------------------------------------- the framework's calls ---


def _own_delta(s, form):
    kda, v = _kda(), _value(s)
    if form == "token":
        return kda.delta_decode_step(s["q"], s["k"], v, s["g"], s["beta"], s["state"]), s["state"]
    if form == "prompt":
        return kda.delta_prefill(s["q"], s["k"], v, s["g"], s["beta"], cu_seqlens=s.get("cu_seqlens"), initial_state=s["state"])
    g = kda.delta_backward(s["q"], s["k"], v, s["g"], s["beta"], s["d_o"], cu_seqlens=s.get("cu_seqlens"),
                           initial_state=s["state"], d_final_state=s["d_final"])
    return [g[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state")]


def _own_norm(s, form):
    kda, c = _kda(), s["case"]
    more = dict(bias=s["bias"], gate=_gate(s) if c["gate"] else None, activation=c["gate"] or "silu",
                norm="rms" if c["rms"] else "layer", eps=1e-6)
    if form != "backward":
        return kda.layer_norm(s["x"], s["weight"], residual=s["residual"], **more)
    g = kda.layer_norm_backward(s["x"], s["weight"], s["dy"], d_sum=s["d_sum"], **more)
    return [g[n] for n in ("dx", "dweight", "dbias", "dgate")]


_own = {"delta": _own_delta, "norm": _own_norm}


# ------------------------------------------------------------------------- plain forms ---


def _places(s):
    """For every place [sequence, token of it] its row, and whether it has one."""
    c = s["case"]
    if s.get("cu_seqlens") is None:
        rows = torch.arange(c["batch"] * c["tokens"], device=DEV).view(c["batch"], c["tokens"])
        return rows, torch.ones_like(rows, dtype=torch.bool)
    cu = s["cu_seqlens"].long()
    at = cu[:-1, None] + torch.arange(int((cu[1:] - cu[:-1]).max()), device=DEV)
    return at.clamp(max=c["tokens"] - 1), at < cu[1:, None]


CHUNK = 64


def _chunks(x, rows, some, per, wide=torch.float32):
    """[rows, heads, ...] as [sequence, value head, chunk, row, ...], zeros where a sequence has no row."""
    x = x[rows].to(wide) * some.view(*some.shape, *[1] * (x.dim() - 1))
    x = x.repeat_interleave(per, 2) if per > 1 else x
    more = -x.shape[1] % CHUNK
    x = torch.cat([x, x.new_zeros(x.shape[0], more, *x.shape[2:])], 1) if more else x
    return x.unflatten(1, (-1, CHUNK)).movedim(3, 1)


def _rows(x, rows, some):
    """The other way: [sequence, head, chunk, row, ...] to [rows, head, ...]."""
    x = x.movedim(1, 3).flatten(1, 2)[:, :rows.shape[1]]
    return x[some]


def _inverse(a):
    """(I + a)^-1 of strictly lower triangular a, by Newton's iteration: every step doubles the diagonals that are right."""
    eye = torch.eye(CHUNK, device=a.device)
    x = eye - a
    for _ in range(6):
        x = x @ (2 * eye - (x + a @ x))
    return x


def _plain_delta(s, form):
    c = s["case"]
    per, kind, lead = c["v_heads"] // c["k_heads"], s["q"].dtype, s["q"].shape[:-2]
    v = _value(s)
    if form == "token":
        q, k, v = (t.float() for t in (s["q"].repeat_interleave(per, 1), s["k"].repeat_interleave(per, 1), v))
        S = s["state"] * torch.exp(s["g"])[..., None, None]
        u = s["beta"][..., None] * (v - (k[..., None] * S).sum(-2))
        S = S + k[..., None] * u[..., None, :]
        s["state"].copy_(S)
        return (q[..., None] * S).sum(-2).to(kind), s["state"]
    rows, some = _places(s)
    q, k = (_chunks(s[n].flatten(0, 1), rows, some, per) for n in ("q", "k"))
    v = _chunks(v.flatten(0, 1), rows, some, 1)
    beta = _chunks(s["beta"].flatten(0, 1), rows, some, 1)[..., None]
    G = _chunks(s["g"].flatten(0, 1), rows, some, 1, torch.float64).cumsum(-1)
    D = torch.exp((G[..., :, None] - G[..., None, :]).float().tril())
    first, last, whole = (torch.exp(t.float()) for t in (G[..., None], (G[..., -1:] - G)[..., None], G[..., -1:, None]))
    del G
    A = (beta * D * (k @ k.mT)).tril(-1)
    P = (D * (q @ k.mT)).tril()
    T = _inverse(A)
    n = rows.shape[0]
    S = torch.zeros(n, c["v_heads"], c["dk"], c["dv"], device=DEV) if s["state"] is None else s["state"]
    before, U, o = [], [], []
    for i in range(q.shape[2]):
        before.append(S)
        u = T[:, :, i] @ (beta[:, :, i] * (v[:, :, i] - first[:, :, i] * (k[:, :, i] @ S)))
        if form == "prompt":
            o.append(first[:, :, i] * (q[:, :, i] @ S) + P[:, :, i] @ u)
            before.clear()
        else:
            U.append(u)
        S = whole[:, :, i] * S + (last[:, :, i] * k[:, :, i]).mT @ u
    if form == "prompt":
        return _rows(torch.stack(o, 2), rows, some).to(kind).view(*lead, c["v_heads"], c["dv"]), S.clone()
    d_o = _chunks(s["d_o"].flatten(0, 1), rows, some, 1)
    U, before = torch.stack(U, 2), torch.stack(before, 2)
    dS = torch.zeros_like(S) if s["d_final"] is None else s["d_final"]
    behind, dR, joined = [None] * q.shape[2], [None] * q.shape[2], [None] * q.shape[2]
    for i in reversed(range(q.shape[2])):
        behind[i], joined[i] = dS, (S * dS).sum((-1, -2))
        dR[i] = T[:, :, i].mT @ (P[:, :, i].mT @ d_o[:, :, i] + last[:, :, i] * (k[:, :, i] @ dS))
        dS = (whole[:, :, i] * dS + (first[:, :, i] * q[:, :, i]).mT @ d_o[:, :, i]
              - (beta[:, :, i] * first[:, :, i] * k[:, :, i]).mT @ dR[i])
        S = before[:, :, i]
    behind, dR, joined = torch.stack(behind, 2), torch.stack(dR, 2), torch.stack(joined, 2)
    gp = D * (d_o @ U.mT).tril()
    ga = D * (-(dR @ U.mT)).tril(-1)
    dq = first * (d_o @ before.mT) + gp @ k
    row = ga @ k - first * (dR @ before.mT)
    col = last * (U @ behind.mT) + gp.mT @ q + (beta * ga).mT @ k
    kr = (k * row).sum(-1, keepdim=True)
    dbeta = ((dR * v).sum(-1, keepdim=True) + kr)[..., 0]
    dG = ((q * dq).sum(-1, keepdim=True) + beta * kr - (k * col).sum(-1, keepdim=True))[..., 0]
    dG[..., -1] += joined
    dg = dG.double().flip(-1).cumsum(-1).flip(-1).float()

    def shared(x):  # summed over the value heads of a key head
        x = _rows(x, rows, some)
        return x.unflatten(1, (c["k_heads"], per)).sum(2).view(*lead, c["k_heads"], c["dk"])

    return [shared(dq), shared(beta * row + col), _rows(beta * dR, rows, some).view(*lead, c["v_heads"], c["dv"]),
            _rows(dg, rows, some).view(*lead, c["v_heads"]), _rows(dbeta, rows, some).view(*lead, c["v_heads"]), dS.clone()]


def _plain_norm(s, form):
    c, kind = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    z = _gate(s).float() if c["gate"] else None
    if form != "backward" and s["residual"] is not None:
        x = x + s["residual"].float()
    h = x if c["rms"] else x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
    h = h * r
    n = h * w if s["bias"] is None else h * w + s["bias"].float()
    sg = None if z is None else torch.sigmoid(z)
    act = None if z is None else z * sg if c["gate"] == "silu" else sg
    if form != "backward":
        return (n if act is None else n * act).to(kind), None if s["residual"] is None else x.to(kind)
    d, dz = s["dy"].float(), None
    if z is not None:
        dz = d * n * (sg * (1 + z * (1 - sg)) if c["gate"] == "silu" else sg * (1 - sg))
        d = d * act
    dw = (d * h).flatten(0, -2).sum(0, dtype=torch.float64).float()
    db = None if s["bias"] is None else d.flatten(0, -2).sum(0, dtype=torch.float64).float()
    d = d * w
    dx = d - h * (d * h).mean(-1, keepdim=True)
    dx = r * (dx if c["rms"] else dx - d.mean(-1, keepdim=True))
    return [dx if s["d_sum"] is None else dx + s["d_sum"].float(), dw, db, dz]


_plain = {"delta": _plain_delta, "norm": _plain_norm}


# --------------------------------------------------------------------- in 64 bits ---------


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "norm": _exact_norm}[case["op"]](s, case["form"])


def _exact_delta(s, form):
    """Token by token; sequences side by side, each token on those that are that long."""
    c = s["case"]
    hk, hv, dk, dv = c["k_heads"], c["v_heads"], c["dk"], c["dv"]
    lead, per = s["q"].shape[:-2], hv // hk
    q, k, v = (t.reshape(-1, *t.shape[-2:]).double() for t in (s["q"], s["k"], _value(s)))
    a, b = torch.exp(s["g"].reshape(-1, hv).double()), s["beta"].reshape(-1, hv).double()
    if s.get("cu_seqlens") is not None:
        cu = s["cu_seqlens"].tolist()
        spans = list(zip(cu[:-1], cu[1:]))
    else:
        spans = [(n * c["tokens"], (n + 1) * c["tokens"]) for n in range(c["batch"])]
    order = sorted(range(len(spans)), key=lambda n: spans[n][0] - spans[n][1])  # longest first
    start = torch.tensor([spans[n][0] for n in order], device=DEV)
    lens = [spans[n][1] - spans[n][0] for n in order]
    live = [sum(1 for x in lens if x > t) for t in range(max(lens))] if len(lens) < 64 or max(lens) < 10000 else None
    if live is None or (form == "backward" and q.shape[0] * hv * dk * dv * 8 > 40e9):
        return None
    S = torch.zeros(len(order), hv, dk, dv, device=DEV, dtype=torch.float64) if s["state"] is None else s["state"][order].double()
    o = torch.empty(q.shape[0], hv, dv, device=DEV, dtype=torch.float64)
    kept = torch.empty(q.shape[0], hv, dk, dv, device=DEV, dtype=torch.float64) if form == "backward" else None

    def at(x, rows):  # a key head's rows for each of its value heads
        return x[rows].repeat_interleave(per, 1)

    for t, m in enumerate(live):
        rows = start[:m] + t
        kt = at(k, rows)
        if kept is not None:
            kept[rows] = S[:m]
        S[:m] *= a[rows][..., None, None]
        u = b[rows][..., None] * (v[rows] - torch.einsum("nhkv,nhk->nhv", S[:m], kt))
        S[:m] += torch.einsum("nhk,nhv->nhkv", kt, u)
        o[rows] = torch.einsum("nhkv,nhk->nhv", S[:m], at(q, rows))
    there = torch.tensor(order, device=DEV)
    if form != "backward":
        final = torch.empty_like(S)
        final[there] = S
        return o.view(*lead, hv, dv), final
    d_o = s["d_o"].reshape(-1, hv, dv).double()
    dS = torch.zeros_like(S) if s["d_final"] is None else s["d_final"][order].double()
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(a), torch.empty_like(b)
    for t, m in reversed(list(enumerate(live))):
        rows = start[:m] + t
        kt, at_, bt = at(k, rows), a[rows][..., None, None], b[rows]
        old = at_ * kept[rows]  # the state after the decay
        miss = v[rows] - torch.einsum("nhkv,nhk->nhv", old, kt)
        u = bt[..., None] * miss
        new = old + torch.einsum("nhk,nhv->nhkv", kt, u)
        grad = dS[:m] + torch.einsum("nhk,nhv->nhkv", at(q, rows), d_o[rows])
        dqt = torch.einsum("nhkv,nhv->nhk", new, d_o[rows])
        du = torch.einsum("nhkv,nhk->nhv", grad, kt)
        db[rows] = (du * miss).sum(-1)
        w = bt[..., None] * du
        dv_[rows] = w
        dkt = torch.einsum("nhkv,nhv->nhk", grad, u) - torch.einsum("nhkv,nhv->nhk", old, w)
        grad = grad - torch.einsum("nhk,nhv->nhkv", kt, w)
        dg[rows] = (grad * old).sum((-1, -2))
        dS[:m] = at_ * grad
        dq[rows], dk_[rows] = (x.view(m, hk, per, dk).sum(2) for x in (dqt, dkt))
    d_init = torch.empty_like(dS)
    d_init[there] = dS
    return [dq.view(*lead, hk, dk), dk_.view(*lead, hk, dk), dv_.view(*lead, hv, dv), dg.view(*lead, hv), db.view(*lead, hv), d_init]


def _exact_norm(s, form):
    c = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    b = 0.0 if s["bias"] is None else s["bias"].double()
    total = x if form == "backward" or s["residual"] is None else x + s["residual"].double()
    middle = 0.0 if c["rms"] else total.mean(-1, keepdim=True)
    size = torch.sqrt((total - middle).square().mean(-1, keepdim=True) + 1e-6)
    unit = (total - middle) / size
    z = _gate(s).double() if c["gate"] else None
    e = None if z is None else 1 / (1 + torch.exp(-z))
    times = 1.0 if z is None else z * e if c["gate"] == "silu" else e
    if form != "backward":
        return (unit * w + b) * times, None if s["residual"] is None else total
    d = s["dy"].double() * times
    dz = None
    if z is not None:
        slope = e * (1 - e)
        dz = s["dy"].double() * (unit * w + b) * (e + z * slope if c["gate"] == "silu" else slope)
    dw, db = ((d * y).reshape(-1, c["width"]).sum(0) for y in (unit, torch.ones_like(unit)))
    t = d * w
    dx = t - unit * (t * unit).mean(-1, keepdim=True) - (0.0 if c["rms"] else t.mean(-1, keepdim=True))
    dx = dx / size + (0.0 if s["d_sum"] is None else s["d_sum"].double())
    return [dx, dw, None if s["bias"] is None else db, dz]
