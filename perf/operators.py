"""Workloads of the operators around the KDA mixer: the short causal convolution, the selective state space scan, and the
per-head norm of queries and keys with the position rotation, each for prompts, for single tokens and with its gradients.

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
        # Convolution of q, k and v side by side (32 heads of 128 channels each) over the headline prompt batch.
        dict(name="conv prompt qkv", op="conv", form="prompt", dtype="bf16", batch=4, tokens=8192, seqs=0, channels=12288,
             width=4, silu=True, bias=False, states=False),
        # Packed prompts of ragged lengths that go on from cached states, as a server runs them.
        dict(name="conv prompt packed", op="conv", form="prompt", dtype="bf16", batch=1, tokens=20011, seqs=37, channels=4096,
             width=4, silu=True, bias=True, states=True),
        # A training step's gradients through the convolution of one projection.
        dict(name="conv backward", op="conv", form="backward", dtype="bf16", batch=4, tokens=8192, seqs=0, channels=4096,
             width=4, silu=True, bias=True, states=False),
        # One token for each of 256 sequences: q, k and v side by side, the state updated in place.
        dict(name="conv token", op="conv", form="token", dtype="bf16", batch=256, tokens=1, seqs=0, channels=12288, width=4,
             silu=True, bias=False, states=True),
        # One long prompt, as wide as 32 heads of 128: few sequences, so the work has to be found along the sequence.
        dict(name="scan prompt long", op="scan", form="prompt", dtype="bf16", batch=1, tokens=16384, seqs=0, channels=4096,
             state=16, groups=1, gate=True, skip=True, states=False),
        # Packed prompts of ragged lengths that go on from cached states.
        dict(name="scan prompt packed", op="scan", form="prompt", dtype="bf16", batch=1, tokens=12345, seqs=24, channels=2048,
             state=16, groups=2, gate=True, skip=True, states=True),
        # The smallest: a short fp32 prompt over 2 heads of 64, where latency counts.
        dict(name="scan prompt short", op="scan", form="prompt", dtype="fp32", batch=1, tokens=256, seqs=0, channels=128,
             state=16, groups=1, gate=False, skip=True, states=True),
        # A training step's gradients through the scan.
        dict(name="scan backward", op="scan", form="backward", dtype="bf16", batch=4, tokens=2048, seqs=0, channels=4096,
             state=16, groups=1, gate=True, skip=True, states=False),
        # One token for each of 256 sequences, the states updated in place.
        dict(name="scan token", op="scan", form="token", dtype="bf16", batch=256, tokens=1, seqs=0, channels=4096, state=16,
             groups=1, gate=True, skip=True, states=True),
        # Unit-length q and k with rotation for the KDA mixer over the headline prompt batch.
        dict(name="rotary prompt", op="rotary", form="prompt", dtype="bf16", batch=4, tokens=8192, q_heads=32, k_heads=32,
             head=128, rotary=128, rms=False, interleaved=False, table=65536),
        # Gradients through the weighted norm with shared key heads.
        dict(name="rotary backward", op="rotary", form="backward", dtype="bf16", batch=2, tokens=4096, q_heads=32, k_heads=8,
             head=128, rotary=64, rms=True, interleaved=False, table=32768),
        # One token for each of 256 sequences.
        dict(name="rotary token", op="rotary", form="token", dtype="bf16", batch=256, tokens=1, q_heads=32, k_heads=8,
             head=128, rotary=128, rms=True, interleaved=False, table=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "rotary"])
    form = rng.choice(["prompt", "prompt", "backward", "token"])
    case = dict(op=op, form=form, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "rotary":
        head = rng.choice([32, 64, 96, 128, 128, 256])
        k_heads = rng.choice([1, 2, 4, 8, 32])
        q_heads = k_heads * rng.choice([1, 2, 4])
        most = (1 << 27) // (head * (q_heads + k_heads)) // (4 if form == "backward" else 1)
        rows = _log(rng, 1, 512) if form == "token" else _log(rng, 64, max(65, min(32768, most)))
        batch = rows if form == "token" else rng.choice([1, 1, 2, 3])
        return dict(case, batch=batch, tokens=1 if form == "token" else max(1, rows // batch), q_heads=q_heads, k_heads=k_heads,
                    head=head, rotary=rng.choice([head, head // 2]), rms=rng.random() < 0.6, interleaved=rng.random() < 0.3,
                    table=rng.choice([4096, 32768, 131072]))
    channels = rng.choice([_log(rng, 64, 8192) // 8 * 8, _log(rng, 64, 8192) // 8 * 8, _log(rng, 33, 4099)])
    if op == "conv":
        most = (1 << 27) // channels
        more = dict(width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8, bias=rng.random() < 0.5)
    else:
        state = rng.choice([4, 8, 16, 16, 16, 24, 64])
        most = (1 << (28 if form == "backward" else 29)) // (channels * state)
        groups = rng.choice([1, 1, 2]) if channels % 2 == 0 else 1
        more = dict(state=state, groups=groups, gate=rng.random() < 0.7, skip=rng.random() < 0.7)
    if form == "token":
        return dict(case, batch=_log(rng, 1, max(2, min(512, (1 << 27) // (channels * more.get("state", 1))))), tokens=1, seqs=0, channels=channels, states=True, **more)
    tokens = _log(rng, 64, max(65, min(16384, most)))
    packed = rng.random() < 0.5
    batch = 1 if packed else rng.choice([1, 1, 2, 3, 5])
    return dict(case, batch=batch, tokens=tokens if packed else max(1, tokens // batch),
                seqs=rng.randint(1, max(1, min(64, tokens // 16))) if packed else 0, channels=channels,
                states=rng.random() < 0.5, **more)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows, back = case["batch"] * case["tokens"], case["form"] == "backward"
    if case["op"] == "rotary":
        d, heads = case["head"], case["q_heads"] + case["k_heads"]
        n = rows * heads * d
        table = min(rows, case["table"]) * case["rotary"] * 4 + rows * 4
        return {"bytes": n * (2 * e + 4) + table if back else n * 2 * e + table, "flops": n * (16 if back else 8)}
    C, seqs = case["channels"], case["seqs"] or case["batch"]
    n = rows * C
    if case["op"] == "conv":
        W = case["width"]
        states = (2 if case["states"] else 0) * seqs * (W - 1) * C * (4 if back else e)
        if back:
            return {"bytes": n * (2 * e + 4) + states + C * (W + 1) * (e + 4), "flops": n * (6 * W + 8)}
        return {"bytes": n * 2 * e + states + C * (W + 1) * e, "flops": n * (2 * W + 4)}
    N, G = case["state"], case["groups"]
    gate = 1 if case["gate"] else 0
    states = (2 if case["states"] else 1) * seqs * C * N * 4
    if back:
        # x, dt, z, dy read; dx, ddt, dz written in 32 bits; B and C read, their gradients written.
        return {"bytes": n * (e * (3 + gate) + 4 * (2 + gate)) + rows * G * N * 2 * (e + 4) + 2 * states + C * (N + 2) * 8,
                "flops": n * (N * 20 + 20)}
    return {"bytes": n * e * (3 + gate) + rows * G * N * 2 * e + states + C * (N + 2) * 4, "flops": n * (N * 7 + 10)}


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
    if case["op"] == "rotary":
        d, hq, hk, r = case["head"], case["q_heads"], case["k_heads"], case["rotary"]
        s["qkv"] = (rand(*lead, (hq + 2 * hk) * d) * 1.5).to(dt)  # one projection; v passes by
        if case["rms"]:
            s["q_weight"] = (1 + 0.2 * rand(d)).to(dt)
            s["k_weight"] = (1 + 0.2 * rand(d)).to(dt)
        freq = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        angle = torch.arange(case["table"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        first = torch.randint(0, max(1, case["table"] - T), (B, 1), generator=g, device=DEV)
        pos = ((first + torch.arange(T, device=DEV)) % case["table"]).to(torch.int32)
        s["positions"] = pos[:, 0].contiguous() if form == "token" else pos
        if form == "backward":
            s["dq_out"], s["dk_out"] = rand(*lead, hq, d).to(dt), rand(*lead, hk, d).to(dt)
        return s
    C, n_seqs = case["channels"], case["seqs"] or B
    if case["seqs"]:
        s["cu_seqlens"] = _lengths(case, seed).to(DEV)
    if case["op"] == "conv":
        W = case["width"]
        s["x"] = rand(*lead, C).to(dt)
        s["weight"] = (rand(C, W) / math.sqrt(W)).to(dt)
        s["bias"] = (0.3 * rand(C)).to(dt) if case["bias"] else None
        s["state"] = rand(n_seqs, W - 1, C).to(dt) if case["states"] else None
        if form == "backward":
            s["dy"] = rand(*lead, C).to(dt)
            s["d_final"] = rand(n_seqs, W - 1, C) if case["states"] else None
        return s
    N, G = case["state"], case["groups"]
    x = rand(*lead, C)
    s["x"] = (x * torch.sigmoid(x)).to(dt)  # what the convolution's SiLU leaves
    s["dt"] = (0.5 * rand(*lead, C)).to(dt)
    s["bc"] = rand(*lead, 2 * G * N).to(dt)  # B and C come out of one projection
    s["gate"] = rand(*lead, C).to(dt) if case["gate"] else None
    s["D"] = 1 + 0.1 * rand(C) if case["skip"] else None
    first = torch.exp(torch.rand(C, generator=g, device=DEV) * math.log(100.0)) * 1e-3  # time steps of 1e-3 to 1e-1
    s["dt_bias"] = first + torch.log(-torch.expm1(-first))
    s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(0.1 * rand(C, N))
    s["state"] = 0.5 * rand(n_seqs, C, N) if case["states"] else None
    if form == "backward":
        s["dy"] = rand(*lead, C).to(dt)
        s["d_final"] = 0.1 * rand(n_seqs, C, N) if case["states"] else None
    return s


def _views(s):
    """B and C, or q and k, out of the projection that holds them."""
    c = s["case"]
    if c["op"] == "rotary":
        d, hq, hk = c["head"], c["q_heads"], c["k_heads"]
        v = s["qkv"].unflatten(-1, (hq + 2 * hk, d))
        return v[..., :hq, :], v[..., hq:hq + hk, :]
    v = s["bc"].unflatten(-1, (2 * c["groups"], c["state"]))
    return v[..., :c["groups"], :], v[..., c["groups"]:, :]


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c["form"])


# --------------------------------------------------------------- the framework's calls ---


def _own_conv(s, form):
    kda, act = _kda(), "silu" if s["case"]["silu"] else None
    if form == "token":
        return kda.conv_decode_step(s["x"], s["weight"], s["state"], bias=s["bias"], activation=act), s["state"]
    if form == "prompt":
        return kda.conv_prefill(s["x"], s["weight"], bias=s["bias"], activation=act, cu_seqlens=s.get("cu_seqlens"),
                                initial_state=s["state"])
    g = kda.conv_backward(s["x"], s["weight"], s["dy"], bias=s["bias"], activation=act, cu_seqlens=s.get("cu_seqlens"),
                          initial_state=s["state"], d_final_state=s["d_final"])
    return [g["dx"], g["dweight"], g["dbias"], g["d_initial_state"]]


def _own_scan(s, form):
    kda = _kda()
    B, C = _views(s)
    more = dict(D=s["D"], z=s["gate"], dt_bias=s["dt_bias"], dt_softplus=True)
    if form == "token":
        return kda.scan_decode_step(s["x"], s["dt"], s["A"], B, C, s["state"], **more), s["state"]
    if form == "prompt":
        return kda.scan_prefill(s["x"], s["dt"], s["A"], B, C, cu_seqlens=s.get("cu_seqlens"), initial_state=s["state"], **more)
    g = kda.scan_backward(s["x"], s["dt"], s["A"], B, C, s["dy"], cu_seqlens=s.get("cu_seqlens"), initial_state=s["state"],
                          d_final_state=s["d_final"], **more)
    return [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state")]


def _own_rotary(s, form):
    kda, c = _kda(), s["case"]
    q, k = _views(s)
    more = dict(q_weight=s.get("q_weight"), k_weight=s.get("k_weight"), norm="rms" if c["rms"] else "l2", eps=1e-6,
                interleaved=c["interleaved"])
    if form != "backward":
        return kda.qk_norm_rotary(q, k, s["cos"], s["sin"], s["positions"], **more)
    g = kda.qk_norm_rotary_backward(q, k, s["cos"], s["sin"], s["positions"], s["dq_out"], s["dk_out"], **more)
    return [g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]]


_own = {"conv": _own_conv, "scan": _own_scan, "rotary": _own_rotary}


# ------------------------------------------------------------------------- plain forms ---


def _places(s):
    """For every row: its sequence and its place in it; for every sequence: its first row and its length."""
    c = s["case"]
    rows = torch.arange(c["batch"] * c["tokens"], device=DEV)
    if s.get("cu_seqlens") is None:
        n = torch.arange(c["batch"], device=DEV)
        return rows // c["tokens"], rows % c["tokens"], n * c["tokens"], torch.full_like(n, c["tokens"])
    cu = s["cu_seqlens"].long()
    seq = (rows[:, None] >= cu[None, 1:]).sum(1)
    return seq, rows - cu[seq], cu[:-1], cu[1:] - cu[:-1]


def _plain_conv(s, form):
    c, x, W = s["case"], s["x"], s["case"]["width"]
    w, bias, state = s["weight"].float(), s["bias"], s["state"]
    if form == "token":
        taps = torch.cat([state, x[:, None]], 1).float()
        y = (taps * w.t()).sum(1) + (0 if bias is None else bias.float())
        y = y * torch.sigmoid(y) if c["silu"] else y
        state.copy_(torch.cat([state[:, 1:], x[:, None]], 1))
        return y.to(x.dtype), state
    shape, x = x.shape, x.flatten(0, 1)
    seq, pos, first, length = _places(s)
    back = torch.arange(W, device=DEV) - (W - 1)
    old = ((pos[:, None] + back) < 0)[..., None]
    taps = x[(torch.arange(x.shape[0], device=DEV)[:, None] + back).clamp(min=0)].float()
    zero = torch.zeros((), device=DEV)
    before = zero if state is None else state[seq[:, None], (pos[:, None] + back + W - 1).clamp(max=W - 2)].float()
    taps = torch.where(old, before, taps)
    y = (taps * w.t()).sum(1) + (0 if bias is None else bias.float())
    # Places of the last W - 1 inputs of each sequence: those below 0 are in the state before it.
    ends = length[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)
    if form == "prompt":
        y = y * torch.sigmoid(y) if c["silu"] else y
        fresh = x[(first[:, None] + ends).clamp(min=0, max=x.shape[0] - 1)]
        kept = torch.zeros_like(fresh) if state is None else torch.gather(
            state, 1, (ends + W - 1).clamp(max=W - 2)[..., None].expand_as(state))
        return y.to(x.dtype).view(shape), torch.where((ends >= 0)[..., None], fresh, kept)
    dp = s["dy"].flatten(0, 1).float()
    if c["silu"]:
        sg = torch.sigmoid(y)
        dp = dp * (sg * (1 + y * (1 - sg)))
    dweight = torch.stack([(dp * taps[:, j]).sum(0, dtype=torch.float64) for j in range(W)], 1).float()
    dbias = None if bias is None else dp.sum(0, dtype=torch.float64).float()
    rows = torch.arange(x.shape[0], device=DEV)
    dx = sum(w[:, W - 1 - k] * torch.where((pos + k < length[seq])[:, None], dp[(rows + k).clamp(max=x.shape[0] - 1)], zero)
             for k in range(W))
    head = torch.arange(W - 1, device=DEV)
    dhead = torch.where((head < length[:, None])[..., None], dp[(first[:, None] + head).clamp(max=x.shape[0] - 1)], zero)
    d_init = torch.stack([sum(w[:, m - p] * dhead[:, p] for p in range(m + 1)) for m in range(W - 1)], 1)
    if s["d_final"] is not None:
        n, j = (ends >= 0).nonzero(as_tuple=True)
        dx[first[n] + ends[n, j]] += s["d_final"][n, j]
        n, j = (ends < 0).nonzero(as_tuple=True)
        d_init[n, ends[n, j] + W - 1] += s["d_final"][n, j]
    return [dx.view(shape), dweight, dbias, d_init]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _plain_scan(s, form):
    c, A = s["case"], s["A"]
    C_, N, G = c["channels"], c["state"], c["groups"]
    Bm, Cm = _views(s)
    shape, kind = s["x"].shape, s["x"].dtype
    x, raw = s["x"].reshape(-1, C_).float(), s["dt"].reshape(-1, C_).float() + s["dt_bias"]
    Bm, Cm = Bm.reshape(-1, G, 1, N).float(), Cm.reshape(-1, G, 1, N).float()
    z = None if s["gate"] is None else s["gate"].reshape(-1, C_).float()
    dt = _softplus(raw)
    a = torch.exp(dt[..., None] * A)
    b = ((dt * x).view(-1, G, C_ // G, 1) * Bm).view(-1, C_, N)

    def out(h):
        y = (h.view(-1, G, C_ // G, N) * Cm).sum(-1).view(-1, C_)
        return y if s["D"] is None else y + s["D"] * x

    if form == "token":
        s["state"].copy_(a * s["state"] + b)
        y = out(s["state"])
        return (y if z is None else y * (z * torch.sigmoid(z))).to(kind).view(shape), s["state"]
    seq, pos, first, length = _places(s)
    some = length > 0
    start, end = first[some], (first + length - 1)[some]
    init = torch.zeros(first.shape[0], C_, N, device=DEV) if s["state"] is None else s["state"]
    b[start] += a[start] * init[some]
    a0 = a.clone()
    a0[start] = 0
    h = _scan(a0, b)
    if form == "prompt":
        y = out(h)
        final = init.clone()
        final[some] = h[end]
        return (y if z is None else y * (z * torch.sigmoid(z))).to(kind).view(shape), final
    del b
    dy = s["dy"].reshape(-1, C_).float()
    dz = None
    if z is not None:
        sg = torch.sigmoid(z)
        dz = dy * out(h) * (sg * (1 + z * (1 - sg)))
        dy = dy * (z * sg)
    g = (dy.view(-1, G, C_ // G, 1) * Cm).view(-1, C_, N)
    if s["d_final"] is not None:
        g[end] += s["d_final"][some]
    g = _scan(torch.cat([a0[1:], torch.zeros_like(a0[:1])]).flip(0), g.flip(0)).flip(0)
    del a0
    dC = (dy.view(-1, G, C_ // G, 1) * h.view(-1, G, C_ // G, N)).sum(2)
    dB = (g.view(-1, G, C_ // G, N) * (dt * x).view(-1, G, C_ // G, 1)).sum(2)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[start] = init[some]
    d_init = torch.zeros_like(init) if s["d_final"] is None else s["d_final"].clone()
    d_init[some] = a[start] * g[start]
    gah = g * a * before
    gB = (g.view(-1, G, C_ // G, N) * Bm).sum(-1).view(-1, C_)
    ddt = ((gah * A).sum(-1) + gB * x) * torch.sigmoid(raw)
    dA = (gah * dt[..., None]).sum(0, dtype=torch.float64).float()
    dx = gB * dt if s["D"] is None else gB * dt + dy * s["D"]
    dD = None if s["D"] is None else (dy * x).sum(0, dtype=torch.float64).float()
    lead = shape[:-1]
    return [dx.view(shape), ddt.view(shape), dA, dB.view(*lead, G, N), dC.view(*lead, G, N), dD,
            None if dz is None else dz.view(shape), ddt.sum(0, dtype=torch.float64).float(), d_init]


def _pairs(x, rotary, interleaved):
    """The two halves of each rotated pair, and what stays as it is."""
    u, rest = x[..., :rotary], x[..., rotary:]
    return (u[..., 0::2], u[..., 1::2], rest) if interleaved else (u[..., :rotary // 2], u[..., rotary // 2:], rest)


def _joined(u, v, rest, interleaved):
    w = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([w, rest], -1)


def _plain_rotary(s, form):
    c = s["case"]
    cos, sin = (s[k][s["positions"].long()][..., None, :] for k in ("cos", "sin"))
    outs, grads, weights = [], [], []
    for x, weight, d_out in zip(_views(s), (s.get("q_weight"), s.get("k_weight")), (s.get("dq_out"), s.get("dk_out"))):
        kind, x = x.dtype, x.float()
        w = torch.ones(c["head"], device=DEV) if weight is None else weight.float()
        scale = c["head"] if c["rms"] else 1
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / scale + 1e-6)
        if form != "backward":
            u, v, rest = _pairs(x * r * w, c["rotary"], c["interleaved"])
            outs.append(_joined(u * cos - v * sin, v * cos + u * sin, rest, c["interleaved"]).to(kind))
            continue
        u, v, rest = _pairs(d_out.float(), c["rotary"], c["interleaved"])
        d = _joined(u * cos + v * sin, v * cos - u * sin, rest, c["interleaved"])
        weights.append(None if weight is None else (d * (x * r)).flatten(0, -2).sum(0, dtype=torch.float64).float())
        d = d * w
        grads.append(r * (d - x * (r * r * (d * x).sum(-1, keepdim=True) / scale)))
    return tuple(outs) if form != "backward" else grads + weights


_plain = {"conv": _plain_conv, "scan": _plain_scan, "rotary": _plain_rotary}


# --------------------------------------------------------------------- in 64 bits ---------


def _bounds(s):
    c = s["case"]
    if s.get("cu_seqlens") is not None:
        cu = s["cu_seqlens"].tolist()
        return list(zip(cu[:-1], cu[1:]))
    return [(n * c["tokens"], (n + 1) * c["tokens"]) for n in range(c["batch"])]


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "rotary": _exact_rotary}[case["op"]](s, case["form"])


def _exact_conv(s, form):
    c, W = s["case"], s["case"]["width"]
    x = s["x"].reshape(-1, c["channels"]).double()
    w, bias = s["weight"].double(), 0.0 if s["bias"] is None else s["bias"].double()
    old = torch.zeros(c["seqs"] or c["batch"], W - 1, c["channels"], device=DEV, dtype=torch.float64)
    old = old if s["state"] is None else s["state"].double()
    y, final, d_init, dx = torch.empty_like(x), torch.empty_like(old), torch.empty_like(old), torch.empty_like(x)
    dw, db = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for n, (lo, hi) in enumerate(_bounds(s)):
        line = torch.cat([old[n], x[lo:hi]])  # the inputs of the sequence behind its state
        p = bias + sum(w[:, j] * line[j:j + hi - lo] for j in range(W))
        final[n] = line[line.shape[0] - (W - 1):]
        if form != "backward":
            y[lo:hi] = p / (1 + torch.exp(-p)) if c["silu"] else p
            continue
        d = s["dy"].reshape(-1, c["channels"])[lo:hi].double()
        if c["silu"]:
            e = 1 / (1 + torch.exp(-p))
            d = d * (e + p * e * (1 - e))
        dline = torch.zeros_like(line)
        for j in range(W):
            dline[j:j + hi - lo] += w[:, j] * d
            dw[:, j] += (d * line[j:j + hi - lo]).sum(0)
        db += d.sum(0)
        if s["d_final"] is not None:
            dline[line.shape[0] - (W - 1):] += s["d_final"][n]
        d_init[n], dx[lo:hi] = dline[:W - 1], dline[W - 1:]
    if form != "backward":
        return y.view(s["x"].shape), final
    return [dx.view(s["x"].shape), dw, None if s["bias"] is None else db, d_init]


def _exact_scan(s, form):
    c = s["case"]
    C_, N, G = c["channels"], c["state"], c["groups"]
    Bm, Cm = (v.reshape(-1, G, N).double() for v in _views(s))
    x = s["x"].reshape(-1, C_).double()
    raw = s["dt"].reshape(-1, C_).double() + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    A, skip = s["A"].double(), 0.0 if s["D"] is None else s["D"].double()
    bounds = _bounds(s)
    order = sorted(range(len(bounds)), key=lambda n: bounds[n][0] - bounds[n][1])  # longest first
    lo = torch.tensor([bounds[n][0] for n in order], device=DEV)
    lens = [bounds[n][1] - bounds[n][0] for n in order]
    live, k = [], len(lens)  # how many sequences still run at each step
    for t in range(max(lens)):
        while lens[k - 1] <= t:
            k -= 1
        live.append(k)
    n = len(order)
    h = torch.zeros(n, C_, N, device=DEV, dtype=torch.float64) if s["state"] is None else s["state"][order].double()
    h0, per = h.clone(), C_ // G
    back = form == "backward"
    kept = torch.empty(x.shape[0], C_, N, device=DEV, dtype=torch.float64) if back else None
    y = torch.empty_like(x)

    def wide(v):  # [k, G, N] over the channels of each group
        return v.repeat_interleave(per, 1)

    for t, k in enumerate(live):
        at = lo[:k] + t
        h[:k] = torch.exp(dt[at][..., None] * A) * h[:k] + (dt[at] * x[at])[..., None] * wide(Bm[at])
        y[at] = (h[:k] * wide(Cm[at])).sum(-1) + skip * x[at]
        if back:
            kept[at] = h[:k]
    z = None if s["gate"] is None else s["gate"].reshape(-1, C_).double()
    e = None if z is None else 1 / (1 + torch.exp(-z))
    there = torch.tensor(order, device=DEV)
    if not back:
        final = torch.empty_like(h)
        final[there] = h
        return (y if z is None else y * z * e).view(s["x"].shape), final
    dy = s["dy"].reshape(-1, C_).double()
    dz = None if z is None else dy * y * (e + z * e * (1 - e))
    dy = dy if z is None else dy * z * e
    g = torch.zeros_like(h) if s["d_final"] is None else s["d_final"][order].double()
    dx, ddt, dA = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(A)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    for t, k in reversed(list(enumerate(live))):
        at = lo[:k] + t
        g[:k] += dy[at][..., None] * wide(Cm[at])
        a = torch.exp(dt[at][..., None] * A)
        p = h0[:k] if t == 0 else kept[at - 1]
        dC[at] = (dy[at][..., None] * kept[at]).view(k, G, per, N).sum(2)
        dB[at] = (g[:k] * (dt[at] * x[at])[..., None]).view(k, G, per, N).sum(2)
        gb, gap = (g[:k] * wide(Bm[at])).sum(-1), g[:k] * a * p
        dx[at] = gb * dt[at] + dy[at] * skip
        ddt[at] = (gb * x[at] + (gap * A).sum(-1)) / (1 + torch.exp(-raw[at]))
        dA += (gap * dt[at][..., None]).sum(0)
        g[:k] = g[:k] * a
    d_init = torch.empty_like(g)
    d_init[there] = g
    lead = s["x"].shape[:-1]
    return [dx.view(s["x"].shape), ddt.view(s["x"].shape), dA, dB.view(*lead, G, N), dC.view(*lead, G, N),
            None if s["D"] is None else (dy * x).sum(0), None if dz is None else dz.view(s["x"].shape), ddt.sum(0), d_init]


def _exact_rotary(s, form):
    c, r = s["case"], s["case"]["rotary"]
    at = s["positions"].long()
    turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[..., None, :]
    ones = torch.ones(c["head"], device=DEV, dtype=torch.float64)

    def rotated(v, by):
        u = v[..., :r]
        z = torch.view_as_complex(u.unflatten(-1, (-1, 2)).contiguous()) if c["interleaved"] else torch.complex(
            u[..., :r // 2].contiguous(), u[..., r // 2:].contiguous())
        z = torch.view_as_real(z * by)
        u = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([u, v[..., r:]], -1)

    grads, weights, outs = [], [], []
    for x, weight, d in zip(_views(s), (s.get("q_weight"), s.get("k_weight")), (s.get("dq_out"), s.get("dk_out"))):
        x, w = x.double(), ones if weight is None else weight.double()
        size = torch.sqrt((x.square().mean(-1, keepdim=True) if c["rms"] else x.square().sum(-1, keepdim=True)) + 1e-6)
        if form != "backward":
            outs.append(rotated(x / size * w, turn))
            continue
        d = rotated(d.double(), turn.conj())
        weights.append(None if weight is None else (d * x / size).flatten(0, -2).sum(0))
        d = d * w
        mean = (d * x).mean(-1, keepdim=True) if c["rms"] else (d * x).sum(-1, keepdim=True)
        grads.append(d / size - x * mean / size ** 3)
    return tuple(outs) if form != "backward" else grads + weights
