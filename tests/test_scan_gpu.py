"""The selective state space scan on the GPU against its definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda

import layers_ref as ref
from layers_cases import DEV, HALF, ULP32, close, cu_of, d64, gen, near, strided

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, dtype, B, T, D, N, G=1, lengths=None, gate=True, skip=True, bias=True, softplus=True, states=True, seed=0,
                 slow=False):
        r = gen(seed)
        if lengths is not None:
            B, T = 1, sum(lengths)
        self.shape, self.n = (B, T, D, N, G), B if lengths is None else len(lengths)
        self.cu = None if lengths is None else cu_of(lengths)
        self.x, self.z = r(B, T, D).to(dtype), r(B, T, D).to(dtype) if gate else None
        self.dt = (0.5 * r(B, T, D) if softplus else 0.05 * r(B, T, D).abs()).to(dtype)
        self.B, self.C = r(B, T, G, N).to(dtype), r(B, T, G, N).to(dtype)
        self.A = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(0.1 * r(D, N)) * (0.01 if slow else 1)
        self.D, self.dt_bias = r(D) if skip else None, (r(D) - 3 if softplus else 0.05 * r(D).abs()) if bias else None
        self.softplus, self.state = softplus, r(self.n, D, N) if states else None
        self.dy, self.d_final = r(B, T, D).to(dtype), r(self.n, D, N) if states else None
        self.dtype = dtype

    def options(self):
        return dict(D=self.D, z=self.z, dt_bias=self.dt_bias, dt_softplus=self.softplus)

    def prefill(self, **kw):
        args = dict(cu_seqlens=self.cu, initial_state=self.state, **self.options())
        args.update(kw)
        return kda.scan_prefill(self.x, self.dt, self.A, self.B, self.C, **args)

    def backward(self, **kw):
        args = dict(cu_seqlens=self.cu, initial_state=self.state, d_final_state=self.d_final, **self.options())
        args.update(kw)
        return kda.scan_backward(self.x, self.dt, self.A, self.B, self.C, self.dy, **args)

    def sequences(self):
        """The reference's arguments for every sequence."""
        B, T, D, N, G = self.shape
        wide = [d64(t).reshape(-1, G, N).repeat_interleave(D // G, 1) for t in (self.B, self.C)]
        flat = [d64(t).reshape(-1, D) for t in (self.x, self.dt, self.dy)]
        z = None if self.z is None else d64(self.z).reshape(-1, D)
        raw = flat[1] if self.dt_bias is None else flat[1] + d64(self.dt_bias)
        for i, (lo, hi) in enumerate(ref.spans(B, T, None if self.cu is None else self.cu.cpu())):
            zero = torch.zeros(D, N, dtype=torch.float64)
            yield dict(x=flat[0][lo:hi], dt=raw[lo:hi], A=d64(self.A), B=wide[0][lo:hi], C=wide[1][lo:hi], D=d64(self.D),
                       z=None if z is None else z[lo:hi], softplus=self.softplus, init=zero if self.state is None else d64(self.state)[i]), \
                flat[2][lo:hi], zero if self.d_final is None else d64(self.d_final)[i]

    def check_prefill(self, y, fin):
        D, T = self.shape[2], max(s["x"].shape[0] for s, _, _ in self.sequences())
        ys, fins, mags, hmags = [], [], [], []
        for s, _, _ in self.sequences():
            a = ref.scan(**s)
            positive = {k: None if s[k] is None else s[k].abs() for k in ("x", "B", "C", "D", "init")}
            m = ref.scan(**{**s, **positive, "z": None})
            gate = 1 if s["z"] is None else ref.silu(s["z"]).abs()
            ys.append(a[0])
            fins.append(a[1])
            mags.append(m[0] * gate)
            hmags.append(m[1])
        y_ref, mag = torch.cat(ys), torch.cat(mags)
        # One rounding of the output. In fp32 every step of the state rounds its decay (the step's time, its product with
        # A, the exponential: 6 half steps) and its sum (2), so a term that lived for t tokens is off by at most
        # 8 t half steps; 64 for the time step's own function, the products around it, the sum over the states and the gate.
        tol = (8 * T + 64) * ULP32
        close("y", y.reshape(-1, D), y_ref, HALF[self.dtype] * 1.001 * y_ref.abs() + tol * mag + 1e-30)
        if fin is not None:
            close("final_state", fin, torch.stack(fins), tol * torch.stack(hmags) + 1e-30)


SHAPES = [  # B, T, D, N, G, lengths
    (1, 1, 8, 16, 1, None), (2, 3, 5, 1, 1, None), (3, 70, 40, 4, 2, None), (2, 130, 72, 16, 1, None), (1, 300, 33, 24, 3, None),
    (1, 50, 6, 100, 1, None), (1, 20, 4, 256, 2, None), (2, 65, 7, 7, 7, None), (1, 0, 40, 16, 1, [3, 0, 1, 70, 2, 290]),
    (1, 0, 24, 8, 2, [0, 2, 40, 0]), (1, 0, 130, 16, 1, [1, 1, 1, 0, 1])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts(dtype, shape):
    B, T, D, N, G, lengths = shape
    c = Case(dtype, B, T, D, N, G, lengths, seed=1)
    c.check_prefill(*c.prefill())
    kda.check_status()


@pytest.mark.parametrize("off", ["gate", "skip", "bias", "softplus", "states"])
def test_each_option_left_out(off):
    c = Case(torch.float32, 2, 75, 40, 16, 1, None, seed=2, **{off: False})
    c.check_prefill(*c.prefill())
    _check_backward(c)


def _check_backward(c):
    g = c.backward()
    kda.check_status()
    B, T, D, N, G = c.shape
    want = [ref.scan_backward(**s, dy=dy, d_final=df) for s, dy, df in c.sequences()]
    longest = max(s["x"].shape[0] for s, _, _ in c.sequences())
    # As for prompts, doubled: the states and their gradients both carry it; sums of terms of both signs lose up to a
    # small factor against their absolute sum, 4.
    tol = 4 * 2 * (8 * min(longest, 64) + 64) * ULP32
    per = lambda k: torch.cat([w[k] for w in want])  # noqa: E731
    near("dx", g["dx"].reshape(-1, D), per("dx"), tol)
    near("ddt", g["ddt"].reshape(-1, D), per("ddt"), tol)
    for k in ("dB", "dC"):
        near(k, g[k].reshape(-1, G, N), per(k).reshape(-1, G, D // G, N).sum(2), tol)
    near("dA", g["dA"], sum(w["dA"] for w in want), tol)
    near("d_initial_state", g["d_initial_state"], torch.stack([w["d_init"] for w in want]), tol)
    if c.D is not None:
        near("dD", g["dD"], sum(w["dD"] for w in want), tol)
    if c.z is not None:
        near("dz", g["dz"].reshape(-1, D), per("dz"), tol)
    if c.dt_bias is not None:
        near("ddt_bias", g["ddt_bias"], per("ddt").sum(0), tol)
    assert (g["dD"] is None) == (c.D is None) and (g["dz"] is None) == (c.z is None)
    again = c.backward()
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None), "the same bits every time"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(dtype, shape):
    B, T, D, N, G, lengths = shape
    _check_backward(Case(dtype, B, T, D, N, G, lengths, seed=3))


@pytest.mark.parametrize("B,T,D,lengths", [(1, 2500, 64, None), (2, 1100, 48, None), (1, 0, 40, [700, 1, 0, 1500, 64, 90])])
def test_long_prompts_are_cut_along_the_sequence(B, T, D, lengths):
    """Few channels and many tokens: the call is split along the rows, with the carries joined."""
    c = Case(torch.float32, B, T, D, 16, 1, lengths, seed=4, slow=True)
    c.check_prefill(*c.prefill())
    c = Case(torch.float32, B, T, D, 16, 1, lengths, seed=5)
    _check_backward(c)


def test_strided_rows():
    for dtype, pads in ((torch.bfloat16, ((8, 8), (3, 1))), (torch.float32, ((4, 4), (5, 3)))):
        c = Case(dtype, 2, 45, 48, 16, 2, seed=6)
        y, fin = c.prefill()
        g = c.backward()
        for pad, offset in pads:
            v = Case(dtype, 2, 45, 48, 16, 2, seed=6)
            v.x, v.dt, v.z, v.B, v.C = (strided(t, 2, pad, offset) for t in (c.x, c.dt, c.z, c.B, c.C))
            y2, fin2 = v.prefill()
            assert torch.equal(y, y2) and torch.equal(fin, fin2)
            g2 = v.backward()
            assert all(torch.equal(g[k], g2[k]) for k in g)
            first = [t[:, 0] for t in (v.x, v.dt, v.B, v.C, v.z)]
            dense = [t.contiguous() for t in first]
            s1, s2 = c.state.clone(), c.state.clone()
            one = [kda.scan_decode_step(f[0], f[1], c.A, f[2], f[3], s, D=c.D, z=f[4], dt_bias=c.dt_bias)
                   for f, s in ((first, s1), (dense, s2))]
            assert torch.equal(*one) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype,D,N,G", [(torch.bfloat16, 72, 16, 1), (torch.float32, 13, 7, 1), (torch.bfloat16, 6, 100, 2),
                                         (torch.float32, 40, 4, 4), (torch.bfloat16, 8, 256, 1), (torch.float32, 24, 1, 1)])
def test_prefill_then_tokens(dtype, D, N, G):
    T, more, B = 21, 5, 3
    c = Case(dtype, B, T + more, D, N, G, seed=7)
    y, fin = c.prefill()
    head = {k: getattr(c, k)[:, :T].contiguous() for k in ("x", "dt", "B", "C", "z")}
    y1, st = kda.scan_prefill(head["x"], head["dt"], c.A, head["B"], head["C"], D=c.D, z=head["z"], dt_bias=c.dt_bias, initial_state=c.state)
    pool = torch.zeros(B + 1, D, N, device=DEV)
    idx = torch.tensor([3, 0, 2], dtype=torch.int32, device=DEV)
    pool[idx.long()] = st
    ys = [y1]
    for t in range(T, T + more):
        at = {k: getattr(c, k)[:, t].contiguous() for k in ("x", "dt", "B", "C", "z")}
        more_args = dict(D=c.D, z=at["z"], dt_bias=c.dt_bias)
        ys.append(kda.scan_decode_step(at["x"], at["dt"], c.A, at["B"], at["C"], st, **more_args)[:, None])
        yp = kda.scan_decode_step(at["x"], at["dt"], c.A, at["B"], at["C"], pool, state_indices=idx, **more_args)
        assert torch.equal(yp, ys[-1][:, 0])
    assert torch.equal(pool[idx.long()], st) and not pool[1].any()
    c.check_prefill(torch.cat(ys, 1), st)
    # branching, and a sequence without a slot
    frm, to = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([3, 0, -1], [1, -1, 2]))
    before = pool.clone()
    yb = kda.scan_decode_step(at["x"], at["dt"], c.A, at["B"], at["C"], pool, state_indices=frm, final_state_indices=to, **more_args)
    start = torch.stack([before[3], before[0], torch.zeros_like(before[0])])
    want = kda.scan_decode_step(at["x"], at["dt"], c.A, at["B"], at["C"], start, **more_args)
    kda.check_status()
    assert torch.equal(yb, want)
    before[1], before[2] = start[0], start[2]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("lengths", [[5, 1, 0, 2, 130], [700, 0, 90]])
def test_pools_in_place(lengths):
    n = len(lengths)
    c = Case(torch.float32, 1, 0, 40, 16, 1, lengths, seed=8)
    pool = gen(9)(n + 2, 40, 16)
    slots = torch.randperm(n + 2)[:n]
    pool[slots.to(DEV)] = c.state
    slots[1] = -1
    c.state[1] = 0
    y, fin = c.prefill()
    kept = pool.clone()
    for i in range(n):
        if slots[i] >= 0:
            kept[slots[i]] = fin[i]
    idx = slots.to(torch.int32).to(DEV)
    y2, out = c.prefill(initial_state=pool, final_state=pool, initial_state_indices=idx, final_state_indices=idx)
    kda.check_status()
    assert out is pool and torch.equal(y, y2) and torch.equal(pool, kept)


def test_no_rows():
    c = Case(torch.float32, 2, 0, 8, 16, seed=10)
    y, fin = c.prefill()
    assert y.shape == (2, 0, 8) and torch.equal(fin, c.state)
    g = c.backward()
    kda.check_status()
    assert torch.equal(g["d_initial_state"], c.d_final) and not g["dA"].any() and not g["dD"].any()


def test_large_time_steps_forget_and_growth_stays_exact():
    """Decays that underflow to 0, time steps past the softplus's linear end, and a positive A."""
    c = Case(torch.float32, 1, 60, 24, 16, seed=11)
    c.dt_bias = torch.linspace(-30, 80, 24, device=DEV)
    c.check_prefill(*c.prefill())
    _check_backward(c)
    c = Case(torch.float32, 1, 40, 24, 16, seed=12, bias=True)
    c.A = 0.1 * c.A.abs()
    c.check_prefill(*c.prefill())


def test_infinities_and_nan_stay_in_their_channel():
    c = Case(torch.float32, 1, 40, 48, 16, seed=13)
    clean, _ = c.prefill()
    c.x[0, 5, 3], c.x[0, 9, 7] = float("nan"), float("inf")
    y, _ = c.prefill()
    hit = torch.zeros(40, 48, dtype=torch.bool, device=DEV)
    hit[5:, 3], hit[9:, 7] = True, True
    assert torch.equal(y[0][~hit], clean[0][~hit]) and torch.isnan(y[0, 5:, 3]).all()


def test_a_bad_cu_seqlens_and_a_bad_slot_are_reported():
    for cu in ([0, 12, 8, 20], [0, 25, 30, 20], [3, 5, 9, 20], [0, 4, 9, 19], [0, -5, 9, 20]):
        c = Case(torch.bfloat16, 1, 0, 16, 16, 1, [10, 5, 5], seed=14)
        c.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        c.prefill()
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_status()
        c.backward()
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_status()
    c = Case(torch.bfloat16, 1, 1, 16, 16, seed=15)
    pool = torch.zeros(2, 16, 16, device=DEV)
    bad = torch.tensor([2], dtype=torch.int32, device=DEV)
    kda.scan_decode_step(c.x[:, 0], c.dt[:, 0], c.A, c.B[:, 0], c.C[:, 0], pool, state_indices=bad)
    with pytest.raises(kda.KDAError, match="pool"):
        kda.check_status()
    assert not pool.any()


def test_another_stream_and_a_captured_graph():
    c = Case(torch.bfloat16, 1, 1500, 64, 16, seed=16)
    y, fin = c.prefill()
    g = c.backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, fin2 = c.prefill()
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, fin3 = c.prefill()
        g3 = c.backward()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, y) and torch.equal(fin3, fin) and all(torch.equal(g3[k], g[k]) for k in g)
    kda.check_status()


@pytest.mark.parametrize("dtype,D,N,G", [(torch.bfloat16, 64, 16, 1), (torch.float32, 64, 16, 2), (torch.bfloat16, 64, 4, 1),
                                         (torch.float32, 32, 8, 1), (torch.bfloat16, 48, 32, 1), (torch.bfloat16, 32, 64, 2),
                                         (torch.float32, 96, 12, 1), (torch.bfloat16, 128, 16, 4), (torch.float32, 64, 52, 1)])
def test_tokens_of_whole_warps(dtype, D, N, G):
    """Channels in whole warps: the form of the token step that streams the states of many sequences."""
    test_prefill_then_tokens(dtype, D, N, G)


@pytest.mark.parametrize("n", [1, 2, 69, 200])
@pytest.mark.parametrize("off", ["", "gate", "skip", "bias", "softplus"])
def test_many_sequences_take_one_token(n, off):
    c = Case(torch.float32, n, 1, 64, 16, 1, seed=17, **({off: False} if off else {}))
    pool = torch.zeros(n + 5, 64, 16, device=DEV)
    slots = torch.randperm(n + 5)[:n].to(torch.int32).to(DEV)
    pool[slots.long()] = c.state
    args = [t[:, 0] for t in (c.x, c.dt)], [t[:, 0] for t in (c.B, c.C)]
    more = dict(D=c.D, z=None if c.z is None else c.z[:, 0], dt_bias=c.dt_bias, dt_softplus=c.softplus)
    y = kda.scan_decode_step(*args[0], c.A, *args[1], pool, state_indices=slots, **more)
    kda.check_status()
    c.check_prefill(y, pool[slots.long()])
