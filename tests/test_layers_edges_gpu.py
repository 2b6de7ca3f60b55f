"""The operators around the mixer on the GPU at the ends of their ranges."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers

import layers_ref as ref
from layers_cases import DEV, HALF, ULP32, close, cu_of, d64, gen, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["qk", "q", "k"])
def test_weight_gradients_over_no_rows_are_zeros(which):
    q, w = torch.empty(0, 2, 64, device=DEV), torch.ones(64, device=DEV)
    weights = dict(q_weight=w if "q" in which else None, k_weight=w if "k" in which else None)
    # The library's own call, on outputs that hold NaN; its workspace has no bytes here, so it may be NULL.
    a, dev = layers._rotary_args(q, q, None, None, None, weights["q_weight"], weights["k_weight"], "rms", 1e-6, False)
    out = [torch.full((64,), float("nan"), device=DEV) if n in which else None for n in "qk"]
    layers._call(dev, layers._library().kda_qk_norm_rotary_backward, a, 0, 0, 0, 0, *map(layers._address, out), 0, 0)
    assert all(t is None or not t.any() for t in out)
    # The binding's, whose outputs come from memory that held NaN.
    del out
    poison = [torch.full((64,), float("nan"), device=DEV) for _ in range(64)]
    del poison
    g = kda.qk_norm_rotary_backward(q, q, None, None, None, q, q, **weights)
    kda.check_status()
    for n in "qk":
        assert g[f"d{n}_weight"] is None if n not in which else not g[f"d{n}_weight"].any()


def test_a_bad_cu_seqlens_over_no_rows_is_reported():
    x, w = torch.empty(1, 0, 8, device=DEV), torch.ones(8, 4, device=DEV)
    B, A = torch.empty(1, 0, 1, 4, device=DEV), -torch.ones(8, 4, device=DEV)
    pool = torch.ones(2, 3, 8, device=DEV)
    calls = [lambda cu: kda.conv_prefill(x, w, cu_seqlens=cu), lambda cu: kda.conv_prefill(x, w, cu_seqlens=cu, output_final_state=False),
             lambda cu: kda.conv_prefill(x, w, cu_seqlens=cu, initial_state=pool[:cu.numel() - 1], final_state=pool[:cu.numel() - 1]),
             lambda cu: kda.conv_backward(x, w, x, cu_seqlens=cu),
             lambda cu: kda.conv_backward(x, w, x, cu_seqlens=cu, want_d_initial_state=False),
             lambda cu: kda.scan_prefill(x, x, A, B, B, cu_seqlens=cu), lambda cu: kda.scan_backward(x, x, A, B, B, x, cu_seqlens=cu),
             lambda cu: kda.scan_backward(x, x, A, B, B, x, cu_seqlens=cu, want_d_initial_state=False)]
    for i, call in enumerate(calls):
        for bad in ([0, 5], [3], [0, 2, 0]):
            call(torch.tensor(bad, dtype=torch.int32, device=DEV))
            with pytest.raises(kda.KDAError, match="cu_seqlens"):
                kda.check_status()
                raise AssertionError((i, bad))
        for good in ([0], [0, 0], [0, 0, 0]):
            call(torch.tensor(good, dtype=torch.int32, device=DEV))
            kda.check_status()
    assert torch.equal(pool, torch.ones_like(pool))


def test_an_empty_prompt_reads_only_its_states():
    """No rows: the C call needs neither the rows' inputs nor A."""
    s, out = gen(1)(2, 8, 16), torch.full((2, 8, 16), float("nan"), device=DEV)
    a = layers._scan_struct(1, 2, 0, 8, 16, 1, 1, *[0] * 5, *[0] * 5, 0, 0, 0, 0, 0, s.data_ptr(), 0, 0, 0)
    layers._call(s.device, layers._library().kda_scan_prefill, a, 0, out.data_ptr(), 0, 0)
    kda.check_status()
    assert torch.equal(out, s)
    x, B, A = torch.empty(1, 0, 8, device=DEV), torch.empty(1, 0, 1, 16, device=DEV), -torch.ones(8, 16, device=DEV)
    cu, pool = cu_of([0, 0, 0]), gen(2)(5, 8, 16)
    frm, to = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([4, -1, 0], [1, 3, -1]))
    want = pool.clone()
    want[1], want[3] = pool[4], 0
    kda.scan_prefill(x, x, A, B, B, cu_seqlens=cu, initial_state=pool, final_state=pool, initial_state_indices=frm, final_state_indices=to)
    kda.check_status()
    assert torch.equal(pool, want)
    frm[0] = 5
    y, fin = kda.scan_prefill(x, x, A, B, B, cu_seqlens=cu, initial_state=pool, initial_state_indices=frm)
    with pytest.raises(kda.KDAError, match="pool"):
        kda.check_status()
    assert not fin[:2].any() and torch.equal(fin[2], pool[0])


def test_sums_past_the_largest_fp32_are_infinite():
    """Weight gradients whose parts overflow: the infinity that the sum rounds to, as for any other sum, and not NaN."""
    inf, big = float("inf"), 3e38
    x, w, dy = torch.ones(1, 700, 8, device=DEV), torch.zeros(8, 4, device=DEV), torch.zeros(1, 700, 8, device=DEV)
    dy[0, 10:14, 2] = big     # in one thread's run
    dy[0, ::300, 5] = -big    # in several blocks' parts
    g = kda.conv_backward(x, w, dy, torch.zeros(8, device=DEV), activation=None)
    want = torch.zeros(8, device=DEV)
    want[2], want[5] = inf, -inf
    assert torch.equal(g["dbias"], want) and torch.equal(g["dweight"], want[:, None].expand(8, 4)) and not g["dx"].any()
    zero = torch.zeros(1, 700, 1, 4, device=DEV)
    g = kda.scan_backward(x, x, -torch.ones(8, 4, device=DEV), zero, zero, dy, D=torch.zeros(8, device=DEV), dt_softplus=False)
    assert torch.equal(g["dD"], want) and not g["dA"].any() and not g["dx"].any()
    q, d = torch.ones(700, 1, 8, device=DEV), dy.view(700, 1, 8)
    g = kda.qk_norm_rotary_backward(q, q, None, None, None, d, d * 0, q_weight=torch.zeros(8, device=DEV), k_weight=torch.zeros(8, device=DEV))
    kda.check_status()
    assert torch.equal(g["dq_weight"], want) and not g["dk_weight"].any()
    dy[0, 20, 3], dy[0, 600, 3] = inf, -inf
    g = kda.conv_backward(x, w, dy, torch.zeros(8, device=DEV), activation=None)
    assert torch.isnan(g["dbias"][3]) and g["dbias"][5] == -inf


def _growing(lengths, at, rate, n):
    """Packed sequences whose state grows by exp(rate) a row in the sequence `at` and hardly changes in the others."""
    r, T, D = gen(2), sum(lengths), 8
    lo, hi = ref.spans(1, T, cu_of(lengths).cpu())[at]
    dt = torch.full((1, T, D), 2.0 ** -10, device=DEV)
    dt[:, lo:hi] = rate
    return torch.zeros(1, T, D, device=DEV), dt, torch.ones(D, n, device=DEV), r(1, T, 1, n), r(1, T, 1, n), lo, hi


# 15 rows that are not its own, then chunks of 16 rows: the second sequence has one row before a whole chunk and one behind it.
@pytest.mark.parametrize("lengths", [[15, 18, 15], [15, 18, 400]])
@pytest.mark.parametrize("n", [4, 24])
def test_states_that_grow_across_a_chunk(lengths, n):
    """exp(A sum dt) over a chunk may pass fp32's range where the state after it does not."""
    x, dt, A, B, C, lo, hi = _growing(lengths, 1, 6.0, n)
    cu = cu_of(lengths)
    y, fin = kda.scan_prefill(x, dt, A, B, C, dt_softplus=False, cu_seqlens=cu)
    assert not y.any() and not fin.any()  # zeros stay zeros
    init = gen(3)(len(lengths), 8, n) * 2.0 ** -100
    y, fin = kda.scan_prefill(x, dt, A, B, C, dt_softplus=False, cu_seqlens=cu, initial_state=init)
    kda.check_status()
    a = ref.scan(d64(x)[0, lo:hi], d64(dt)[0, lo:hi], d64(A), *(d64(t)[0, lo:hi].expand(-1, 8, -1) for t in (B, C)), None, None, False,
                 d64(init)[1])
    # Each row's exponent, |dt A| log2(e) = 9 at most, takes three roundings (A log2(e), the product, the instruction's argument) of 9 half
    # steps each, and the decay and the state 6 more: rows * (3 * 9 + 6) half steps, and over a chunk the same in one exponent.
    tol = (hi - lo) * (3 * 9 + 6) * ULP32
    close("final_state", fin[1], a[1], tol * a[1].abs())
    mag = ref.scan(d64(x)[0, lo:hi], d64(dt)[0, lo:hi], d64(A), *(d64(t)[0, lo:hi].abs().expand(-1, 8, -1) for t in (B, C)), None, None, False,
                   d64(init)[1].abs())[0]
    close("y", y[0, lo:hi], a[0], (tol + 64 * ULP32) * mag)


def test_gradients_of_states_that_grow_across_a_chunk():
    # Chunks of 64 rows; 2.2 a row are 2^203 over a chunk.
    x, dt, A, B, C, lo, hi = _growing([63, 66, 127], 1, 2.2, 4)
    cu, dy = cu_of([63, 66, 127]), torch.zeros_like(x)
    g = kda.scan_backward(x, dt, A, B, C, dy, dt_softplus=False, cu_seqlens=cu)
    assert all(t is None or not t.any() for t in g.values())  # zeros stay zeros
    init, df = (gen(s)(3, 8, 4) * 2.0 ** -100 for s in (4, 5))
    g = kda.scan_backward(x, dt, A, B, C, dy, dt_softplus=False, cu_seqlens=cu, initial_state=init, d_final_state=df)
    kda.check_status()
    wide = [d64(t)[0, lo:hi].expand(-1, 8, -1) for t in (B, C)]
    a = ref.scan_backward(d64(x)[0, lo:hi], d64(dt)[0, lo:hi], d64(A), *wide, None, None, False, d64(init)[1], d64(dy)[0, lo:hi], d64(df)[1])
    # As above with exponents of 3.2, for the states and for their gradients; 4 for sums of both signs.
    tol = 4 * 2 * (hi - lo) * (3 * 3.2 + 6) * ULP32
    near("d_initial_state", g["d_initial_state"][1], a["d_init"], tol)
    for k in ("dx", "ddt"):
        near(k, g[k][0, lo:hi], a[k], tol)
    assert torch.isfinite(g["dA"]).all()


def _pool(states, spare, seed):
    """A pool with the states in slots of any order, two sequences without one (zeros, nothing written), and the slots."""
    n = states.shape[0]
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(n + spare, generator=g)[:n].to(torch.int32).to(DEV)
    pool = gen(seed)(n + spare, *states.shape[1:]).to(states.dtype)
    pool[slots.long()] = states
    slots[n // 3], slots[n - 1] = -1, -1
    states[n // 3], states[n - 1] = 0, 0
    return pool, slots


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,D,N", [(511, 8192, 4), (257, 4096, 16), (129, 512, 64), (301, 96, 80), (65, 52, 130)])
def test_tokens_of_many_sequences_and_channels(dtype, n, D, N):
    """Warps that walk over more than 32 sequences each, and the form for sizes that do not fill warps."""
    r = gen(6)
    x, dt, z, B, C = (r(*s).to(dtype) for s in ((n, D), (n, D), (n, D), (n, 1, N), (n, 1, N)))
    A, skip, bias, s = -torch.rand(D, N, device=DEV) * 4, r(D), r(D) - 2, r(n, D, N)
    pool, slots = _pool(s, 3, 7)
    want_pool, s = pool.clone(), s.double()
    y = kda.scan_decode_step(x, dt, A, B, C, pool, D=skip, z=z, dt_bias=bias, state_indices=slots)
    kda.check_status()
    x, dt, z, B, C = (t.double() for t in (x, dt, z, B, C))
    step = ref.time_step(dt + bias.double(), True)
    u = (step * x)[..., None] * B
    h = torch.exp(step[..., None] * A.double()) * s + u
    # One token: the exponent |dt' A| log2(e) in three roundings and the time step's own 4, then 8 for the state; the output rounds once, after
    # 64 for the products around it and the gate and N for the sum over the states.
    mag = (4 * 1.45 * step[..., None] * A.double().abs() + 8) * torch.exp(step[..., None] * A.double()) * s.abs() + 16 * u.abs()
    want = ((h * C).sum(-1) + skip.double() * x) * ref.silu(z)
    size = (mag * C.abs()).sum(-1) + (64 + N) * (((h * C).abs()).sum(-1) + (skip.double() * x).abs())
    close("y", y, want.cpu(), (HALF[dtype] * 1.001 * want.abs() + ULP32 * size * ref.silu(z).abs() + 1e-30).cpu())
    used = slots >= 0
    close("state", pool[slots[used].long()], h[used].cpu(), (ULP32 * mag[used] + 1e-30).cpu())
    want_pool[slots[used].long()] = pool[slots[used].long()]
    assert torch.equal(pool, want_pool), "the other slots are untouched"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,C,W", [(255, 4096, 4), (1210, 300, 2), (1213, 37, 3)])
def test_convolution_tokens_of_many_sequences(dtype, n, C, W):
    """Four sequences per thread."""
    r = gen(8)
    x, w, b, s = r(n, C).to(dtype), (r(C, W) / W ** 0.5).to(dtype), r(C).to(dtype), r(n, W - 1, C).to(dtype)
    pool, slots = _pool(s, 4, 9)
    want_pool = pool.clone()
    y = kda.conv_decode_step(x, w, pool, b, state_indices=slots)
    kda.check_status()
    line = torch.cat([s, x[:, None]], 1)
    p = (line.double() * w.double().t()).sum(1) + b.double()
    mag = (line.double().abs() * w.double().abs().t()).sum(1) + b.double().abs()
    want = ref.silu(p)
    half = HALF[dtype]
    close("y", y, want.cpu(), (half * 1.001 * want.abs() + 16 * ULP32 * mag + 1e-30).cpu())
    used = slots >= 0
    want_pool[slots[used].long()] = line[used, 1:]
    assert torch.equal(pool, want_pool)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hk,d,half,inter", [(33, 7, 64, 32, False), (3, 17, 128, 32, True), (40, 9, 32, 16, False)])
def test_many_tokens_and_heads_of_the_norm(dtype, hq, hk, d, half, inter):
    """One warp per token, which goes over its heads in several batches; in the backward pass warps take several tokens."""
    rows, r = 5000, gen(10)
    q, k, dq, dk = (r(rows, h, d).to(dtype) for h in (hq, hk, hq, hk))
    qw, kw = (1 + 0.3 * r(d)).to(dtype), (1 + 0.3 * r(d)).to(dtype)
    angle = torch.rand(777, half, device=DEV, dtype=torch.float64) * 6
    cos, sin = angle.cos().float(), angle.sin().float()
    pos = torch.randint(0, 777, (rows,), device=DEV).to(torch.int32)
    kind = dict(q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    out = kda.qk_norm_rotary(q, k, cos, sin, pos, **kind)
    g = kda.qk_norm_rotary_backward(q, k, cos, sin, pos, dq, dk, **kind)
    kda.check_status()
    c, s = (t[pos.long()].double() for t in (cos, sin))
    for name, x, w, got, dout, h in (("q", q, qw, out[0], dq, hq), ("k", k, kw, out[1], dk, hk)):
        x, w, dout = x.double(), w.double(), dout.double()
        want = ref.norm_rotary(x, w, c, s, True, 1e-5, inter)
        u = ref.norm_rotary(x, w, c[:, :0], s[:, :0], True, 1e-5, inter).abs()
        size = torch.maximum(ref.turn(u, c.abs(), -s.abs(), inter), ref.turn(u, c.abs(), s.abs(), inter))
        half_step = HALF[dtype]
        # As at small sizes: one rounding of the output, the squares' sum (d / 2 + 2 half steps), the root and the products, of both terms.
        close(name, got, want.cpu(), (half_step * 1.001 * want.abs() + (d / 2 + 12) * ULP32 * size * 1.5 + 1e-30).cpu())
        rdx, rdw = ref.norm_rotary_backward(x, w, c, s, True, 1e-5, inter, dout)
        near("d" + name, g["d" + name], rdx.cpu(), (d + 24) * ULP32)
        # A warp adds rows / 2432 tokens of h heads in one accumulator, at worst all of them.
        near(f"d{name}_weight", g[f"d{name}_weight"], rdw.cpu(), (d + 24 + 3 * h + 8 * 32) * 4 * ULP32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D,N,G", [(160, 70, 300, 16, 1), (160, 70, 24, 16, 3), (160, 70, 24, 4, 3), (155, 97, 15, 24, 3)])
def test_whole_sequences_that_fill_the_gpu(dtype, B, T, D, N, G):
    """Enough sequences that no chunks are joined, in the forward and in the backward pass."""
    r = gen(11)
    x, dt, z, dy = (r(B, T, D).to(dtype) for _ in range(4))
    Bm, Cm = r(B, T, G, N).to(dtype), r(B, T, G, N).to(dtype)
    A, skip, bias, s, df = -torch.arange(1, N + 1, device=DEV).float().repeat(D, 1), r(D), r(D) - 3, r(B, D, N), r(B, D, N)
    kind = dict(D=skip, z=z, dt_bias=bias, initial_state=s)
    y, fin = kda.scan_prefill(x, dt, A, Bm, Cm, **kind)
    g = kda.scan_backward(x, dt, A, Bm, Cm, dy, d_final_state=df, **kind)
    kda.check_status()
    # One sequence of B * D channels for the reference.
    flat = lambda t: t.double().transpose(0, 1).reshape(T, B * D)  # noqa: E731
    wide = lambda t: t.double().repeat_interleave(D // G, 2).transpose(0, 1).reshape(T, B * D, N)  # noqa: E731
    args = dict(x=flat(x), dt=flat(dt.double() + bias.double()), A=A.double().repeat(B, 1), B=wide(Bm), C=wide(Cm), D=skip.double().repeat(B),
                z=flat(z), softplus=True, init=s.double().view(B * D, N))
    ry, rf = ref.scan(**args)
    m = ref.scan(**{**args, **{k: args[k].abs() for k in ("x", "B", "C", "D", "init")}, "z": None})
    half = HALF[dtype]
    tol = (8 * T + 64) * ULP32  # as for a few sequences: 8 half steps of the state per token, 64 for the output's products
    close("y", y.transpose(0, 1).reshape(T, B * D), ry.cpu(), (half * 1.001 * ry.abs() + tol * m[0] * ref.silu(args["z"]).abs() + 1e-30).cpu())
    close("final_state", fin.view(B * D, N), rf.cpu(), (tol * m[1] + 1e-30).cpu())
    w = ref.scan_backward(**args, dy=flat(dy), d_final=df.double().view(B * D, N))
    tol = 4 * 2 * (8 * 64 + 64) * ULP32  # as for a few sequences: states and gradients, sums of both signs
    for k in ("dx", "ddt", "dz"):
        near(k, g[k].transpose(0, 1).reshape(T, B * D), w[k].cpu(), tol)
    for k in ("dB", "dC"):
        near(k, g[k].transpose(0, 1), w[k].view(T, B, G, D // G, N).sum(3).cpu(), tol)
    near("dA", g["dA"], w["dA"].view(B, D, N).sum(0).cpu(), tol)
    near("dD", g["dD"], w["dD"].view(B, D).sum(0).cpu(), tol)
    near("ddt_bias", g["ddt_bias"], w["ddt"].view(T, B, D).sum((0, 1)).cpu(), tol)
    near("d_initial_state", g["d_initial_state"].view(B * D, N), w["d_init"].cpu(), tol)


@pytest.mark.parametrize("lengths", [[96], [33], [5, 80, 1], [17, 46], [256], [250, 6], [33, 100, 123], [256, 3000], [1, 3, 252, 2000], [4000]])
def test_slow_states_are_carried_whole(lengths):
    """States that forget little over a chunk, joined by the main kernel (few chunks) or by the walk over them (more)."""
    T, D, N, r = sum(lengths), 96, 16, gen(12)
    x, dt, B, C, dy = r(1, T, D), torch.full((1, T, D), 2.0 ** -7, device=DEV), r(1, T, 1, N), r(1, T, 1, N), r(1, T, D)
    A, s, df, cu = -torch.rand(D, N, device=DEV) / 16, r(len(lengths), D, N), r(len(lengths), D, N), cu_of(lengths)
    y, fin = kda.scan_prefill(x, dt, A, B, C, dt_softplus=False, cu_seqlens=cu, initial_state=s)
    g = kda.scan_backward(x, dt, A, B, C, dy, dt_softplus=False, cu_seqlens=cu, initial_state=s, d_final_state=df)
    kda.check_status()
    # A token's roundings (8 half steps at most, of both signs) add up like the root of their number; what does not change sign is the
    # decays' mean error, below 2e-8 each. Over 4000 tokens: 8 * 64 half steps + 4000 * 2e-8 = 1.1e-4 of a state that kept them all at worst.
    tol = 8 * max(lengths) ** 0.5 * ULP32 + max(lengths) * 2e-8
    for i, (lo, hi) in enumerate(ref.spans(1, T, cu.cpu())):
        part = [t[0, lo:hi].double() for t in (x, dt)], [t[0, lo:hi].double().expand(-1, D, -1) for t in (B, C)]
        args = (*part[0], A.double(), *part[1], None, None, False, s[i].double())
        ry, rf = ref.scan(*args)
        near("y", y[0, lo:hi], ry.cpu(), tol)
        near("final_state", fin[i], rf.cpu(), tol)
        w = ref.scan_backward(*args, dy[0, lo:hi].double(), df[i].double())
        near("d_initial_state", g["d_initial_state"][i], w["d_init"].cpu(), tol)
        for k in ("dx", "ddt"):
            near(k, g[k][0, lo:hi], w[k].cpu(), 4 * tol)  # sums over the states of terms of both signs


def _tall(rows, width, tail, seed):
    """bf16 rows of 64 that repeat, with `tail` rows of their own at the end."""
    r = gen(seed)
    t = r(64, width).bfloat16().repeat(rows // 64 + 1, 1)[:rows]
    t[-tail:] = r(tail, width).bfloat16()
    return t.unsqueeze(0)


def test_scan_offsets_past_32_bits():
    """2.2e9 elements: states forget 300 rows, so the first and the last rows are those of short prompts of their own."""
    D, N, T, near_rows = 4096, 4, 530000, 100
    x, dt, z = (_tall(T, D, 700, s) for s in (13, 14, 15))
    B, C = (_tall(T, N, 700, s).view(1, T, 1, N) for s in (16, 17))
    A, bias = -torch.arange(1, N + 1, device=DEV).float().repeat(D, 1), torch.ones(D, device=DEV)  # a row keeps exp(-1.3) on average
    y, fin = kda.scan_prefill(x, dt, A, B, C, z=z, dt_bias=bias)
    short = [t[:, -600:].contiguous() for t in (x, dt, B, C, z)]
    y2, fin2 = kda.scan_prefill(*short[:2], A, *short[2:4], z=short[4], dt_bias=bias)
    kda.check_status()
    off = (y[:, -near_rows:].float() - y2[:, -near_rows:].float()).abs()
    # Both round the same values, cut at other rows, to bf16: a step apart at most, and only where fp32 differs next to a border.
    assert bool((off <= 2.0 ** -7 * y2[:, -near_rows:].float().abs() + 1e-5).all()) and float((off > 0).float().mean()) < 0.01
    # States forget all but 2^-24 within 16 rows: 8 half steps for each of them and 64, as for short prompts; for gradients those of the
    # states and of their gradients, in sums of both signs.
    near("final_state", fin, d64(fin2), (8 * 16 + 64) * ULP32)
    del y, y2
    dy = _tall(T, D, 700, 18)
    g = kda.scan_backward(x, dt, A, B, C, dy, z=z, dt_bias=bias, want_d_initial_state=False)
    kda.check_status()
    for rows in (slice(0, 600), slice(T - 600, T)):
        part = [t[:, rows].contiguous() for t in (x, dt, B, C, dy, z)]
        w = kda.scan_backward(*part[:2], A, *part[2:4], part[4], z=part[5], dt_bias=bias, want_d_initial_state=False)
        inner = slice(0, near_rows) if rows.start == 0 else slice(600 - near_rows, 600)
        for k in ("dx", "ddt", "dz", "dB", "dC"):
            near(k, g[k][:, rows][:, inner], d64(w[k][:, inner]), 4 * 2 * (8 * 16 + 64) * ULP32)
    kda.check_status()


def test_norm_and_convolution_gradients_past_32_bits():
    """2.2e9 elements: the last rows against a call of their own."""
    T, heads, d, tail = 270000, 64, 128, 300
    q, dq = (_tall(T, heads * d, tail, s)[0].view(T, heads, d) for s in (19, 20))
    none = torch.empty(T, 0, d, dtype=torch.bfloat16, device=DEV)
    angle = torch.rand(1000, 64, device=DEV) * 6
    pos = torch.arange(T, device=DEV).remainder(1000).to(torch.int32)
    cos, sin = angle.cos(), angle.sin()
    end = [t[-tail:].contiguous() for t in (q, none, pos, dq)]
    out, _ = kda.qk_norm_rotary(q, none, cos, sin, pos)
    want, _ = kda.qk_norm_rotary(end[0], end[1], cos, sin, end[2])
    assert torch.equal(out[-tail:], want)
    del out, want
    g = kda.qk_norm_rotary_backward(q, none, cos, sin, pos, dq, none)
    w = kda.qk_norm_rotary_backward(end[0], end[1], cos, sin, end[2], end[3], end[1])
    kda.check_status()
    assert torch.equal(g["dq"][-tail:], w["dq"])
    del g, w
    x, dy, f = q.view(1, T, heads * d), dq.view(1, T, heads * d), gen(21)(heads * d, 4).bfloat16()
    g = kda.conv_backward(x, f, dy)
    w = kda.conv_backward(x[:, -tail:].contiguous(), f, dy[:, -tail:].contiguous(), initial_state=x[:, -tail - 3:-tail].contiguous())
    kda.check_status()
    assert torch.equal(g["dx"][:, -tail:], w["dx"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [16, 7])
def test_infinities_and_nan_of_a_sequence_stay_in_it(dtype, N):
    """Between packed neighbours, over chunk borders and in windows that hold several sequences, forward and backward."""
    lengths, D, r = [70, 3, 400, 1, 0, 129, 5, 64, 200], 40, gen(22)
    T, cu, spans = sum(lengths), cu_of(lengths), ref.spans(1, sum(lengths), cu_of(lengths).cpu())
    x, dt, z, dy = (r(1, T, D).to(dtype) for _ in range(4))
    B, C, w, b = r(1, T, 1, N).to(dtype), r(1, T, 1, N).to(dtype), r(D, 4).to(dtype), r(D).to(dtype)
    A, s, df = -torch.rand(D, N, device=DEV), r(len(lengths), D, N), r(len(lengths), D, N)
    cs, cdf = r(len(lengths), 3, D).to(dtype), r(len(lengths), 3, D)

    def outputs():
        scan = dict(z=z, cu_seqlens=cu, initial_state=s)
        conv = dict(bias=b, cu_seqlens=cu, initial_state=cs)
        y, fin = kda.scan_prefill(x, dt, A, B, C, **scan)
        g = kda.scan_backward(x, dt, A, B, C, dy, d_final_state=df, **scan)
        cy, cfin = kda.conv_prefill(x, w, **conv)
        c = kda.conv_backward(x, w, dy, d_final_state=cdf, **conv)
        rows = [t[0].clone() for t in (y, g["dx"], g["ddt"], g["dz"], g["dB"], g["dC"], cy, c["dx"])]
        return rows, [fin, g["d_initial_state"], cfin, c["d_initial_state"]]

    clean = outputs()
    hit = [2, 6]
    for n in hit:
        for i, t in enumerate((x, dt, z, dy, B, C)):
            t[0, spans[n][0] + i % lengths[n]] = (float("nan"), float("inf"), float("-inf"))[i % 3]
        for t in (s, df, cs, cdf):
            t[n] = float("nan")
    dirty = outputs()
    kda.check_status()
    for n, (lo, hi) in enumerate(spans):
        same = [torch.equal(u[lo:hi], v[lo:hi]) for u, v in zip(clean[0], dirty[0])]
        states = [torch.equal(u[n], v[n]) for u, v in zip(clean[1], dirty[1])]
        assert n in hit or (all(same) and all(states)), (n, same, states)
