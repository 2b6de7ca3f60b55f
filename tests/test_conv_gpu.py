"""The short causal convolution on the GPU against its definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda

import layers_ref as ref
from layers_cases import DEV, HALF, ULP32, close, cu_of, d64, gen, near, strided

pytestmark = pytest.mark.gpu


def _inputs(dtype, B, T, C, W, bias, states, seqs, seed):
    r = gen(seed)
    x, w = r(B, T, C).to(dtype), (r(C, W) / W ** 0.5).to(dtype)
    return x, w, r(C).to(dtype) if bias else None, r(seqs, W - 1, C).to(dtype) if states else None, r


def _reference(x, w, b, act, init, spans, W):
    """y, final states, and the sum of the terms' absolute values (for the tolerance)."""
    C = x.shape[-1]
    x, w, b, init = d64(x).reshape(-1, C), d64(w), d64(b), d64(init)
    y, fin, mag = torch.zeros_like(x), torch.zeros(len(spans), W - 1, C, dtype=torch.float64), torch.zeros_like(x)
    zero = torch.zeros(W - 1, C, dtype=torch.float64)
    for n, (lo, hi) in enumerate(spans):
        s = zero if init is None else init[n]
        y[lo:hi], fin[n] = ref.conv(x[lo:hi], w, b, act, s)
        mag[lo:hi] = ref.conv(x[lo:hi].abs(), w.abs(), None if b is None else b.abs(), False, s.abs())[0]
    return y, fin, mag


def _tol(dtype, y, mag):
    # One rounding of the output; W + 1 roundings of the terms in fp32 and the sigmoid's 2^-21 (slope of SiLU at most 1.1).
    return HALF[dtype] * 1.001 * y.abs() + 16 * ULP32 * mag + 1e-30


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,C,W,act,bias,states", [
    (1, 1, 8, 4, True, False, False), (2, 3, 13, 4, True, True, True), (3, 70, 40, 3, False, True, False),
    (2, 257, 264, 4, True, False, True), (1, 515, 1, 2, True, True, True), (2, 31, 300, 2, False, False, False)])
def test_prompts(dtype, B, T, C, W, act, bias, states):
    x, w, b, s, _ = _inputs(dtype, B, T, C, W, bias, states, B, 1)
    y, fin = kda.conv_prefill(x, w, b, activation="silu" if act else None, initial_state=s)
    kda.check_status()
    ry, rf, mag = _reference(x, w, b, act, s, ref.spans(B, T), W)
    close("y", y.reshape(-1, C), ry, _tol(dtype, ry, mag))
    assert torch.equal(fin.double().cpu(), rf)


@pytest.mark.parametrize("dtype,C", [(torch.bfloat16, 72), (torch.float32, 20), (torch.bfloat16, 37)])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lengths", [[5, 1, 0, 2, 130, 0, 33], [0, 0, 7], [300], [1, 1, 1, 1, 1, 0]])
def test_packed_sequences_states_and_pools(dtype, C, W, lengths):
    n, T = len(lengths), sum(lengths)
    x, w, b, s, r = _inputs(dtype, 1, T, C, W, True, True, n, 2)
    cu = cu_of(lengths)
    spans = ref.spans(1, T, cu.cpu())
    y, fin = kda.conv_prefill(x, w, b, cu_seqlens=cu, initial_state=s)
    ry, rf, mag = _reference(x, w, b, True, s, spans, W)
    close("y", y[0], ry, _tol(dtype, ry, mag))
    assert torch.equal(fin.double().cpu(), rf)
    # the same through a pool, in place; one sequence without a slot
    pool = r(n + 3, W - 1, C).to(dtype)
    slots = torch.randperm(n + 3)[:n]
    pool[slots.to(DEV)] = s
    slots[n // 2] = -1
    kept = pool.clone()
    idx = slots.to(torch.int32).to(DEV)
    y2, out = kda.conv_prefill(x, w, b, cu_seqlens=cu, initial_state=pool, final_state=pool, initial_state_indices=idx,
                               final_state_indices=idx)
    kda.check_status()
    assert out is pool
    s2 = s.clone()
    s2[n // 2] = 0
    ry, rf, mag = _reference(x, w, b, True, s2, spans, W)
    close("y", y2[0], ry, _tol(dtype, ry, mag))
    for i in range(n):
        if slots[i] >= 0:
            kept[slots[i]] = rf[i].to(dtype).to(DEV)
    assert torch.equal(pool, kept), "slots of the call hold its final states, the others are untouched"


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1), (16, 5)])
def test_strided_rows(pad, offset):
    for dtype in (torch.bfloat16, torch.float32):
        x, w, b, s, r = _inputs(dtype, 2, 45, 48, 4, True, True, 2, 3)
        v = strided(x, 2, pad, offset)
        dy = r(2, 45, 48).to(dtype)
        y, fin = kda.conv_prefill(x, w, b, initial_state=s)
        y2, fin2 = kda.conv_prefill(v, w, b, initial_state=s)
        assert torch.equal(y, y2) and torch.equal(fin, fin2)
        g, g2 = (kda.conv_backward(t, w, dy, b, initial_state=s) for t in (x, v))
        for k in ("dx", "d_initial_state"):
            assert torch.equal(g[k], g2[k]), k
        near("dweight", g2["dweight"], d64(g["dweight"]), 1e-5)  # another split of the sum over 90 rows
        st, st2 = s.clone(), s.clone()
        assert torch.equal(kda.conv_decode_step(x[:, 0].contiguous(), w, st, b), kda.conv_decode_step(v[:, 0], w, st2, b))
        assert torch.equal(st, st2)


@pytest.mark.parametrize("dtype,C,W,act", [(torch.bfloat16, 264, 4, True), (torch.float32, 13, 3, False), (torch.bfloat16, 7, 2, True)])
def test_prefill_then_tokens_is_one_prefill(dtype, C, W, act):
    T, more, B = 21, 6, 3
    x, w, b, s, _ = _inputs(dtype, B, T + more, C, W, True, True, B, 4)
    act = "silu" if act else None
    y, fin = kda.conv_prefill(x, w, b, activation=act, initial_state=s)
    y1, st = kda.conv_prefill(x[:, :T].contiguous(), w, b, activation=act, initial_state=s)
    assert torch.equal(y1, y[:, :T])
    pool = torch.zeros(B + 1, W - 1, C, dtype=dtype, device=DEV)
    idx = torch.tensor([3, 0, 2], dtype=torch.int32, device=DEV)
    pool[idx.long()] = st
    for t in range(T, T + more):
        yt = kda.conv_decode_step(x[:, t].contiguous(), w, st, b, activation=act)
        yp = kda.conv_decode_step(x[:, t].contiguous(), w, pool, b, activation=act, state_indices=idx)
        assert torch.equal(yt, y[:, t]) and torch.equal(yp, yt)
    assert torch.equal(st, fin) and torch.equal(pool[idx.long()], fin)
    assert not pool[1].any()
    # branching: read one slot, write another; a sequence without a slot starts from zeros and writes none
    to = torch.tensor([1, -1, 2], dtype=torch.int32, device=DEV)
    frm = torch.tensor([3, 0, -1], dtype=torch.int32, device=DEV)
    before = pool.clone()
    xt = x[:, 0].contiguous()
    yb = kda.conv_decode_step(xt, w, pool, b, activation=act, state_indices=frm, final_state_indices=to)
    start = torch.stack([before[3], before[0], torch.zeros_like(before[0])])
    want = kda.conv_decode_step(xt, w, start, b, activation=act)
    kda.check_status()
    assert torch.equal(yb, want)
    before[1], before[2] = start[0], start[2]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,W,act,bias,states,lengths", [
    (40, 4, True, True, True, None), (13, 3, True, False, True, [3, 0, 1, 70, 2, 290]), (264, 2, False, True, False, [1]),
    (8, 4, True, True, True, [0, 2, 40, 0]), (64, 4, True, True, True, [600, 1])])
def test_gradients(dtype, C, W, act, bias, states, lengths):
    B, T = (2, 37) if lengths is None else (1, sum(lengths))
    n = B if lengths is None else len(lengths)
    x, w, b, s, r = _inputs(dtype, B, T, C, W, bias, states, n, 5)
    dy, df = r(B, T, C).to(dtype), r(n, W - 1, C) if states else None
    cu = None if lengths is None else cu_of(lengths)
    g = kda.conv_backward(x, w, dy, b, activation="silu" if act else None, cu_seqlens=cu, initial_state=s, d_final_state=df)
    kda.check_status()
    rx, rw, rb, ri = [], 0, 0, []
    for i, (lo, hi) in enumerate(ref.spans(B, T, None if cu is None else cu.cpu())):
        zero = torch.zeros(W - 1, C, dtype=torch.float64)
        a = ref.conv_backward(d64(x).reshape(-1, C)[lo:hi], d64(w), d64(b), act, zero if s is None else d64(s)[i],
                              d64(dy).reshape(-1, C)[lo:hi], zero if df is None else d64(df)[i])
        rx.append(a[0])
        rw, rb = rw + a[1], rb + a[2]
        ri.append(a[3])
    # fp32 roundings of W + 4 terms and the sigmoid's 2^-21 for rows; sqrt-free worst case of a sum over T rows for the filter
    near("dx", g["dx"].reshape(-1, C), torch.cat(rx), 32 * ULP32)
    near("d_initial_state", g["d_initial_state"], torch.stack(ri), 32 * ULP32)
    near("dweight", g["dweight"], rw, (32 + T) * 4 * ULP32)
    if bias:
        near("dbias", g["dbias"], rb, (32 + T) * 4 * ULP32)
    else:
        assert g["dbias"] is None
    again = kda.conv_backward(x, w, dy, b, activation="silu" if act else None, cu_seqlens=cu, initial_state=s, d_final_state=df)
    assert all(torch.equal(g[k], again[k]) for k in g if g[k] is not None), "the same bits every time"


def test_no_rows():
    w, s = torch.ones(8, 4, device=DEV), gen(6)(2, 3, 8)
    x = torch.empty(2, 0, 8, device=DEV)
    y, fin = kda.conv_prefill(x, w, initial_state=s)
    assert y.shape == (2, 0, 8) and torch.equal(fin, s)
    df = gen(7)(2, 3, 8)
    g = kda.conv_backward(x, w, x, initial_state=s, d_final_state=df)
    assert torch.equal(g["d_initial_state"], df) and not g["dweight"].any()
    _, fin = kda.conv_prefill(x, w)
    kda.check_status()
    assert not fin.any()


def test_offsets_past_32_bits():
    """2.2e9 elements: the last rows against the same rows as a prompt of their own."""
    C, T = 8192, 268500
    r = gen(8)
    x = r(64, C).bfloat16().repeat(T // 64 + 1, 1)[:T].unsqueeze(0)
    x[0, -100:] = r(100, C).bfloat16()
    w = r(C, 4).bfloat16()
    y, fin = kda.conv_prefill(x, w)
    y2, fin2 = kda.conv_prefill(x[:, -100:].contiguous(), w, initial_state=x[:, -103:-100].contiguous())
    kda.check_status()
    assert torch.equal(y[:, -100:], y2) and torch.equal(fin, fin2)


def test_infinities_and_nan_stay_in_their_channel_and_window():
    x, w, _, _, _ = _inputs(torch.float32, 1, 20, 16, 4, False, False, 1, 9)
    clean, _ = kda.conv_prefill(x, w)
    x[0, 5, 3], x[0, 9, 7] = float("nan"), float("inf")
    y, _ = kda.conv_prefill(x, w)
    hit = torch.zeros(20, 16, dtype=torch.bool, device=DEV)
    hit[5:9, 3], hit[9:13, 7] = True, True
    assert torch.equal(y[0][~hit], clean[0][~hit]) and torch.isnan(y[0, 5:9, 3]).all()


def test_a_bad_cu_seqlens_and_a_bad_slot_are_reported():
    x, w, _, _, _ = _inputs(torch.bfloat16, 1, 20, 16, 4, False, False, 1, 10)
    for cu in ([0, 12, 8, 20], [0, 25, 30, 20], [3, 5, 9, 20], [0, 4, 9, 19], [0, -5, 9, 20]):
        kda.conv_prefill(x, w, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_status()
    pool = torch.zeros(2, 3, 16, dtype=torch.bfloat16, device=DEV)
    kda.conv_decode_step(x[0, :1].contiguous(), w, pool, state_indices=torch.tensor([2], dtype=torch.int32, device=DEV))
    with pytest.raises(kda.KDAError, match="pool"):
        kda.check_status()
    assert not pool.any()
    kda.check_status()


def test_another_stream_and_a_captured_graph():
    x, w, b, s, _ = _inputs(torch.bfloat16, 2, 50, 64, 4, True, True, 2, 11)
    y, fin = kda.conv_prefill(x, w, b, initial_state=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, fin2 = kda.conv_prefill(x, w, b, initial_state=s)
        dy = y2 * 1
        g2 = kda.conv_backward(x, w, dy, b, initial_state=s)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    graph = torch.cuda.CUDAGraph()
    st, xt = s.clone(), x[:, 0].contiguous()
    with torch.cuda.graph(graph):
        y3, fin3 = kda.conv_prefill(x, w, b, initial_state=s)
        g3 = kda.conv_backward(x, w, dy, b, initial_state=s)
        y4 = kda.conv_decode_step(xt, w, st, b)
    st.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, y) and torch.equal(fin3, fin) and all(torch.equal(g3[k], g2[k]) for k in g2)
    assert torch.equal(y4, y[:, 0])
    kda.check_status()
