"""The delta rule with one decay per value head on the GPU against its 64-bit definition."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from delta_cases import GRADS, Case
from layers_cases import DEV, gen, strided

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32

SHAPES = [  # B, T, hk, hv, dk, dv, lengths
    (1, 1, 1, 1, 128, 128, None), (2, 3, 1, 2, 32, 64, None), (1, 64, 2, 2, 128, 128, None), (2, 65, 1, 3, 64, 32, None),
    (1, 200, 2, 4, 128, 64, None), (1, 127, 1, 2, 64, 128, None), (3, 63, 2, 2, 32, 32, None), (1, 300, 1, 2, 128, 128, None),
    (1, 129, 1, 1, 32, 128, None), (1, 191, 2, 2, 64, 64, None), (1, 66, 1, 4, 128, 32, None),
    (1, 0, 2, 4, 128, 128, [1, 0, 64, 65, 7, 130]), (1, 0, 1, 2, 64, 64, [0, 2, 63, 0, 128, 0]), (1, 0, 2, 2, 128, 128, [1, 1, 1]),
    (1, 0, 1, 1, 32, 32, [0, 0, 5])]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts(dtype, shape):
    c = Case(dtype, *shape, seed=1)
    c.check_prefill(*c.prefill())
    kda.check_status()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(dtype, shape):
    c = Case(dtype, *shape, seed=2)
    g = c.backward()
    kda.check_status()
    c.check_backward(g)
    again = c.backward()
    assert all(torch.equal(g[k], again[k]) for k in GRADS), "the same bits every time"


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_without_states(dtype):
    c = Case(dtype, 2, 150, 2, 4, 128, 128, seed=3, states=False)
    o, fin = c.prefill()
    c.check_prefill(o, fin)
    o2, none = c.prefill(output_final_state=False)
    assert none is None and torch.equal(o, o2)
    c.check_backward()
    g = c.backward(want_d_initial_state=False)
    assert g["d_initial_state"] is None
    c.check_backward(g)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("decay", [0.0, 1e-3, 20.0, 500.0])
def test_decays_from_none_to_complete(dtype, decay):
    """Up to exp(-500): the chunk's sums of decays keep the differences of their neighbours."""
    c = Case(dtype, 1, 200, 1, 2, 128, 128, seed=4, decay=decay)
    c.check_prefill(*c.prefill())
    c.check_backward()
    kda.check_status()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_minus_infinity_clears_the_state_and_zero_beta_writes_nothing(dtype):
    c = Case(dtype, 1, 150, 1, 2, 128, 128, seed=5)
    c.g[0, 70], c.g[0, 100, 1] = float("-inf"), float("-inf")
    c.beta[0, 20:40] = 0
    c.beta[0, 140:] = 1
    c.check_prefill(*c.prefill())
    c.check_backward()
    o, _ = c.prefill()
    half = Case(dtype, 1, 80, 1, 2, 128, 128, seed=5, states=False)
    for name in ("q", "k", "v", "g", "beta"):
        setattr(half, name, getattr(c, name)[:, 70:].contiguous())
    half.check_prefill(o[:, 70:], None)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_equal_keys(dtype):
    """The same key in every row: the triangular systems at their worst."""
    c = Case(dtype, 1, 130, 1, 2, 128, 128, seed=6, decay=0.01)
    c.k[:] = c.k[:, :1].clone()
    c.check_prefill(*c.prefill())
    c.check_backward()


@pytest.mark.parametrize("dtype,pads", [(BF16, ((8, 8), (3, 1))), (FP32, ((4, 4), (5, 3)))])
@pytest.mark.parametrize("T", [45, 130])
def test_strided_rows(dtype, pads, T):
    c = Case(dtype, 2, T, 2, 4, 128, 64, seed=7)
    o, fin = c.prefill()
    c.check_prefill(o, fin)
    g = c.backward()
    for pad, offset in pads:
        s = Case(dtype, 2, T, 2, 4, 128, 64, seed=7)
        s.q, s.k, s.v = (strided(t, 2, pad, offset) for t in (c.q, c.k, c.v))
        o2, fin2 = s.prefill()
        s.check_prefill(o2, fin2)
        s.check_backward(s.backward())
        one = [kda.delta_decode_step(*(t[:, 0] if x is s else t[:, 0].contiguous() for t in x.inputs()[:3]), x.g[:, 0].contiguous(),
                                     x.beta[:, 0].contiguous(), st) for x, st in ((s, s.state.clone()), (c, c.state.clone()))]
        assert torch.equal(*one)
    kda.check_status()
    assert g["dq"].shape == c.q.shape


@pytest.mark.parametrize("dtype,hk,hv,dk,dv", [(BF16, 2, 4, 128, 128), (FP32, 1, 3, 64, 32), (BF16, 1, 1, 32, 128), (FP32, 2, 2, 128, 64)])
def test_prefill_then_tokens(dtype, hk, hv, dk, dv):
    T, more, B = 70, 5, 3
    c = Case(dtype, B, T + more, hk, hv, dk, dv, seed=8)
    o1, st = kda.delta_prefill(*(t[:, :T].contiguous() for t in c.inputs()), initial_state=c.state)
    pool = torch.zeros(B + 1, hv, dk, dv, device=DEV)
    idx = torch.tensor([3, 0, 2], dtype=torch.int32, device=DEV)
    pool[idx.long()] = st
    os = [o1]
    for t in range(T, T + more):
        at = [x[:, t].contiguous() for x in c.inputs()]
        os.append(kda.delta_decode_step(*at, st)[:, None])
        op = kda.delta_decode_step(*at, pool, state_indices=idx)
        assert torch.equal(op, os[-1][:, 0])
    assert torch.equal(pool[idx.long()], st) and not pool[1].any()
    c.check_prefill(torch.cat(os, 1), st)
    # branching, and a sequence without a slot
    frm, to = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([3, 0, -1], [1, -1, 2]))
    before = pool.clone()
    ob = kda.delta_decode_step(*at, pool, state_indices=frm, final_state_indices=to)
    start = torch.stack([before[3], before[0], torch.zeros_like(before[0])])
    want = kda.delta_decode_step(*at, start)
    kda.check_status()
    assert torch.equal(ob, want)
    before[1], before[2] = start[0], start[2]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lengths", [[5, 1, 0, 2, 130], [300, 0, 64]])
def test_pools_in_place(dtype, lengths):
    n = len(lengths)
    c = Case(dtype, 1, 0, 1, 2, 128, 128, lengths, seed=9)
    pool = gen(10)(n + 2, 2, 128, 128)
    slots = torch.randperm(n + 2)[:n]
    pool[slots.to(DEV)] = c.state
    slots[1] = -1
    c.state[1] = 0
    o, fin = c.prefill()
    kept = pool.clone()
    for i in range(n):
        if slots[i] >= 0:
            kept[slots[i]] = fin[i]
    idx = slots.to(torch.int32).to(DEV)
    o2, out = c.prefill(initial_state=pool, final_state=pool, initial_state_indices=idx, final_state_indices=idx)
    kda.check_status()
    assert out is pool and torch.equal(o, o2) and torch.equal(pool, kept)
    own = c.state.clone()
    o3, _ = c.prefill(initial_state=own, final_state=own)
    assert torch.equal(o, o3) and torch.equal(own, fin)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_no_rows_and_no_sequences(dtype):
    c = Case(dtype, 2, 0, 1, 2, 64, 64, seed=11)
    o, fin = c.prefill()
    assert o.shape == (2, 0, 2, 64) and torch.equal(fin, c.state)
    g = c.backward()
    assert torch.equal(g["d_initial_state"], c.d_final) and g["dq"].shape == (2, 0, 1, 64)
    e = Case(dtype, 0, 5, 1, 2, 64, 64, seed=11)
    assert e.prefill()[0].shape == (0, 5, 2, 64)
    e.backward()
    packed = Case(dtype, 1, 0, 1, 2, 128, 128, [0, 0], seed=11)
    o, fin = packed.prefill()
    assert torch.equal(fin, packed.state)
    assert torch.equal(packed.backward()["d_initial_state"], packed.d_final)
    kda.check_status()


def test_nan_and_infinity_stay_in_their_sequence_and_head():
    for dtype in (BF16, FP32):
        c = Case(dtype, 2, 140, 2, 4, 128, 128, seed=12)
        clean, fin = c.prefill()
        gc = c.backward()
        c.v[0, 50, 1, 3], c.g[0, 80, 2] = float("nan"), float("nan")
        o, f2 = c.prefill()
        g = c.backward()
        kda.check_status()
        assert torch.equal(o[1], clean[1]) and torch.equal(f2[1], fin[1])
        for h in (0, 3):
            assert torch.equal(o[0, :, h], clean[0, :, h])
            assert torch.equal(g["dv"][0, :, h], gc["dv"][0, :, h])
        assert torch.isnan(o[0, 80:, 2].float()).all() and torch.isnan(o[0, 50:, 1, 3].float()).all()
        assert all(torch.equal(g[k][1], gc[k][1]) for k in GRADS)


def test_a_bad_cu_seqlens_and_a_bad_slot_are_reported():
    for dtype in (BF16, FP32):
        for cu in ([0, 120, 80, 200], [0, 250, 300, 200], [3, 5, 90, 200], [0, 40, 90, 190], [0, -5, 90, 200]):
            c = Case(dtype, 1, 0, 1, 1, 128, 128, [100, 50, 50], seed=14)
            c.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
            c.prefill()
            with pytest.raises(kda.KDAError, match="cu_seqlens"):
                kda.check_status()
            c.backward()
            with pytest.raises(kda.KDAError, match="cu_seqlens"):
                kda.check_status()
        c = Case(dtype, 1, 100, 1, 1, 128, 128, seed=15)
        pool = torch.zeros(2, 1, 128, 128, device=DEV)
        bad = torch.tensor([2], dtype=torch.int32, device=DEV)
        c.prefill(initial_state=pool, final_state=pool, initial_state_indices=bad, final_state_indices=bad)
        with pytest.raises(kda.KDAError, match="pool"):
            kda.check_status()
        kda.delta_decode_step(*(x[:, 0].contiguous() for x in c.inputs()), pool, state_indices=bad)
        with pytest.raises(kda.KDAError, match="pool"):
            kda.check_status()
        assert not pool.any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_captured_twice_and_replayed(dtype):
    """Two graphs over the same inputs, replayed in turn, with a call of another size between them."""
    c = Case(dtype, 2, 200, 1, 2, 128, 128, seed=16)
    o, fin = c.prefill()
    g = c.backward()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((c.prefill(), c.backward()))
        graphs.append(graph)
    other = Case(dtype, 1, 77, 1, 2, 128, 128, seed=17)
    for i in (0, 1, 0, 1):
        graphs[i].replay()
        other.backward()
    torch.cuda.synchronize()
    for (o2, fin2), g2 in outs:
        assert torch.equal(o, o2) and torch.equal(fin, fin2) and all(torch.equal(g[k], g2[k]) for k in GRADS)
    kda.check_status()


def test_two_streams_at_once():
    a, b = (Case(BF16, 1, 500, 1, 2, 128, 128, seed=s) for s in (18, 19))
    want = [(x.prefill(), x.backward()) for x in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append((x.prefill(), x.backward()))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for (o, f), g in gs:
            assert torch.equal(o, w[0][0]) and torch.equal(f, w[0][1]) and all(torch.equal(g[k], w[1][k]) for k in GRADS)
