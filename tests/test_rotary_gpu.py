"""The norm of q and k with the position rotation on the GPU against its definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda

import layers_ref as ref
from layers_cases import DEV, HALF, ULP32, close, d64, gen, near, strided

pytestmark = pytest.mark.gpu


def _tables(rows, half):
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / max(half, 1))
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


CASES = [  # lead, q heads, k heads, head, half, rms, weights, interleaved
    ((1,), 1, 1, 8, 4, True, True, True), ((2, 5), 4, 2, 64, 32, True, True, False), ((3, 7), 3, 1, 128, 32, False, False, False),
    ((1, 70), 32, 8, 128, 64, True, True, False), ((5,), 5, 5, 96, 48, False, True, False), ((9,), 2, 1, 256, 128, True, False, True),
    ((4, 3), 7, 2, 40, 0, True, True, False), ((2, 300), 2, 2, 16, 8, True, True, False), ((6,), 3, 0, 32, 16, False, True, False),
    ((2, 11), 6, 3, 72, 32, True, True, True)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_gradients(dtype, case):
    lead, hq, hk, d, half, rms, weights, inter = case
    r = gen(1)
    q, k = (2 * r(*lead, hq, d)).to(dtype), (0.1 * r(*lead, hk, d)).to(dtype)
    qw, kw = ((1 + 0.3 * r(d)).to(dtype), (1 + 0.3 * r(d)).to(dtype)) if weights else (None, None)
    cos, sin = _tables(50000, half) if half else (None, None)
    pos = torch.randint(0, 50000, lead, device=DEV).to(torch.int32) if half else None
    kind = dict(q_weight=qw, k_weight=kw, norm="rms" if rms else "l2", eps=1e-5, interleaved=inter)
    qo, ko = kda.qk_norm_rotary(q, k, cos, sin, pos, **kind)
    dq, dk = r(*lead, hq, d).to(dtype), r(*lead, hk, d).to(dtype)
    g = kda.qk_norm_rotary_backward(q, k, cos, sin, pos, dq, dk, **kind)
    kda.check_status()
    rows = q.numel() // (hq * d)
    c, s = ((t[pos.long().reshape(-1)].double().cpu() for t in (cos, sin)) if half else
            (torch.zeros(rows, 0, dtype=torch.float64),) * 2)
    for name, x, w, got, dout, dx, dw, h in (("q", q, qw, qo, dq, g["dq"], g["dq_weight"], hq), ("k", k, kw, ko, dk, g["dk"], g["dk_weight"], hk)):
        x, w, dout = d64(x).reshape(rows, h, d), d64(w), d64(dout).reshape(rows, h, d)
        want = ref.norm_rotary(x, w, c, s, rms, 1e-5, inter)
        # One rounding of the output; in fp32 the squares' sum (at most d + 2 half steps, halved by the root), the root's two
        # steps, four products: of the pair's two terms, whose sizes are within sqrt(2) of the pair's length.
        u = ref.norm_rotary(x, w, c[:, :0], s[:, :0], rms, 1e-5, inter).abs()
        size = torch.maximum(ref.turn(u, c.abs(), -s.abs(), inter), ref.turn(u, c.abs(), s.abs(), inter))
        close(name, got.reshape(rows, h, d), want, HALF[dtype] * 1.001 * want.abs() + (d / 2 + 12) * ULP32 * size * 1.5 + 1e-30)
        rdx, rdw = ref.norm_rotary_backward(x, w, c, s, rms, 1e-5, inter, dout)
        near("d" + name, dx.reshape(rows, h, d), rdx, (d + 24) * ULP32)
        if weights and h:
            near(f"d{name}_weight", dw, rdw, (d + 24 + rows * h) * 4 * ULP32)
        elif weights:
            assert not dw.any()
        else:
            assert dw is None
    again = kda.qk_norm_rotary_backward(q, k, cos, sin, pos, dq, dk, **kind)
    assert all(torch.equal(g[n], again[n]) for n in g if g[n] is not None), "the same bits every time"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1), (12, 4)])
def test_strided_rows(dtype, pad, offset):
    r = gen(2)
    q, k = r(2, 9, 4, 64).to(dtype), r(2, 9, 2, 64).to(dtype)
    cos, sin = _tables(64, 32)
    pos = torch.randint(0, 64, (2, 9), device=DEV).to(torch.int32)
    a = kda.qk_norm_rotary(q, k, cos, sin, pos)
    vq, vk = strided(q, 2, pad, offset), strided(k, 2, pad, offset)
    b = kda.qk_norm_rotary(vq, vk, cos, sin, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (kda.qk_norm_rotary_backward(u, v, cos, sin, pos, a[0], a[1]) for u, v in ((q, k), (vq, vk)))
    assert torch.equal(ga["dq"], gb["dq"]) and torch.equal(ga["dk"], gb["dk"])


def test_unit_rows_are_what_the_mixer_normalises_itself():
    """L2 without rotation, then the mixer, against the mixer's own normalisation."""
    import kda_inputs as ki
    x = ki.prefill_inputs(1, 100, 2, 64, 64, dtype=torch.float32, device=DEV, seed=3)
    q, k = 3 * gen(4)(1, 100, 2, 64), 0.3 * gen(5)(1, 100, 2, 64)
    qn, kn = kda.qk_norm_rotary(q, k, norm="l2", eps=1e-6)
    o, s = kda.prefill(qn, kn, x["v"], x["g"], x["beta"])
    o2, s2 = kda.prefill(q, k, x["v"], x["g"], x["beta"], qk_l2norm=True)
    kda.check_status()
    assert (o - o2).norm() <= 5e-3 * o2.norm() and (s - s2).norm() <= 5e-3 * s2.norm()  # tf32 products on one side


def test_rows_of_zeros_and_far_positions():
    q = torch.zeros(3, 2, 64, device=DEV)
    cos, sin = _tables(1 << 17, 32)
    pos = torch.tensor([0, 5, (1 << 17) - 1], dtype=torch.int32, device=DEV)
    for norm in ("rms", "l2"):
        a, b = kda.qk_norm_rotary(q, q, cos, sin, pos, norm=norm)
        assert not a.any() and not b.any()
    kda.check_status()


def test_no_rows():
    q = torch.empty(0, 2, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    a, b = kda.qk_norm_rotary(q, q, q_weight=w)
    g = kda.qk_norm_rotary_backward(q, q, None, None, None, q, q, q_weight=w, k_weight=w)
    kda.check_status()
    assert a.shape == q.shape and not g["dq_weight"].any() and not g["dk_weight"].any()


def test_a_position_outside_the_tables_is_reported():
    q = gen(6)(4, 2, 64)
    cos, sin = _tables(10, 32)
    good = torch.tensor([0, 9, 3, 1], dtype=torch.int32, device=DEV)
    a, _ = kda.qk_norm_rotary(q, q, cos, sin, good)
    plain, _ = kda.qk_norm_rotary(q, q)
    kda.check_status()
    for bad in (-1, 10):
        pos = good.clone()
        pos[2] = bad
        b, _ = kda.qk_norm_rotary(q, q, cos, sin, pos)
        with pytest.raises(kda.KDAError, match="position"):
            kda.check_status()
        assert torch.equal(b[[0, 1, 3]], a[[0, 1, 3]]) and torch.equal(b[2], plain[2])
    kda.check_status()


def test_another_stream_and_a_captured_graph():
    q, w = gen(7)(50, 4, 128).bfloat16(), (1 + 0.1 * gen(8)(128)).bfloat16()
    cos, sin = _tables(64, 64)
    pos = torch.arange(50, device=DEV, dtype=torch.int32)
    a = kda.qk_norm_rotary(q, q, cos, sin, pos, w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = kda.qk_norm_rotary(q, q, cos, sin, pos, w, w)
        g = kda.qk_norm_rotary_backward(q, q, cos, sin, pos, *b, q_weight=w, k_weight=w)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = kda.qk_norm_rotary(q, q, cos, sin, pos, w, w)
        h = kda.qk_norm_rotary_backward(q, q, cos, sin, pos, *c, q_weight=w, k_weight=w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) and torch.equal(u, t) for u, v, t in zip(a, b, c))
    assert all(torch.equal(g[n], h[n]) for n in g)
    kda.check_status()
