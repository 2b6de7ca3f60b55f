"""The operators around the mixer on the GPU at the ends of their ranges."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers

import layers_ref as ref
from layers_cases import DEV, ULP32, close, cu_of, d64, gen, near

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
