"""The operators around the mixer on the GPU at the ends of their ranges."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers

from layers_cases import DEV, cu_of, gen

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
