"""The operators around the mixer on the GPU at the ends of their ranges."""

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers

from layers_cases import DEV

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
