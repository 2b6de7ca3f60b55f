"""The gate's gradient of the layer norm, value by value, at gates far from zero."""

import pytest
import torch

import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from layers_cases import DEV, HALF, ULP32, close, d64, gen

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("D", [128, 135, 1000])
def test_gates_far_from_zero(dtype, kind, D):
    r = gen(40)
    x, dy = r(64, D).to(dtype), r(64, D).to(dtype)
    z = torch.linspace(-60, 60, 64 * D, device=DEV).reshape(D, 64).t().contiguous().to(dtype)
    g = kda.layer_norm_backward(x, None, dy, gate=z, activation=kind, norm="rms")
    X, Z, DY = d64(x), d64(z), d64(dy)
    # exp(-z): z log2(e) is rounded and log2(e) itself is (a half step each, of an exponent of |z|), the instruction's 2^-22.7 and the
    # reciprocal's 2^-23 are five half steps together. The normed value: a sum of D squares over 8 to 1024 lanes and its root, 16. The
    # products and sums around them: 8. A sum of both signs (SiLU's slope) is off by this of its terms' size.
    # 1 - sigmoid(z) is sigmoid(-z) here too: the difference has 2^-53 of 1 at best, also in 64 bits.
    e, other = 1 / (1 + torch.exp(-Z)), 1 / (1 + torch.exp(Z))
    n = X / torch.sqrt((X * X).mean(-1, keepdim=True) + 1e-6)
    slope, size = (e + Z * e * other, e + Z.abs() * e * other) if kind == "silu" else (e * other, e * other)
    close("dgate", g["dgate"], DY * n * slope, (DY * n).abs() * size * ULP32 * (2 * Z.abs() + 32) + 1e-37)


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
def test_gates_at_the_ends(kind):
    """Gates of fp32's largest values close and open: nothing is not a number."""
    x = gen(41)(4, 64)
    z = torch.full((4, 64), 3e38, device=DEV)
    z[::2] = -3e38
    g = kda.layer_norm_backward(x, None, torch.ones_like(x), gate=z, activation=kind, norm="rms")
    assert not g["dgate"][::2].any()
    n = ref.layer_norm(d64(x), None, None, None, None, None, True, 1e-6)[0]
    close("open", g["dgate"][1::2], n[1::2] * (kind == "silu"), 32 * ULP32 * n[1::2].abs())
