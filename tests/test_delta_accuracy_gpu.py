"""How exact the delta rule with one decay per value head is, for every sequence and head by itself.

Tolerances. A value held as two bf16 values is off by at most 2^-18 (half a step of the second, which is at most 2^-9 of the value), evenly
spread: 2^-18 / sqrt(3) = 2.2e-6 at the start of a binade, 1.6e-6 over one. A final state of the bf16 path carries three such operands (the
state, R and T - I): sqrt(3) * 1.6e-6 = 2.8e-6. A gradient carries those, the three of the chain backward, and up to four of the chunk
(dR, U, S0 or dS, the pairs): sqrt(10) * 1.6e-6 = 5e-6. Errors of a norm over one head scatter little; a factor of 2 for the state and of 3
for the gradients, which meet one another. That is where T's norm is about 1 (keys that have little to do with one another, beta up to 1).
In fp32 a value goes through sums of 128 terms in chains of 8 to 32 and some ten more roundings per chunk, of random signs: 32 half
steps for the state, twice that for the gradients, which the state and the gradient behind it both enter."""

import pytest
import torch

import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from delta_cases import GRADS, Case
from layers_cases import DEV, ULP32

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
STATE = {BF16: 2 * 2.8e-6, FP32: 32 * ULP32}
GRADIENT = {BF16: 3 * 5e-6, FP32: 64 * ULP32}


def uniform(c, g):
    """Log-decays within a tenth of g in every row."""
    r = torch.rand(c.g.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(21))
    c.g = g * (0.9 + 0.2 * r)
    return c


def off(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item() if want.numel() else 0.0


def gradients_of_each(c, g):
    """{name: the largest distance over sequences and heads} of gradients of one value head per key head."""
    worst = dict.fromkeys(GRADS, 0.0)
    at = 0
    for n, (s, do, df) in enumerate(c.sequences()):
        want = ref.delta_backward(*s, do, df)
        rows = slice(at, at + do.shape[0])
        at += do.shape[0]
        for name, w in zip(GRADS, want):
            got = g[name][n] if name == "d_initial_state" else g[name].flatten(0, 1)[rows]
            for h in range(c.heads[1]):
                i = (h,) if name == "d_initial_state" else (slice(None), h)
                worst[name] = max(worst[name], off(got[i], w[i]))
    return worst


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("g", [-0.01, -1.0, -5.0, -12.0, -20.0, -60.0])
@pytest.mark.parametrize("shape", [(1, 150, 2, 2, 128, 128, None), (1, 0, 2, 2, 64, 32, [70, 17, 130])])
def test_the_decays_gradients_behind_strong_decays(dtype, g, shape):
    """Every row decays strongly, so dg is as small as exp(g) everywhere: it must not be the rest of terms that are not."""
    c = uniform(Case(dtype, *shape, seed=20), g)
    worst = gradients_of_each(c, c.backward())
    kda.check_status()
    assert all(v <= GRADIENT[dtype] for v in worst.values()), worst


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("what", ["q", "k", "v", "beta", "d_o"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_reaches_the_gradients_that_the_formulas_give_it_to(dtype, what, value):
    """Gradients that do not depend on the bad value are those of a call without it, bit for bit (bf16: outside the value's chunk of 64)."""
    T, row = 200, 101
    c = Case(dtype, 1, T, 2, 2, 128, 128, seed=22)
    clean = c.backward()
    getattr(c, what)[(0, row, 1) if what == "beta" else (0, row, 1, 5)] = value
    g = c.backward()
    kda.check_status()
    (s, do, df), = c.sequences()
    s = list(s)
    # What depends on it, by the definition in 64 bits: NaN there.
    names = ("q", "k", "v", "g", "beta")
    if what == "d_o":
        do[row, 1, 5] = float("nan")
    else:
        s[names.index(what)][(row, 1) if what == "beta" else (row, 1, 5)] = float("nan")
    finite = 0
    for name, w in zip(GRADS, ref.delta_backward(*s, do, df)):
        got, before = g[name].cpu(), clean[name].cpu()
        free = torch.isfinite(w).reshape(got.shape)
        if dtype == BF16 and name != "d_initial_state":
            free[:, 64:128, 1] = False
        finite += int(free.sum())
        assert torch.equal(got[free], before[free]), name
    assert finite > 0
