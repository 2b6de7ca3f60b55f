"""How exact the delta rule with one decay per value head is, for every sequence and head by itself.

Tolerances are what the header says. Where they come from: a value held as two bf16 values is off by at most 2^-18 (half a step of the second, which
is at most 2^-9 of the value), evenly spread: 2^-18 / sqrt(3) = 2.2e-6 at the start of a binade, 1.6e-6 over one. A final state of the bf16
path carries two such operands (the state and R), a gradient those, the two of the chain backward and up to four of the chunk (dR, U, S0 or dS,
the pairs): sqrt(2) and sqrt(8) times 1.6e-6, 2.3e-6 and 4.5e-6, and up to three times that where they meet one another. That is where T's
norm is about 1 (keys that have little to do with one another, beta up to 1). In fp32 a value goes through sums of 128 terms in chains of 8 to 32
and some ten more roundings per chunk, of random signs: 32 half steps for the state, twice that for the gradients, which the state and the
gradient behind it both enter. Other keys and larger beta: errors of A's chunk meet |A| |T|, see the model."""

import math

import pytest
import torch

import delta_model as model
import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from delta_cases import GRADS, Case
from layers_cases import DEV, ULP32

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
STATE = {BF16: 6e-6, FP32: 2e-6}
GRADIENT = {BF16: 1.5e-5, FP32: 4e-6}
# (states, gradients) whatever the keys and decays, for beta up to 1 and up to 2; of the header's bounds for states and beta up to 1 at 8192 rows, those
# at the tests' 832 (equal keys without decays add up the chunks' errors)
ANY_KEYS = {BF16: {1: (4e-5, 2e-4), 2: (1e-3, 1e-3)}, FP32: {1: (2e-6, 1e-5), 2: (3e-4, 3e-4)}}


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


def alike(c, cosine, seed):
    """Keys with that cosine with one another, in every head."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    mean, own = (torch.nn.functional.normalize(torch.randn(x, device=DEV, generator=g), dim=-1) for x in ((1, 1, *c.k.shape[2:]), c.k.shape))
    c.k = torch.nn.functional.normalize(math.sqrt(cosine) * mean + math.sqrt(1 - cosine) * own, dim=-1).to(c.dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shape", [(1, 900, 2, 2, 128, 128, None), (1, 0, 1, 1, 128, 64, [837, 1, 64, 401]), (2, 450, 1, 1, 64, 128, None)])
def test_states_and_gradients_of_many_chunks(dtype, shape):
    """Six chunks and more: every combination of the kernels' stages of two and three. Each sequence and head by itself."""
    c = Case(dtype, *shape, seed=23)
    c.beta = c.beta.clamp(max=1.0)
    o, fin = c.prefill()
    worst = gradients_of_each(c, c.backward())
    kda.check_status()
    for n, (s, _, _) in enumerate(c.sequences()):
        want = ref.delta(*s)[1]
        for h in range(c.heads[1]):
            assert off(fin[n, h], want[h]) <= STATE[dtype], (n, h)
    assert all(v <= GRADIENT[dtype] for v in worst.values()), worst


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cosine", [0.0, 0.8, 0.98, 1.0])
@pytest.mark.parametrize("beta", [1.0, 1.9, 2.0])
@pytest.mark.parametrize("decay", [0.0, 0.3])
def test_keys_that_are_alike_and_large_beta(dtype, cosine, beta, decay):
    """What the header promises; and in bf16 the state as the model of its roundings has it: errors of 16 000 values scatter little, so a half
    more than the model's, and the sums' share in fp32: four half steps (R, U, the state's product and sum), and of A's and T's own an eighth,
    as errors of 64 rows of random signs, of what the largest could meet. One operand with a value less than the model's is beyond it."""
    c = Case(dtype, 1, 832, 2, 2, 128, 128, seed=24, decay=decay)
    alike(c, cosine, 25)
    c.beta[:] = beta
    _, fin = c.prefill()
    worst = gradients_of_each(c, c.backward())
    kda.check_status()
    (s, _, _), = c.sequences()
    want = ref.delta(*s)[1]
    state, gradient = ANY_KEYS[dtype][1 if beta <= 1 else 2]
    for h in range(2):
        q, k, v, g, b, S = (x[h] if x is s[5] else x[:, h] for x in s)
        far = off(fin[0, h], want[h])
        assert far <= (STATE[dtype] if cosine == 0 and beta <= 1 else state), far
        if dtype == BF16:
            expected = off(model.final_state(k, v, g, b, S), want[h])
            assert far <= 1.5 * expected + ULP32 * (4 + model.growth(k, g, b) / 8), (far, expected)
    assert all(v <= (GRADIENT[dtype] if cosine == 0 and beta <= 1 else gradient) for v in worst.values()), worst
