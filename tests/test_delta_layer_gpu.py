"""The delta rule and the layer norm in a run, as a model uses them: the example's layer, tokens against prompts, and its gradients against those of
the whole layer written out in 64 bits."""

import importlib.util
import os

import pytest
import torch

import delta_ref as ref
from layers_cases import DEV, ULP32, d64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_layer.py")
    spec = importlib.util.spec_from_file_location("delta_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs_and_tokens_follow_prompts(example):
    # Both sides round the same eight tensors to bf16 (half steps of 2^-8); they differ only where a rounding falls the other way, by a step of
    # one of them: eight steps of 2^-7 of a row's size at the very most, and the projections average over 256 of them.
    assert example.main() <= 1e-2


def _layer(w, x, residual, hk, hv, d):
    """The layer in 64 bits, one batch row at a time: outputs and sums, differentiable."""
    B, T, _ = x.shape
    n, total = ref.layer_norm(x, w["norm"], None, residual, None, "silu", True, 1e-6)
    p = n @ w["proj"].t()
    mixed = (2 * hk + hv) * d
    line = torch.cat([torch.zeros(B, 3, mixed, dtype=torch.float64), p[..., :mixed]], 1)
    y = sum(w["conv"][:, j] * line[:, j:j + T] for j in range(4))
    y = y / (1 + torch.exp(-y))
    q, k, v = y[..., :hk * d].unflatten(-1, (hk, d)), y[..., hk * d:2 * hk * d].unflatten(-1, (hk, d)), y[..., 2 * hk * d:].unflatten(-1, (hv, d))
    q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    q, k = (t.repeat_interleave(hv // hk, 2) for t in (q, k))
    logits = p[..., mixed + hv * d:]
    g = -w["rate"] * torch.log1p(torch.exp(logits[..., :hv] + w["dt_bias"]))
    beta = 1 / (1 + torch.exp(-logits[..., hv:]))
    S, os = torch.zeros(B, hv, d, d, dtype=torch.float64), []
    for t in range(T):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + torch.einsum("bhk,bhv->bhkv", k[:, t], u)
        os.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    z = p[..., mixed:mixed + hv * d].unflatten(-1, (hv, d))
    n, _ = ref.layer_norm(torch.stack(os, 1), w["head_norm"], None, None, z, "silu", True, 1e-6)
    return n.flatten(-2) @ w["out"].t(), total


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_the_whole_layer(example, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    model, hk, hv, d, T = 64, 1, 2, 32, 70
    layer = example.DeltaLayer(model, hk, hv, d, 1, dtype, DEV, gen)
    x, res, d_out, d_total = (torch.randn(2, T, model, generator=gen, device=DEV).to(dtype) for _ in range(4))
    grads, dx = layer.gradients(x, res, d_out, d_total)
    w = {name: d64(t).requires_grad_() for name, t in layer.weights.items()}
    xr = d64(x).requires_grad_()
    out, total = _layer(w, xr, d64(res), hk, hv, d)
    ((d64(d_out) * out).sum() + (d64(d_total) * total).sum()).backward()
    # fp32: ten operators deep, sums of up to 140 rows: the operators' own 64 half steps each and a product's root of 140, of random signs.
    # bf16: activations and gradients are rounded between the operators, some 25 roundings of half steps of 2^-8 on the way there and back;
    # their relative errors add up at the most.
    tol = 10 * 64 * ULP32 + 140 * ULP32 if dtype == torch.float32 else 25 * 2.0 ** -8
    for name, got in list(grads.items()) + [("x", dx)]:
        want = xr.grad if name == "x" else w[name].grad
        off = float((d64(got) - want).norm() / want.norm())
        assert off <= tol, f"{name}: off by {off:.3e}, allowed {tol:.3e}"
