"""The model of the bf16 path's roundings, without them, is the definition; with them it is off by what the header says."""

import pytest
import torch

import delta_model as model
import delta_ref as ref


def _head(T, cosine, beta, decay):
    g = torch.Generator().manual_seed(3)
    mean, own = (torch.nn.functional.normalize(torch.randn(*s, generator=g), dim=-1) for s in ((64,), (T, 64)))
    k = torch.nn.functional.normalize(cosine ** 0.5 * mean + (1 - cosine) ** 0.5 * own, dim=-1).bfloat16().double()
    v, S = torch.randn(T, 48, generator=g).bfloat16().double(), torch.randn(64, 48, generator=g).double()
    return k, v, -decay * torch.rand(T, generator=g).double(), torch.full((T,), float(beta), dtype=torch.float64), S


def _exact(k, v, g, b, S):
    return ref.delta(k[:, None], k[:, None], v[:, None], g[:, None], b[:, None], S[None])[1][0]


@pytest.mark.parametrize("T,cosine,beta,decay", [(64, 0.0, 1, 0), (130, 0.9, 0.7, 0.1), (200, 0.5, 2, 1.0), (1, 0, 1, 0)])
def test_without_roundings_it_is_the_definition(monkeypatch, T, cosine, beta, decay):
    monkeypatch.setattr(model, "bf16_values", lambda x, n: [x] + [torch.zeros_like(x)] * (n - 1))
    monkeypatch.setattr(model, "tf32_values", lambda x: [x, torch.zeros_like(x)])
    head = _head(T, cosine, beta, decay)
    want = _exact(*head)
    assert (model.final_state(*head) - want).norm() <= 1e-11 * want.norm()


@pytest.mark.parametrize("cosine,beta,bound", [(0.0, 1, 6e-6), (0.8, 1, 4e-5), (0.98, 1, 4e-5), (1.0, 1, 4e-5), (0.0, 2, 1e-3), (0.98, 2, 1e-3),
                                               (1.0, 1.9, 1e-3), (1.0, 2, 1e-3)])
@pytest.mark.parametrize("T", [64, 2048])
def test_with_them_it_is_as_exact_as_the_header_says(T, cosine, beta, bound):
    head = _head(T, cosine, beta, 0)
    want = _exact(*head)
    assert (model.final_state(*head) - want).norm() <= bound * want.norm()
