"""What the GPU tests of the operators around the mixer share: inputs and comparisons."""

import torch

DEV = "cuda:0"
ULP32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: ULP32}  # the one rounding of an output


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device=DEV)


def cu_of(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def strided(t, lead, pad, offset):
    """The same values as a slice of a wider tensor: `pad` more per row, starting `offset` in."""
    inner = 1
    for d in t.shape[lead:]:
        inner *= d
    wide = torch.full((*t.shape[:lead], inner + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[..., offset:offset + inner].unflatten(-1, t.shape[lead:])
    view.copy_(t)
    return view


def d64(t):
    return None if t is None else t.double().cpu()


def close(name, got, want, tol):
    """|got - want| <= tol everywhere (tol a tensor or a number)."""
    got = got.double().cpu()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} for {tuple(want.shape)}"
    off = (got - want).abs() - tol
    assert bool((off <= 0).all()), f"{name}: beyond its tolerance by {off.max():.3e} (values up to {want.abs().max():.3e})"


def near(name, got, want, rel):
    """The 2-norm of the difference against the 2-norm of the value."""
    got = got.double().cpu()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} for {tuple(want.shape)}"
    off, norm = float((got - want).norm()), float(want.norm())
    assert off <= rel * norm or off == 0, f"{name}: off by {off / max(norm, 1e-300):.3e}, allowed {rel:.3e}"
