"""Workspaces and outputs of the delta rule with one decay per value head at the ends of their sizes."""

import ctypes

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from delta_cases import GRADS, Case
from gated_delta_rule_56_gb300 import layers
from layers_cases import DEV, strided

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def _args(c):
    (B, T), (hk, hv), (dk, dv) = c.shape, c.heads, c.sizes
    n = B if c.lengths is None else len(c.lengths)
    rows = [t.stride(1) for t in (c.q, c.k, c.v)]
    return layers.DeltaArgs(ctypes.sizeof(layers.DeltaArgs), layers._DTYPES[c.dtype], B, T, hk, hv, dk, dv, c.q.data_ptr(), c.k.data_ptr(),
                            c.v.data_ptr(), *rows, c.g.data_ptr(), c.beta.data_ptr(), None if c.cu is None else c.cu.data_ptr(), n,
                            c.state.data_ptr())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32)])
@pytest.mark.parametrize("lengths", [None, [130, 0, 65, 204]])
def test_a_workspace_serves_every_call_of_its_shape(dtype, dk, dv, lengths):
    """Rows that are not 16-byte aligned take another path, in the workspace that the aligned ones were sized for, and the other way round."""
    lib = layers._library()
    c = Case(dtype, 1, 399, 2, 4, dk, dv, lengths, seed=30)
    s = Case(dtype, 1, 399, 2, 4, dk, dv, lengths, seed=30)
    s.q, s.k, s.v = (strided(t, 2, 3, 1) for t in (c.q, c.k, c.v))
    stream = torch.cuda.current_stream().cuda_stream
    for name in ("kda_delta_backward_workspace_size", "kda_delta_prefill_workspace_size"):
        sizes = [getattr(lib, name)(ctypes.byref(_args(x))) for x in (c, s)]
        assert sizes[0] == sizes[1], name
        ws = torch.empty(max(16, sizes[0]), dtype=torch.uint8, device=DEV)
        for x in (c, s):
            if "prefill" in name:
                o = torch.empty(*c.shape, 4, dv, dtype=dtype, device=DEV)
                fin = torch.empty_like(c.state)
                assert lib.kda_delta_prefill(ctypes.byref(_args(x)), o.data_ptr(), fin.data_ptr(), ws.data_ptr(), sizes[0], stream) == 0
                x.check_prefill(o, fin)
            else:
                g = dict(zip(GRADS, (torch.empty(t.shape, dtype=FP32, device=DEV) for t in (c.q, c.k, c.v, c.g, c.beta, c.state))))
                grads = layers.DeltaGrads(ctypes.sizeof(layers.DeltaGrads), x.d_o.data_ptr(), x.d_final.data_ptr(),
                                          *(g[n].data_ptr() for n in GRADS))
                assert lib.kda_delta_backward(ctypes.byref(_args(x)), ctypes.byref(grads), ws.data_ptr(), sizes[0], stream) == 0
                x.check_backward(g)
    kda.check_status()


def _filled(*shape, dtype=FP32, scale=1.0, seed=0):
    return torch.empty(*shape, dtype=dtype, device=DEV).normal_(0, scale, generator=torch.Generator(device=DEV).manual_seed(seed))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_of_more_than_2_to_the_31_values(dtype):
    """Outputs, kept states and operands past 2^31 elements: the last head is that of a call with it alone, and so is a head in the middle."""
    T, H = 1400, 12288
    q, k = (_filled(1, T, H, 128, dtype=dtype, scale=128 ** -0.5, seed=s) for s in (31, 32))
    v, do = (_filled(1, T, H, 128, dtype=dtype, seed=s) for s in (33, 34))
    g, beta = -0.1 * torch.rand(1, T, H, device=DEV), 0.9 * torch.rand(1, T, H, device=DEV)
    assert v.numel() > 2 ** 31
    grads = kda.delta_backward(q, k, v, g, beta, do)
    for h in (H - 1, H // 2):
        one = kda.delta_backward(*(t[:, :, h:h + 1].contiguous() for t in (q, k, v, g, beta, do)))
        for name in GRADS:
            got, want = (grads[name][:, h:h + 1] if name == "d_initial_state" else grads[name][:, :, h:h + 1]), one[name]
            if dtype == BF16:
                assert torch.equal(got, want), (name, h)
            else:  # few heads keep their states in chunks, many row by row: each within the header's bound of the exact one
                off = ((got - want).double().norm() / want.double().norm()).item()
                assert off <= 2 * 4e-6, (name, h, off)
    kda.check_status()
    del grads, q, k, v, do, g, beta, one, got, want
    torch.cuda.empty_cache()


def test_norm_gradients_of_more_than_2_to_the_31_values():
    x, dy, z = (_filled(70000, 256, 128, dtype=BF16, seed=s) for s in (35, 36, 37))
    assert x.numel() > 2 ** 31
    g = kda.layer_norm_backward(x, None, dy, gate=z, norm="rms")
    for rows in (slice(-3, None), slice(40000, 40002)):
        one = kda.layer_norm_backward(*(t[rows].contiguous() if t is not None else None for t in (x, None, dy)), gate=z[rows].contiguous(), norm="rms")
        assert torch.equal(g["dx"][rows], one["dx"]) and torch.equal(g["dgate"][rows], one["dgate"])
    del x, dy, z, g, one
    torch.cuda.empty_cache()
