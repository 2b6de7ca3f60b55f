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
