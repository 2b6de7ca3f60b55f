"""The operators around the mixer without a GPU, at the ends of their ranges: what the host refuses."""

import ctypes

import gated_delta_rule_56_gb300 as kda

from test_layers_host import INVALID, OK, PTR, _conv, _scan, lib  # noqa: F401


def test_rows_without_sequences_are_refused(lib):  # noqa: F811
    a = _conv(B=1, cu_seqlens=PTR, n_seqs=0)
    assert lib.kda_conv_prefill(ctypes.byref(a), PTR, None, None) == INVALID
    assert "sequences" in kda.last_error()
    a = _scan(B=1, cu_seqlens=PTR, n_seqs=0)
    assert lib.kda_scan_prefill(ctypes.byref(a), PTR, None, PTR, 1 << 40, None) == INVALID
    assert "sequences" in kda.last_error()
    for a, f in ((_conv(B=1, C=0, cu_seqlens=PTR, n_seqs=0), lambda a: lib.kda_conv_prefill(a, PTR, None, None)),
                 (_scan(B=1, D=0, cu_seqlens=PTR, n_seqs=0), lambda a: lib.kda_scan_prefill(a, PTR, None, None, 0, None))):
        assert f(ctypes.byref(a)) == OK  # no channels: no outputs either
