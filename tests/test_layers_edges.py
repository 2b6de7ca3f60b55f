"""The operators around the mixer without a GPU, at the ends of their ranges: what the host refuses, and
the bytes it is handed."""

import ctypes

import pytest

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers

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


@pytest.mark.parametrize("cls", [layers.ConvArgs, layers.ScanArgs, layers.ScanGrads, layers.RotaryArgs])
def test_argument_structs_are_as_long_as_they_say(cls):
    """The library reads struct_size bytes: the packed form has them all, and each field where the C struct has it."""
    values = [7 + i for i in range(len(cls._fields_) - 1)]
    packed = layers._packer(cls)(*values)
    assert len(packed) == ctypes.sizeof(cls)
    a = cls.from_buffer_copy(packed)
    assert a.struct_size == ctypes.sizeof(cls)
    assert [getattr(a, name) for name, _ in cls._fields_[1:]] == values
