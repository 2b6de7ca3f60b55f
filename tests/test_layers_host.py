"""The operators around the mixer without a GPU: their references' gradients against differences, and every
refusal, found on the host before the device is touched."""

import ctypes

import pytest
import torch

import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers
from gated_delta_rule_56_gb300.build import build

import layers_ref as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
PTR = 1 << 20  # a 16-byte aligned address: never read, every call below is refused or empty


@pytest.fixture(scope="module")
def lib():
    build()
    return layers._library()


def _rand(*shape):
    return torch.randn(*shape, dtype=torch.float64)


def _difference(f, tensors, grads, step=1e-6):
    """Central differences of f along a random direction against the gradients' products with it."""
    for i, (t, g) in enumerate(zip(tensors, grads)):
        d = _rand(*t.shape)
        lo, hi = ([v - step * d if j == i else v for j, v in enumerate(tensors)],
                  [v + step * d if j == i else v for j, v in enumerate(tensors)])
        slope = (f(*hi) - f(*lo)) / (2 * step)
        # rounding of f (1e-16 f / step) and the third-order term (step^2)
        assert abs(slope - (g * d).sum()) <= 1e-7 * (1 + abs(slope)), i


@pytest.mark.parametrize("act,W,T", [(True, 4, 7), (False, 3, 2), (True, 2, 1)])
def test_conv_gradients_against_differences(act, W, T):
    torch.manual_seed(0)
    x, w, b, s, dy, df = _rand(T, 3), _rand(3, W), _rand(3), _rand(W - 1, 3), _rand(T, 3), _rand(W - 1, 3)

    def loss(x, w, b, s):
        y, f = ref.conv(x, w, b, act, s)
        return (dy * y).sum() + (df * f).sum()

    _difference(loss, [x, w, b, s], ref.conv_backward(x, w, b, act, s, dy, df))


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_scan_gradients_against_differences(softplus, gate):
    torch.manual_seed(1)
    T, D, N = 6, 3, 4
    x, dt, B, C, z = _rand(T, D), 0.3 * _rand(T, D).abs(), _rand(T, D, N), _rand(T, D, N), _rand(T, D) if gate else None
    A, skip, h0, dy, df = -_rand(D, N).abs(), _rand(D), _rand(D, N), _rand(T, D), _rand(D, N)

    def loss(x, dt, A, B, C, skip, h0, z=None):
        y, h = ref.scan(x, dt, A, B, C, skip, z, softplus, h0)
        return (dy * y).sum() + (df * h).sum()

    g = ref.scan_backward(x, dt, A, B, C, skip, z, softplus, h0, dy, df)
    _difference(loss, [x, dt, A, B, C, skip, h0] + ([z] if gate else []),
                [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "d_init")] + ([g["dz"]] if gate else []))


@pytest.mark.parametrize("rms,interleaved,half", [(True, False, 8), (False, True, 4), (True, True, 8)])
def test_rotary_gradients_against_differences(rms, interleaved, half):
    torch.manual_seed(2)
    x, w, d, angle = _rand(3, 2, 16), _rand(16), _rand(3, 2, 16), _rand(3, half)

    def loss(x, w):
        return (d * ref.norm_rotary(x, w, angle.cos(), angle.sin(), rms, 1e-6, interleaved)).sum()

    _difference(loss, [x, w], ref.norm_rotary_backward(x, w, angle.cos(), angle.sin(), rms, 1e-6, interleaved, d))


# ---------------------------------------------------------------------- refusals (C ABI) ---


def _conv(**kw):
    a = layers.ConvArgs(struct_size=ctypes.sizeof(layers.ConvArgs), dtype=0, B=2, T=5, C=24, W=4, activation=1, x=PTR, weight=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _scan(**kw):
    a = layers.ScanArgs(struct_size=ctypes.sizeof(layers.ScanArgs), dtype=0, B=2, T=5, D=24, N=16, G=2, dt_softplus=1, x=PTR, dt=PTR,
                        Bm=PTR, Cm=PTR, A=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _rotary(**kw):
    a = layers.RotaryArgs(struct_size=ctypes.sizeof(layers.RotaryArgs), dtype=0, rows=5, q_heads=4, k_heads=2, head=64, half=32,
                          eps=1e-6, q=PTR, k=PTR, cos_table=PTR, sin_table=PTR, positions=PTR, table_rows=9)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


SHARED = [(dict(struct_size=4), INVALID), (dict(struct_size=5000), INVALID), (dict(dtype=2), INVALID), (dict(B=-1), INVALID),
          (dict(T=-1), INVALID), (dict(B=70000, T=70000), INVALID), (dict(x=None), INVALID), (dict(x=PTR + 1), INVALID),
          (dict(x_stride=23), INVALID), (dict(x_stride=-24), INVALID), (dict(cu_seqlens=PTR, n_seqs=1), INVALID),
          (dict(B=1, cu_seqlens=PTR, n_seqs=-1), INVALID), (dict(B=1, cu_seqlens=PTR + 2, n_seqs=1), INVALID),
          (dict(initial_state_indices=PTR, initial_state=PTR), INVALID),  # no pool size
          (dict(initial_state_indices=PTR, state_pool_size=3), INVALID),  # no pool
          (dict(final_state_indices=PTR, state_pool_size=3), INVALID),
          (dict(initial_state_indices=PTR + 1, initial_state=PTR, state_pool_size=3), INVALID)]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(W=0), INVALID), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(C=-1), INVALID), (dict(C=1 << 21), UNSUPPORTED),
    (dict(activation=2), INVALID), (dict(weight=None), INVALID), (dict(weight=PTR + 1), INVALID), (dict(bias=PTR + 1), INVALID)])
def test_conv_refusals(lib, change, status):
    a = _conv(**change)
    assert lib.kda_conv_prefill(ctypes.byref(a), PTR, None, None) == status
    assert kda.last_error() != ""
    if "T" not in change and "cu_seqlens" not in change and "indices" not in "".join(change):
        a.T = 1
        assert lib.kda_conv_decode_step(ctypes.byref(a), PTR, PTR, None) == status
    if "indices" not in "".join(change):
        a.T = change.get("T", 5)
        assert lib.kda_conv_backward(ctypes.byref(a), PTR, None, PTR, PTR, None, None, PTR, 1 << 30, None) == status
        assert lib.kda_conv_backward_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(N=0), INVALID), (dict(N=257), UNSUPPORTED), (dict(G=0), INVALID), (dict(G=5), INVALID), (dict(D=-24), INVALID),
    (dict(D=1 << 17), UNSUPPORTED), (dict(dt=None), INVALID), (dict(Bm=None), INVALID), (dict(Cm=None), INVALID), (dict(A=None), INVALID),
    (dict(A=PTR + 2), INVALID), (dict(B_stride=31), INVALID), (dict(C_stride=31), INVALID), (dict(dt_stride=1), INVALID),
    (dict(z=PTR, z_stride=1), INVALID), (dict(z=PTR + 1), INVALID), (dict(Dskip=PTR + 2), INVALID), (dict(dt_bias=PTR + 2), INVALID)])
def test_scan_refusals(lib, change, status):
    a = _scan(**change)
    assert lib.kda_scan_prefill(ctypes.byref(a), PTR, None, PTR, 1 << 40, None) == status
    assert kda.last_error() != ""
    if "T" not in change and "cu_seqlens" not in change and "indices" not in "".join(change):
        a.T = 1
        assert lib.kda_scan_decode_step(ctypes.byref(a), PTR, PTR, None) == status
    if "indices" not in "".join(change):
        a.T = change.get("T", 5)
        g = layers.ScanGrads(struct_size=ctypes.sizeof(layers.ScanGrads), **{n: PTR for n in ("dy", "dx", "ddt", "dA", "dB", "dC")})
        g.dz, g.dDskip, g.ddt_bias = (PTR if v else None for v in (a.z, a.Dskip, a.dt_bias))
        assert lib.kda_scan_backward(ctypes.byref(a), ctypes.byref(g), PTR, 1 << 40, None) == status
        assert lib.kda_scan_backward_workspace_size(ctypes.byref(a)) == 0


def test_outputs_workspaces_and_decode_arguments_are_checked(lib):
    conv, scan = lib.kda_conv_prefill, lib.kda_scan_prefill
    assert conv(None, PTR, None, None) == INVALID
    assert conv(ctypes.byref(_conv()), None, None, None) == INVALID
    assert conv(ctypes.byref(_conv()), PTR + 1, None, None) == INVALID
    assert conv(ctypes.byref(_conv()), PTR, PTR + 1, None) == INVALID
    assert scan(ctypes.byref(_scan()), None, None, PTR, 1 << 40, None) == INVALID
    assert scan(ctypes.byref(_scan()), PTR, PTR + 2, PTR, 1 << 40, None) == INVALID
    for f, make in ((lib.kda_conv_decode_step, _conv), (lib.kda_scan_decode_step, _scan)):
        assert f(ctypes.byref(make()), PTR, PTR, None) == INVALID  # T != 1
        assert f(ctypes.byref(make(T=1)), None, PTR, None) == INVALID
        assert f(ctypes.byref(make(T=1)), PTR, None, None) == INVALID
        assert f(ctypes.byref(make(T=1, initial_state=PTR)), PTR, PTR, None) == INVALID
        assert f(ctypes.byref(make(T=1, B=1, cu_seqlens=PTR)), PTR, PTR, None) == INVALID
        assert f(ctypes.byref(make(T=1, final_state_indices=PTR, state_pool_size=2)), PTR, PTR, None) == INVALID
    a = _conv()
    need = lib.kda_conv_backward_workspace_size(ctypes.byref(a))
    assert need > 0
    for ws, size in ((None, need), (PTR, need - 1), (PTR + 4, need)):
        assert lib.kda_conv_backward(ctypes.byref(a), PTR, None, PTR, PTR, None, None, ws, size, None) == INVALID
    pool = _conv(initial_state=PTR, initial_state_indices=PTR, state_pool_size=4)
    assert lib.kda_conv_backward(ctypes.byref(pool), PTR, None, PTR, PTR, None, None, PTR, 1 << 30, None) == UNSUPPORTED
    a = _scan()
    full = {n: PTR for n in ("dy", "dx", "ddt", "dA", "dB", "dC")}
    need = lib.kda_scan_backward_workspace_size(ctypes.byref(a))
    assert need > 0
    size = ctypes.sizeof(layers.ScanGrads)
    for ws, n in ((None, need), (PTR, need - 1), (PTR + 4, need)):
        g = layers.ScanGrads(struct_size=size, **full)
        assert lib.kda_scan_backward(ctypes.byref(a), ctypes.byref(g), ws, n, None) == INVALID
    for name in full:
        g = layers.ScanGrads(struct_size=size, **{k: v for k, v in full.items() if k != name})
        assert lib.kda_scan_backward(ctypes.byref(a), ctypes.byref(g), PTR, need, None) == INVALID, name
    for name in ("dz", "dDskip", "ddt_bias"):  # the gradient of an input that is not there
        g = layers.ScanGrads(struct_size=size, **full, **{name: PTR})
        assert lib.kda_scan_backward(ctypes.byref(a), ctypes.byref(g), PTR, need, None) == INVALID, name
    assert lib.kda_scan_backward(ctypes.byref(a), None, PTR, need, None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=0), INVALID), (dict(dtype=7), INVALID), (dict(rows=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(k_heads=1 << 20), INVALID),
    (dict(head=0), INVALID), (dict(head=60), UNSUPPORTED), (dict(head=264), UNSUPPORTED), (dict(half=33), INVALID), (dict(half=-8), INVALID),
    (dict(half=12), UNSUPPORTED), (dict(half=6, interleaved=1), UNSUPPORTED), (dict(norm=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(q=None), INVALID), (dict(k=PTR + 1), INVALID),
    (dict(q_stride=255), INVALID), (dict(q_weight=PTR + 1), INVALID), (dict(cos_table=None), INVALID), (dict(sin_table=PTR + 2), INVALID),
    (dict(positions=None), INVALID), (dict(table_rows=-1), INVALID)])
def test_rotary_refusals(lib, change, status):
    a = _rotary(**change)
    assert lib.kda_qk_norm_rotary(ctypes.byref(a), PTR, PTR, None) == status
    assert kda.last_error() != ""
    assert lib.kda_qk_norm_rotary_backward(ctypes.byref(a), PTR, PTR, PTR, PTR, PTR if a.q_weight else None, None, PTR, 1 << 30, None) == status


def test_rotary_outputs_are_checked(lib):
    a = _rotary()
    assert lib.kda_qk_norm_rotary(ctypes.byref(a), None, PTR, None) == INVALID
    assert lib.kda_qk_norm_rotary(ctypes.byref(a), PTR, PTR + 8, None) == INVALID
    back = lib.kda_qk_norm_rotary_backward
    assert back(ctypes.byref(a), PTR, PTR, PTR, PTR, PTR, None, PTR, 1 << 30, None) == INVALID  # no weight
    w = _rotary(q_weight=PTR)
    assert back(ctypes.byref(w), PTR, PTR, PTR, PTR, None, None, PTR, 1 << 30, None) == INVALID
    assert back(ctypes.byref(w), PTR, PTR, PTR, PTR, PTR, None, None, 0, None) == INVALID


def test_empty_calls_queue_nothing(lib):
    assert lib.kda_conv_prefill(ctypes.byref(_conv(B=0)), None, None, None) == OK
    assert lib.kda_conv_prefill(ctypes.byref(_conv(C=0)), None, None, None) == OK
    assert lib.kda_conv_decode_step(ctypes.byref(_conv(B=0, T=1)), None, None, None) == OK
    assert lib.kda_scan_prefill(ctypes.byref(_scan(B=0)), None, None, None, 0, None) == OK
    assert lib.kda_scan_prefill(ctypes.byref(_scan(D=0)), None, None, None, 0, None) == OK
    assert lib.kda_scan_decode_step(ctypes.byref(_scan(B=0, T=1)), None, None, None) == OK
    assert lib.kda_qk_norm_rotary(ctypes.byref(_rotary(rows=0)), None, None, None) == OK


def test_a_shorter_struct_of_an_older_caller_is_read_as_far_as_it_goes(lib):
    a = _conv(B=0, state_pool_size=-5, final_state_indices=PTR)
    a.struct_size = layers.ConvArgs.initial_state.offset
    assert lib.kda_conv_prefill(ctypes.byref(a), None, None, None) == OK


# ---------------------------------------------------------------- refusals (the binding) ---


def test_the_binding_refuses_host_tensors_and_wrong_types():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.conv_prefill(x, w)
    with pytest.raises(TypeError, match="dtype"):
        kda.conv_prefill(x.half(), w)
    with pytest.raises(ValueError, match="CUDA"):
        kda.scan_prefill(x, x, torch.zeros(8, 4), torch.zeros(1, 4, 1, 4), torch.zeros(1, 4, 1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        kda.qk_norm_rotary(torch.zeros(2, 2, 16), torch.zeros(2, 1, 16))


@pytest.mark.parametrize("make,stride", [
    (lambda: torch.zeros(2, 5, 8), 8), (lambda: torch.zeros(2, 5, 24)[..., 8:16], 24), (lambda: torch.zeros(1, 5, 24)[:, :, :8], 24),
    (lambda: torch.zeros(2, 1, 24)[..., :8], 24), (lambda: torch.zeros(10, 8)[::2].view(1, 5, 8), 16), (lambda: torch.zeros(0, 5, 8), 0), (lambda: torch.zeros(2, 0, 8), 0)])
def test_row_strides(make, stride):
    t = make()
    assert layers._row_stride("x", t, t.dtype, tuple(t.shape), 2, t.device) == stride


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(2, 8, 5).transpose(1, 2), lambda: torch.zeros(2, 6, 8)[:, :5], lambda: torch.zeros(2, 5, 16)[..., ::2],
    lambda: torch.zeros(1, 1, 8).expand(2, 5, 8)])
def test_rows_without_one_distance_are_refused(make):
    t = make()
    with pytest.raises(ValueError):
        layers._row_stride("x", t, t.dtype, tuple(t.shape), 2, t.device)


def test_too_many_groups_are_refused(lib):
    a = _scan(D=65536, G=65536, N=1)
    assert lib.kda_scan_prefill(ctypes.byref(a), PTR, None, PTR, 1 << 40, None) == UNSUPPORTED
