"""The delta rule with one decay per value head and the layer norm without a GPU: their references' gradients against differences,
and every refusal, found on the host before the device is touched."""

import ctypes

import pytest
import torch

import delta_ref as ref
import gated_delta_rule_56_gb300 as kda
from gated_delta_rule_56_gb300 import layers
from gated_delta_rule_56_gb300.build import build

INVALID, UNSUPPORTED = 1, 2
PTR = 1 << 20  # a 16-byte aligned address: never read, every call below is refused or empty
HUGE = 1 << 50


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


def test_delta_gradients_against_differences():
    torch.manual_seed(0)
    T, H, dk, dv = 7, 2, 4, 3
    q, k, v, g, b, S = _rand(T, H, dk), _rand(T, H, dk), _rand(T, H, dv), -_rand(T, H).abs(), torch.rand(T, H).double(), _rand(H, dk, dv)
    k = k / k.norm(dim=-1, keepdim=True)
    d_o, d_final = _rand(T, H, dv), _rand(H, dk, dv)

    def loss(*x):
        o, last = ref.delta(*x)
        return (d_o * o).sum() + (d_final * last).sum()

    _difference(loss, [q, k, v, g, b, S], ref.delta_backward(q, k, v, g, b, S, d_o, d_final))


@pytest.mark.parametrize("rms,kind", [(False, None), (True, "silu"), (False, "sigmoid")])
def test_layer_norm_gradients_against_differences(rms, kind):
    torch.manual_seed(1)
    x, w, b, dy, ds = _rand(5, 6), _rand(6), _rand(6), _rand(5, 6), _rand(5, 6)
    z = _rand(5, 6) if kind else None

    def loss(x, w, b, z=None):
        y, s = ref.layer_norm(x, w, b, None, z, kind, rms, 1e-6)
        return (dy * y).sum() + (ds * s).sum()

    grads = ref.layer_norm_backward(x, w, b, z, kind, rms, 1e-6, dy, ds)
    _difference(loss, [x, w, b] + ([z] if kind else []), [g for g in grads if g is not None])


# ---------------------------------------------------------------------- refusals (C ABI) ---


def _delta(**kw):
    a = layers.DeltaArgs(struct_size=ctypes.sizeof(layers.DeltaArgs), dtype=0, B=2, T=5, k_heads=2, v_heads=4, dk=128, dv=64, q=PTR,
                         k=PTR, v=PTR, g=PTR, beta=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _delta_grads(**kw):
    g = layers.DeltaGrads(struct_size=ctypes.sizeof(layers.DeltaGrads), **{n: PTR for n in ("d_o", "dq", "dk", "dv", "dg", "dbeta")})
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def _norm(**kw):
    a = layers.LayerNormArgs(struct_size=ctypes.sizeof(layers.LayerNormArgs), dtype=0, rows=5, heads=2, width=24, eps=1e-6, x=PTR,
                             weight=PTR, bias=PTR, z=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=4), INVALID), (dict(struct_size=5000), INVALID), (dict(dtype=2), INVALID), (dict(B=-1), INVALID),
    (dict(T=-1), INVALID), (dict(B=70000, T=70000), INVALID), (dict(k_heads=-1), INVALID), (dict(v_heads=-4), INVALID),
    (dict(k_heads=3), INVALID), (dict(k_heads=0), INVALID), (dict(dk=0), INVALID), (dict(dv=-64), INVALID), (dict(dk=48), UNSUPPORTED),
    (dict(dv=256), UNSUPPORTED), (dict(v_heads=1 << 17), UNSUPPORTED), (dict(B=1 << 20, v_heads=1024), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(beta=None), INVALID),
    (dict(q=PTR + 1), INVALID), (dict(g=PTR + 2), INVALID), (dict(beta=PTR + 2), INVALID), (dict(q_stride=255), INVALID),
    (dict(k_stride=-256), INVALID), (dict(v_stride=255), INVALID), (dict(cu_seqlens=PTR, n_seqs=1), INVALID),
    (dict(B=1, cu_seqlens=PTR, n_seqs=-1), INVALID), (dict(B=1, cu_seqlens=PTR + 2, n_seqs=1), INVALID),
    (dict(initial_state_indices=PTR, initial_state=PTR), INVALID), (dict(initial_state_indices=PTR, state_pool_size=3), INVALID),
    (dict(final_state_indices=PTR, state_pool_size=3), INVALID), (dict(initial_state=PTR + 4), INVALID),
    (dict(initial_state_indices=PTR + 1, initial_state=PTR, state_pool_size=3), INVALID)])
def test_delta_refusals(lib, change, status):
    a = _delta(**change)
    assert lib.kda_delta_prefill(ctypes.byref(a), PTR, None, PTR, HUGE, None) == status
    assert kda.last_error() != ""
    indexed = "indices" in "".join(change)
    if "T" not in change and "cu_seqlens" not in change and not indexed:
        a.T = 1
        assert lib.kda_delta_decode_step(ctypes.byref(a), PTR, PTR, None) == (INVALID if "initial_state" in change else status)
    if not indexed:
        a.T = change.get("T", 5)
        assert lib.kda_delta_backward(ctypes.byref(a), ctypes.byref(_delta_grads()), PTR, HUGE, None) == status
        assert lib.kda_delta_backward_workspace_size(ctypes.byref(a)) == 0


def test_delta_outputs_workspaces_and_decode_arguments_are_checked(lib):
    run = lib.kda_delta_prefill
    assert run(None, PTR, None, None, 0, None) == INVALID
    assert run(ctypes.byref(_delta()), None, None, PTR, HUGE, None) == INVALID
    assert run(ctypes.byref(_delta()), PTR + 2, None, PTR, HUGE, None) == INVALID
    assert run(ctypes.byref(_delta()), PTR, PTR + 4, PTR, HUGE, None) == INVALID
    assert run(ctypes.byref(_delta(B=0)), PTR, None, None, 0, None) == 0
    assert run(ctypes.byref(_delta(v_heads=0)), None, None, None, 0, None) == 0
    assert run(ctypes.byref(_delta(B=1, cu_seqlens=PTR, n_seqs=0)), PTR, None, PTR, HUGE, None) == INVALID  # rows without a sequence
    step = lib.kda_delta_decode_step
    assert step(ctypes.byref(_delta()), PTR, PTR, None) == INVALID  # T != 1
    assert step(ctypes.byref(_delta(T=1)), None, PTR, None) == INVALID
    assert step(ctypes.byref(_delta(T=1)), PTR, None, None) == INVALID
    assert step(ctypes.byref(_delta(T=1)), PTR + 4, PTR, None) == INVALID
    assert step(ctypes.byref(_delta(T=1, initial_state=PTR)), PTR, PTR, None) == INVALID
    assert step(ctypes.byref(_delta(T=1, B=1, cu_seqlens=PTR)), PTR, PTR, None) == INVALID
    assert step(ctypes.byref(_delta(T=1, final_state_indices=PTR, state_pool_size=2)), PTR, PTR, None) == INVALID
    back = lib.kda_delta_backward
    a = _delta()
    need = lib.kda_delta_backward_workspace_size(ctypes.byref(a))
    assert need > 0
    for ws, size in ((None, need), (PTR, need - 1), (PTR + 4, need)):
        assert back(ctypes.byref(a), ctypes.byref(_delta_grads()), ws, size, None) == INVALID
    for name in ("d_o", "dq", "dk", "dv", "dg", "dbeta"):
        assert back(ctypes.byref(a), ctypes.byref(_delta_grads(**{name: None})), PTR, HUGE, None) == INVALID
    for change in (dict(d_o=PTR + 2), dict(dq=PTR + 4), dict(dg=PTR + 2), dict(d_final_state=PTR + 4), dict(d_initial_state=PTR + 4),
                   dict(struct_size=4)):
        assert back(ctypes.byref(a), ctypes.byref(_delta_grads(**change)), PTR, HUGE, None) == INVALID
    assert back(ctypes.byref(a), None, PTR, HUGE, None) == INVALID
    pool = _delta(initial_state=PTR, initial_state_indices=PTR, state_pool_size=4)
    assert back(ctypes.byref(pool), ctypes.byref(_delta_grads()), PTR, HUGE, None) == UNSUPPORTED


@pytest.mark.parametrize("change,status", [
    (dict(struct_size=4), INVALID), (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(heads=-1), INVALID), (dict(width=0), INVALID),
    (dict(width=-3), INVALID), (dict(width=32769), UNSUPPORTED), (dict(rows=1 << 31), INVALID), (dict(rows=1 << 30, heads=2), INVALID),
    (dict(norm=2), INVALID), (dict(activation=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(x=PTR + 1), INVALID), (dict(x_stride=47), INVALID),
    (dict(z_stride=47), INVALID), (dict(z=PTR + 1), INVALID), (dict(weight=PTR + 1), INVALID), (dict(bias=PTR + 1), INVALID)])
def test_layer_norm_refusals(lib, change, status):
    a = _norm(**change)
    assert lib.kda_layer_norm(ctypes.byref(a), PTR, None, None) == status
    assert kda.last_error() != ""
    assert lib.kda_layer_norm_backward(ctypes.byref(a), PTR, None, PTR, PTR, PTR, PTR, PTR, HUGE, None) == status
    assert lib.kda_layer_norm_backward_workspace_size(ctypes.byref(a)) == 0


def test_layer_norm_outputs_are_checked(lib):
    f, b = lib.kda_layer_norm, lib.kda_layer_norm_backward
    assert f(None, PTR, None, None) == INVALID
    assert f(ctypes.byref(_norm()), None, None, None) == INVALID
    assert f(ctypes.byref(_norm()), PTR + 1, None, None) == INVALID
    assert f(ctypes.byref(_norm()), PTR, PTR, None) == INVALID  # a sum without a residual
    assert f(ctypes.byref(_norm(residual=PTR, residual_stride=47)), PTR, PTR, None) == INVALID
    assert f(ctypes.byref(_norm(residual=PTR)), PTR, PTR + 1, None) == INVALID
    assert f(ctypes.byref(_norm(rows=0)), None, None, None) == 0
    good = [PTR, None, PTR, PTR, PTR, PTR, PTR, HUGE, None]  # dy, d_sum, dx, dz, dweight, dbias, workspace
    for i, bad in ((0, None), (0, PTR + 1), (1, PTR + 1), (2, None), (2, PTR + 2), (3, None), (3, PTR + 2), (4, None), (4, PTR + 2), (5, None)):
        args = list(good)
        args[i] = bad
        assert b(ctypes.byref(_norm()), *args) == INVALID, i
    assert b(ctypes.byref(_norm(z=None)), *good) == INVALID  # a gradient without its input
    assert b(ctypes.byref(_norm(weight=None)), *good) == INVALID
    assert b(ctypes.byref(_norm(bias=None)), *good) == INVALID
    assert b(ctypes.byref(_norm(residual=PTR)), *good) == INVALID


# -------------------------------------------------------------------------- refusals (Python) ---


def test_the_binding_refuses_host_tensors_and_unknown_words():
    q, v, g = torch.zeros(1, 2, 1, 32), torch.zeros(1, 2, 2, 32), torch.zeros(1, 2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kda.delta_prefill(q, q, v, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        kda.layer_norm(q)
    with pytest.raises(TypeError, match="dtype"):
        kda.delta_prefill(q.half(), q, v, g, g)
    with pytest.raises(TypeError, match="tensors"):
        kda.layer_norm(None)


@pytest.mark.parametrize("cls", [layers.DeltaArgs, layers.DeltaGrads, layers.LayerNormArgs])
def test_argument_structs_are_as_long_as_they_say(cls):
    """The library reads struct_size bytes: the packed form has them all, and each field where the C struct has it."""
    values = [7 + i for i in range(len(cls._fields_) - 1)]
    packed = layers._packer(cls)(*values)
    assert len(packed) == ctypes.sizeof(cls)
    a = cls.from_buffer_copy(packed)
    assert a.struct_size == ctypes.sizeof(cls)
    assert [getattr(a, name) for name, _ in cls._fields_[1:]] == values


def test_no_value_heads_give_zero_gradients_of_their_key_heads(lib):
    a = _delta(v_heads=0, B=0)
    assert lib.kda_delta_backward(ctypes.byref(a), ctypes.byref(_delta_grads()), None, 0, None) == 0  # no rows either: nothing to clear
    assert lib.kda_delta_backward(ctypes.byref(_delta(v_heads=0)), ctypes.byref(_delta_grads(dq=None)), None, 0, None) == INVALID
