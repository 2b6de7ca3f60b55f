"""ctypes binding of the operators around the mixer: the short causal convolution, the selective
state space scan and the norm of q and k with the position rotation.

As in ``_lib``: argument marshalling only. Inputs named as row inputs (x, dt, z, B, C, q, k) may be
slices of a wider projection: their innermost dimensions are dense and their rows lie at one
uniform distance; everything else is contiguous. There is no fallback without the library.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import _check, _check_indices, _DTYPES, _raise_if, load

_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


def _struct(name, fields):
    return type(name, (ctypes.Structure,), {"_fields_": [("struct_size", _sz)] + fields,
                                            "__doc__": f"{name} of include/kda.h."})


ConvArgs = _struct("kda_conv_args", [
    ("dtype", _i), ("B", _i), ("T", _i), ("C", _i), ("W", _i), ("activation", _i), ("x", _vp), ("x_stride", _i64),
    ("weight", _vp), ("bias", _vp), ("cu_seqlens", _vp), ("n_seqs", _i), ("initial_state", _vp),
    ("initial_state_indices", _vp), ("final_state_indices", _vp), ("state_pool_size", _i)])
ScanArgs = _struct("kda_scan_args", [
    ("dtype", _i), ("B", _i), ("T", _i), ("D", _i), ("N", _i), ("G", _i), ("dt_softplus", _i), ("x", _vp), ("dt", _vp),
    ("Bm", _vp), ("Cm", _vp), ("z", _vp), ("x_stride", _i64), ("dt_stride", _i64), ("B_stride", _i64),
    ("C_stride", _i64), ("z_stride", _i64), ("A", _vp), ("Dskip", _vp), ("dt_bias", _vp), ("cu_seqlens", _vp),
    ("n_seqs", _i), ("initial_state", _vp), ("initial_state_indices", _vp), ("final_state_indices", _vp),
    ("state_pool_size", _i)])
ScanGrads = _struct("kda_scan_grads", [(n, _vp) for n in (
    "dy", "d_final_state", "dx", "ddt", "dA", "dB", "dC", "dDskip", "dz", "ddt_bias", "d_initial_state")])
RotaryArgs = _struct("kda_rotary_args", [
    ("dtype", _i), ("rows", _i64), ("q_heads", _i), ("k_heads", _i), ("head", _i), ("half", _i), ("norm", _i),
    ("interleaved", _i), ("eps", ctypes.c_float), ("q", _vp), ("k", _vp), ("q_stride", _i64), ("k_stride", _i64),
    ("q_weight", _vp), ("k_weight", _vp), ("cos_table", _vp), ("sin_table", _vp), ("positions", _vp),
    ("table_rows", _i64)])

_CODES = {_i: "i", _i64: "q", _sz: "N", _vp: "P", ctypes.c_float: "f"}


def _packer(cls):
    """Makes an argument struct from its fields in order (without struct_size; None is a NULL pointer). Packing bytes costs a
    third of filling a ctypes structure, and a token step has little else to do on the host."""
    size = ctypes.sizeof(cls)
    pack = struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0P").pack  # 0P: up to the C struct's end

    def make(*fields):
        return pack(size, *fields)

    return make


_conv_struct, _scan_struct, _rotary_struct = _packer(ConvArgs), _packer(ScanArgs), _packer(RotaryArgs)
_grads_struct = _packer(ScanGrads)

_typed = None


def _library():
    """The library with the argument types of these entry points set."""
    global _typed
    lib = load()
    if _typed is not lib:
        for name, args in (("kda_conv_prefill", [_vp, _vp, _vp, _vp]),
                           ("kda_conv_decode_step", [_vp, _vp, _vp, _vp]),
                           ("kda_conv_backward", [_vp] + [_vp] * 7 + [_sz, _vp]),
                           ("kda_scan_prefill", [_vp, _vp, _vp, _vp, _sz, _vp]),
                           ("kda_scan_decode_step", [_vp, _vp, _vp, _vp]),
                           ("kda_scan_backward", [_vp, _vp, _vp, _sz, _vp]),
                           ("kda_qk_norm_rotary", [_vp, _vp, _vp, _vp]),
                           ("kda_qk_norm_rotary_backward", [_vp] + [_vp] * 7 + [_sz, _vp])):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, _i
        for name, arg in (("kda_conv_backward_workspace_size", ConvArgs), ("kda_scan_prefill_workspace_size", ScanArgs),
                          ("kda_scan_backward_workspace_size", ScanArgs),
                          ("kda_qk_norm_rotary_backward_workspace_size", RotaryArgs)):
            f = getattr(lib, name)
            f.argtypes, f.restype = [_vp], _sz
        _typed = lib
    return lib


def _device(t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("inputs must be torch tensors")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    device = t.device
    if device.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    return device


def _dense(name, t, dtype, shape, device):
    """``_check``, with the common case decided in a few comparisons (these calls run once per token)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device):
        _check(name, t, dtype, shape, device)


def _address(t):
    return 0 if t is None else t.data_ptr()


def _call(device, function, *args):
    """Calls an entry point with the device's current stream behind ``args``, on that device."""
    if device.index == torch.cuda.current_device():
        status = function(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            status = function(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status:
        _raise_if(status)


def _on_device(device, function, arg):
    """A sizing call, which goes by the current device."""
    if device.index == torch.cuda.current_device():
        return function(arg)
    with torch.cuda.device(device):
        return function(arg)


def _row_stride(name, t, dtype, shape, lead, device):
    """Checks an input whose first ``lead`` dimensions are rows; returns the elements between rows."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device:
        if t.numel() == 0:
            return 0
        if t.is_contiguous():
            return shape[-1] if len(shape) == lead + 1 else shape[-1] * shape[-2]
        strides = t.stride()  # a slice of a wider projection
        width = shape[-1]
        if strides[-1] == 1 and (len(shape) == lead + 1 or strides[-2] == width):
            if len(shape) == lead + 2:
                width *= shape[-2]
            if strides[lead - 1] >= width and (lead == 1 or (lead == 2 and strides[0] == strides[1] * shape[1])):
                return strides[lead - 1]
    else:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    strides = t.stride()
    width = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and strides[d] != width:
            raise ValueError(f"{name}: the values of a row must be dense")
        width *= shape[d]
    stride, rows = width, 1
    for d in range(lead - 1, -1, -1):
        if shape[d] != 1:
            if rows == 1:
                stride = strides[d]
            elif strides[d] != stride * rows:
                raise ValueError(f"{name}: rows must lie at one uniform distance")
            rows *= shape[d]
    if rows > 1 and stride < width:
        raise ValueError(f"{name}: rows must not overlap")
    return stride


def _sequences(cu_seqlens, batch, device):
    if cu_seqlens is None:
        return batch
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor [N+1]")
    _dense("cu_seqlens", cu_seqlens, torch.int32, (cu_seqlens.numel(),), device)
    if batch != 1:
        raise ValueError("cu_seqlens needs a batch of 1 (packed rows)")
    return cu_seqlens.numel() - 1


def _states(initial, final, initial_indices, final_indices, n, shape, dtype, device):
    """Checks states of one call (``shape`` is one sequence's) and returns the pool size (0: no pool)."""
    pools = [t.shape[0] for t, i in ((initial, initial_indices), (final, final_indices)) if t is not None and i is not None]
    if len(set(pools)) > 1:
        raise ValueError("initial and final state pools must have the same number of slots")
    if initial_indices is not None and initial is None:
        raise ValueError("initial_state_indices needs initial_state (the pool)")
    if final_indices is not None and final is None:
        raise ValueError("final_state_indices needs final_state (the pool)")
    pool = pools[0] if pools else 0
    _check_indices("initial_state_indices", initial_indices, n, device)
    _check_indices("final_state_indices", final_indices, n, device)
    for name, t, i in (("initial_state", initial, initial_indices), ("final_state", final, final_indices)):
        if t is not None:
            _dense(name, t, dtype, (pool if i is not None else n, *shape), device)
    return pool


def _decode_slots(state, state_indices, final_state_indices, n, device):
    """Checks the slots of a decode call; returns the pool's size (0 without a pool)."""
    if state_indices is None:
        if final_state_indices is not None:
            raise ValueError("final_state_indices needs state_indices")
        return 0
    _check_indices("state_indices", state_indices, n, device)
    _check_indices("final_state_indices", final_state_indices, n, device)
    return state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0


def _output(name, t, like, shape):
    """``t``, or a new dense tensor of the type and device of ``like``."""
    if t is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    _dense(name, t, like.dtype, shape, like.device)
    return t


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# ------------------------------------------------------------------ short convolution ---


def _conv_front(x, weight, bias, activation, lead):
    """Checks the inputs that all calls share; returns the leading fields of their struct, the device, C and W."""
    dev = _device(x)
    if x.dim() != lead + 1:
        raise ValueError(f"x must have {lead + 1} dimensions")
    if activation is not None and activation != "silu":
        raise ValueError(f"unknown activation {activation!r}: None or 'silu'")
    shape, dtype = x.shape, x.dtype
    C = shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [C, W]")
    W = weight.shape[1]
    _dense("weight", weight, dtype, (C, W), dev)
    if bias is not None:
        _dense("bias", bias, dtype, (C,), dev)
    stride = _row_stride("x", x, dtype, shape, lead, dev)
    return (_DTYPES[dtype], shape[0], shape[1] if lead == 2 else 1, C, W, 1 if activation else 0, x.data_ptr(), stride,
            weight.data_ptr(), _address(bias)), dev, C, W


def conv_prefill(x, weight, bias=None, activation="silu", cu_seqlens=None, initial_state=None, output_final_state=True,
                 y=None, final_state=None, initial_state_indices=None, final_state_indices=None):
    """Short causal convolution of whole sequences, one filter per channel.

    x [B, T, C] (rows may be strided), weight [C, W] with W 2 to 4, bias [C] or None, bf16 or fp32:
    y_t = act(bias + sum_j weight[:, j] x_{t-(W-1)+j}) with act SiLU or none, each sequence on its own. With
    ``cu_seqlens`` (int32 [N+1] on the device) B must be 1 and the rows are packed sequences. The state of a
    sequence is its last W-1 inputs [N, W-1, C] in x's dtype; ``initial_state`` None means zeros. With
    ``initial_state_indices`` / ``final_state_indices`` (int32 [N]) the matching state is a pool, as in
    ``prefill``. ``final_state`` may be ``initial_state``'s memory. Returns (y [B, T, C], final_state or None).
    """
    lib = _library()
    front, dev, C, W = _conv_front(x, weight, bias, activation, 2)
    n = _sequences(cu_seqlens, x.shape[0], dev)
    pool = _states(initial_state, final_state, initial_state_indices, final_state_indices, n, (W - 1, C), x.dtype, dev)
    y = _output("y", y, x, x.shape)
    if final_state is None and output_final_state:
        final_state = torch.empty(n, W - 1, C, dtype=x.dtype, device=dev)
    a = _conv_struct(*front, _address(cu_seqlens), n, _address(initial_state), _address(initial_state_indices),
                     _address(final_state_indices), pool)
    _call(dev, lib.kda_conv_prefill, a, y.data_ptr(), _address(final_state))
    return y, final_state


def conv_decode_step(x, weight, state, bias=None, activation="silu", state_indices=None, final_state_indices=None, y=None):
    """One token of the convolution for N sequences: x [N, C]; ``state`` [N, W-1, C] (or a pool with
    ``state_indices`` int32 [N], as in ``decode_step``) is shifted in place. Returns y [N, C]."""
    lib = _library()
    front, dev, C, W = _conv_front(x, weight, bias, activation, 1)
    n = x.shape[0]
    pool = _decode_slots(state, state_indices, final_state_indices, n, dev)
    _dense("state", state, x.dtype, (n if state_indices is None else pool, W - 1, C), dev)
    y = _output("y", y, x, x.shape)
    a = _conv_struct(*front, 0, 0, 0, _address(state_indices), _address(final_state_indices), pool)
    _call(dev, lib.kda_conv_decode_step, a, state.data_ptr(), y.data_ptr())
    return y


def conv_backward(x, weight, dy, bias=None, activation="silu", cu_seqlens=None, initial_state=None, d_final_state=None,
                  want_d_initial_state=True):
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) through ``conv_prefill`` (no pools).
    dy has y's layout and dtype; d_final_state fp32 [N, W-1, C] or None. Returns a dict of fp32 tensors: dx
    [B, T, C], dweight [C, W], dbias [C] (None without a bias), d_initial_state [N, W-1, C] (or None)."""
    lib = _library()
    front, dev, C, W = _conv_front(x, weight, bias, activation, 2)
    n = _sequences(cu_seqlens, x.shape[0], dev)
    _dense("dy", dy, x.dtype, x.shape, dev)
    _states(initial_state, None, None, None, n, (W - 1, C), x.dtype, dev)
    if d_final_state is not None:
        _dense("d_final_state", d_final_state, torch.float32, (n, W - 1, C), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dx=torch.empty(tuple(x.shape), **f32), dweight=torch.empty(C, W, **f32),
               dbias=None if bias is None else torch.empty(C, **f32),
               d_initial_state=torch.empty(n, W - 1, C, **f32) if want_d_initial_state else None)
    a = _conv_struct(*front, _address(cu_seqlens), n, _address(initial_state), 0, 0, 0)
    ws_bytes = _on_device(dev, lib.kda_conv_backward_workspace_size, a)
    ws = _workspace(ws_bytes, dev)
    _call(dev, lib.kda_conv_backward, a, dy.data_ptr(), _address(d_final_state),
          *(_address(out[k]) for k in ("dx", "dweight", "dbias", "d_initial_state")), _address(ws), ws_bytes)
    return out


# -------------------------------------------------------------- selective state space ---


def _scan_front(x, dt, A, B, C, D, z, dt_bias, dt_softplus, lead):
    """Checks the inputs that all calls share; returns the leading fields of their struct, the device, channels, N and G."""
    dev = _device(x)
    if x.dim() != lead + 1:
        raise ValueError(f"x must have {lead + 1} dimensions")
    shape, dtype = x.shape, x.dtype
    ch = shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a tensor [D, N]")
    N = A.shape[1]
    if not isinstance(B, torch.Tensor) or B.dim() != lead + 2:
        raise ValueError(f"B must have {lead + 2} dimensions")
    G = B.shape[-2]
    small = shape[:-1] + (G, N)
    x_stride = _row_stride("x", x, dtype, shape, lead, dev)
    dt_stride = _row_stride("dt", dt, dtype, shape, lead, dev)
    B_stride = _row_stride("B", B, dtype, small, lead, dev)
    C_stride = _row_stride("C", C, dtype, small, lead, dev)
    z_stride = 0 if z is None else _row_stride("z", z, dtype, shape, lead, dev)
    _dense("A", A, torch.float32, (ch, N), dev)
    if D is not None:
        _dense("D", D, torch.float32, (ch,), dev)
    if dt_bias is not None:
        _dense("dt_bias", dt_bias, torch.float32, (ch,), dev)
    return (_DTYPES[dtype], shape[0], shape[1] if lead == 2 else 1, ch, N, G, 1 if dt_softplus else 0, x.data_ptr(), dt.data_ptr(),
            B.data_ptr(), C.data_ptr(), _address(z), x_stride, dt_stride, B_stride, C_stride, z_stride, A.data_ptr(), _address(D),
            _address(dt_bias)), dev, ch, N, G


def scan_prefill(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, cu_seqlens=None, initial_state=None,
                 output_final_state=True, y=None, final_state=None, initial_state_indices=None, final_state_indices=None):
    """Selective state space scan of whole sequences.

    x, dt, z [B, T, D] and B, C [B, T, G, N], bf16 or fp32, rows may be strided; A [D, N] (negative for a decay), D
    and dt_bias [D], fp32. With dt' = softplus(dt + dt_bias) (or dt + dt_bias), per channel c of group g:
    h_t = exp(dt'_t A) h_{t-1} + dt'_t x_t B_t,  y_t = sum_n C_t h_t + D x_t, times z_t sigmoid(z_t) with a gate.
    ``cu_seqlens``, states (fp32 [N_seqs, D, N]) and pools as in ``prefill``. Returns (y [B, T, D], final_state or None).
    """
    lib = _library()
    front, dev, ch, N, _ = _scan_front(x, dt, A, B, C, D, z, dt_bias, dt_softplus, 2)
    n = _sequences(cu_seqlens, x.shape[0], dev)
    pool = _states(initial_state, final_state, initial_state_indices, final_state_indices, n, (ch, N), torch.float32, dev)
    y = _output("y", y, x, x.shape)
    if final_state is None and output_final_state:
        final_state = torch.empty(n, ch, N, dtype=torch.float32, device=dev)
    a = _scan_struct(*front, _address(cu_seqlens), n, _address(initial_state), _address(initial_state_indices),
                     _address(final_state_indices), pool)
    ws_bytes = _on_device(dev, lib.kda_scan_prefill_workspace_size, a)
    ws = _workspace(ws_bytes, dev)
    _call(dev, lib.kda_scan_prefill, a, y.data_ptr(), _address(final_state), _address(ws), ws_bytes)
    return y, final_state


def scan_decode_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, state_indices=None,
                     final_state_indices=None, y=None):
    """One token of the scan for N sequences: x, dt, z [N, D], B, C [N, G, N_states]; ``state`` fp32
    [N, D, N_states] (or a pool with ``state_indices`` int32 [N]) is updated in place. Returns y [N, D]."""
    lib = _library()
    front, dev, ch, N, _ = _scan_front(x, dt, A, B, C, D, z, dt_bias, dt_softplus, 1)
    n = x.shape[0]
    pool = _decode_slots(state, state_indices, final_state_indices, n, dev)
    _dense("state", state, torch.float32, (n if state_indices is None else pool, ch, N), dev)
    y = _output("y", y, x, x.shape)
    a = _scan_struct(*front, 0, 0, 0, _address(state_indices), _address(final_state_indices), pool)
    _call(dev, lib.kda_scan_decode_step, a, state.data_ptr(), y.data_ptr())
    return y


def scan_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, dt_softplus=True, cu_seqlens=None, initial_state=None,
                  d_final_state=None, want_d_initial_state=True):
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) through ``scan_prefill`` (no pools). Returns a
    dict of fp32 tensors shaped like their inputs: dx, ddt, dA, dB, dC, dD, dz, ddt_bias (the last three None
    without their input) and d_initial_state [N_seqs, D, N] (or None)."""
    lib = _library()
    front, dev, ch, N, G = _scan_front(x, dt, A, B, C, D, z, dt_bias, dt_softplus, 2)
    n = _sequences(cu_seqlens, x.shape[0], dev)
    _dense("dy", dy, x.dtype, x.shape, dev)
    _states(initial_state, None, None, None, n, (ch, N), torch.float32, dev)
    if d_final_state is not None:
        _dense("d_final_state", d_final_state, torch.float32, (n, ch, N), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    rows = tuple(x.shape[:-1])
    out = dict(dx=torch.empty(*rows, ch, **f32), ddt=torch.empty(*rows, ch, **f32), dA=torch.empty(ch, N, **f32),
               dB=torch.empty(*rows, G, N, **f32), dC=torch.empty(*rows, G, N, **f32),
               dD=None if D is None else torch.empty(ch, **f32), dz=None if z is None else torch.empty(*rows, ch, **f32),
               ddt_bias=None if dt_bias is None else torch.empty(ch, **f32),
               d_initial_state=torch.empty(n, ch, N, **f32) if want_d_initial_state else None)
    a = _scan_struct(*front, _address(cu_seqlens), n, _address(initial_state), 0, 0, 0)
    g = _grads_struct(dy.data_ptr(), _address(d_final_state),
                      *(_address(out[k]) for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state")))
    ws_bytes = _on_device(dev, lib.kda_scan_backward_workspace_size, a)
    ws = _workspace(ws_bytes, dev)
    _call(dev, lib.kda_scan_backward, a, g, _address(ws), ws_bytes)
    return out


# ------------------------------------------------------------------- norm and rotation ---


def _rotary_args(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved):
    dev = _device(q)
    lead = q.dim() - 2
    if lead < 0 or not isinstance(k, torch.Tensor) or k.dim() != lead + 2:
        raise ValueError("q and k must be tensors [..., heads, head] with the same rows")
    if norm != "rms" and norm != "l2":
        raise ValueError(f"unknown norm {norm!r}: 'rms' or 'l2'")
    dtype, q_shape, k_shape = q.dtype, q.shape, k.shape
    rows, head = q_shape[:-2], q_shape[-1]
    q_stride = _row_stride("q", q, dtype, q_shape, lead, dev)
    k_stride = _row_stride("k", k, dtype, rows + (k_shape[-2], head), lead, dev)
    if q_weight is not None:
        _dense("q_weight", q_weight, dtype, (head,), dev)
    if k_weight is not None:
        _dense("k_weight", k_weight, dtype, (head,), dev)
    half = table_rows = 0
    if cos is not None or sin is not None or positions is not None:
        if cos is None or sin is None or positions is None:
            raise ValueError("cos, sin and positions are given together or not at all")
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a tensor [table rows, rotated pairs]")
        table = cos.shape
        table_rows, half = table
        _dense("cos", cos, torch.float32, table, dev)
        _dense("sin", sin, torch.float32, table, dev)
        _dense("positions", positions, torch.int32, rows, dev)
    return _rotary_struct(_DTYPES[dtype], rows.numel(), q_shape[-2], k_shape[-2], head, half, 0 if norm == "rms" else 1,
                          1 if interleaved else 0, eps, q.data_ptr(), k.data_ptr(), q_stride, k_stride, _address(q_weight),
                          _address(k_weight), _address(cos), _address(sin), _address(positions), table_rows), dev


def qk_norm_rotary(q, k, cos=None, sin=None, positions=None, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
                   interleaved=False, q_out=None, k_out=None):
    """Norm of every head's row of q and k, then the position rotation, in one pass.

    q [..., Hq, d], k [..., Hk, d] (bf16 or fp32; the leading dimensions are tokens, whose rows may be strided),
    weights [d] or None (ones). norm "rms": x weight / sqrt(mean(x^2) + eps); "l2": x weight / sqrt(sum(x^2) + eps), the
    unit rows ``prefill`` takes. cos, sin fp32 [P, pairs]: line positions[token] (int32) turns the first 2 * pairs
    values, paired as halves (i, pairs + i), or as (2i, 2i + 1) with ``interleaved``. Without tables there is no
    rotation. Returns dense (q_out, k_out)."""
    lib = _library()
    a, dev = _rotary_args(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved)
    q_out = _output("q_out", q_out, q, q.shape)
    k_out = _output("k_out", k_out, q, k.shape)
    _call(dev, lib.kda_qk_norm_rotary, a, q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rotary_backward(q, k, cos, sin, positions, dq_out, dk_out, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
                            interleaved=False):
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) through ``qk_norm_rotary``: a dict of fp32 tensors dq, dk,
    dq_weight, dk_weight (None without the weight). dq_out, dk_out have the outputs' layout and dtype."""
    lib = _library()
    a, dev = _rotary_args(q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved)
    _dense("dq_out", dq_out, q.dtype, q.shape, dev)
    _dense("dk_out", dk_out, q.dtype, k.shape, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty(tuple(q.shape), **f32), dk=torch.empty(tuple(k.shape), **f32),
               dq_weight=None if q_weight is None else torch.empty(q.shape[-1], **f32),
               dk_weight=None if k_weight is None else torch.empty(q.shape[-1], **f32))
    ws_bytes = _on_device(dev, lib.kda_qk_norm_rotary_backward_workspace_size, a)
    ws = _workspace(ws_bytes, dev)
    _call(dev, lib.kda_qk_norm_rotary_backward, a, dq_out.data_ptr(), dk_out.data_ptr(),
          *(_address(out[n]) for n in ("dq", "dk", "dq_weight", "dk_weight")), _address(ws), ws_bytes)
    return out
