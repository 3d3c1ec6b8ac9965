"""The layer operators of ``include/gdp_layer.h`` over torch tensors: the gated linear recurrence
(packed sequences, backward, one-token step) and the grouped norm with an activated gate, with its
8-bit activation checkpoints.  Argument checks and marshalling only; torch supplies device memory and
the current stream, and there is no fallback: without the library every call raises.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import binding
from .binding import (GDP_DTYPE_BF16, GDP_DTYPE_F16, GDP_DTYPE_F32, GDP_ERR_INVALID_ARG, GDP_ERR_UNSUPPORTED,
                      GDP_OK, GdpError)

GDP_GATE_LOG, GDP_GATE_ALPHA, GDP_GATE_SIGMOID = range(3)
GDP_ACT_NONE, GDP_ACT_SILU, GDP_ACT_SIGMOID = range(3)
CHECKPOINT_BLOCK = 128  # channels that share one scale of an 8-bit checkpoint
_GATES = {"log": GDP_GATE_LOG, "alpha": GDP_GATE_ALPHA, "sigmoid": GDP_GATE_SIGMOID}
_ACTS = {None: GDP_ACT_NONE, "silu": GDP_ACT_SILU, "sigmoid": GDP_ACT_SIGMOID}
_TYPES = {torch.bfloat16: GDP_DTYPE_BF16, torch.float16: GDP_DTYPE_F16, torch.float32: GDP_DTYPE_F32}
_vp, _i64, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class GdpRecurrenceArgs(ctypes.Structure):
    """Mirror of ``gdp_recurrence_args``."""
    _fields_ = [
        ("x", _vp), ("x_stride_t", _i64), ("g", _vp), ("g_stride_t", _i64), ("output", _vp), ("cu_seqlens", _vp),
        ("T", _i64), ("N", _i64), ("C", _i64), ("initial_state", _vp), ("output_state", _vp), ("state", _vp),
        ("state_indices", _vp), ("num_slots", _i64), ("device_status", _vp), ("cu_seqlens_int64", _int), ("x_dtype", _int), ("g_dtype", _int), ("gate", _int),
    ]


class GdpRecurrenceBackwardArgs(ctypes.Structure):
    """Mirror of ``gdp_recurrence_backward_args``."""
    _fields_ = [
        ("g", _vp), ("g_stride_t", _i64), ("x", _vp), ("x_stride_t", _i64), ("h", _vp), ("h_stride_t", _i64),
        ("h_codes", _vp), ("h_scales", _vp), ("h_group", _i64), ("d_output", _vp), ("d_output_stride_t", _i64),
        ("cu_seqlens", _vp), ("T", _i64), ("N", _i64), ("C", _i64), ("initial_state", _vp), ("d_final_state", _vp),
        ("dx", _vp), ("dg", _vp), ("d_initial_state", _vp), ("device_status", _vp), ("cu_seqlens_int64", _int), ("x_dtype", _int), ("g_dtype", _int), ("gate", _int),
    ]


class GdpGroupNormArgs(ctypes.Structure):
    """Mirror of ``gdp_group_norm_args``."""
    _fields_ = [
        ("o", _vp), ("o_stride_t", _i64), ("o_stride_h", _i64), ("z", _vp), ("z_stride_t", _i64),
        ("z_stride_h", _i64), ("weight", _vp), ("bias", _vp), ("y", _vp), ("o_codes", _vp), ("o_scales", _vp),
        ("z_codes", _vp), ("z_scales", _vp), ("T", _i64), ("H", _i64), ("D", _i64), ("eps", _f32), ("dtype", _int),
        ("center", _int), ("per_head", _int), ("activation", _int),
    ]


class GdpGroupNormBackwardArgs(ctypes.Structure):
    """Mirror of ``gdp_group_norm_backward_args``."""
    _fields_ = [
        ("d_y", _vp), ("d_y_stride_t", _i64), ("d_y_stride_h", _i64), ("o", _vp), ("o_stride_t", _i64),
        ("o_stride_h", _i64), ("z", _vp), ("z_stride_t", _i64), ("z_stride_h", _i64), ("o_codes", _vp),
        ("o_scales", _vp), ("z_codes", _vp), ("z_scales", _vp), ("weight", _vp), ("bias", _vp), ("d_o", _vp),
        ("d_z", _vp), ("d_weight", _vp), ("d_bias", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("T", _i64),
        ("H", _i64), ("D", _i64), ("eps", _f32), ("dtype", _int), ("center", _int), ("per_head", _int),
        ("activation", _int),
    ]


class ActivationCheckpoint(NamedTuple):
    """8-bit codes [T, H, D] of an activation and the scales [T, H, ceil(D / 128)] of their blocks."""
    codes: torch.Tensor
    scales: torch.Tensor

    def dequantize(self) -> torch.Tensor:
        """The fp32 values that the codes stand for, [T, H, D]."""
        d = self.codes.shape[-1]
        return self.codes.float() * self.scales.repeat_interleave(CHECKPOINT_BLOCK, -1)[..., :d]


class GroupNormCheckpoint(NamedTuple):
    """What gated_group_norm keeps for its backward pass: the norm's input and, with a gate, z."""
    o: ActivationCheckpoint
    z: Optional[ActivationCheckpoint]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = binding.load_library()
        for name, args in (("gdp_linear_recurrence", GdpRecurrenceArgs),
                           ("gdp_linear_recurrence_decode", GdpRecurrenceArgs),
                           ("gdp_linear_recurrence_backward", GdpRecurrenceBackwardArgs),
                           ("gdp_group_norm", GdpGroupNormArgs),
                           ("gdp_group_norm_backward", GdpGroupNormBackwardArgs)):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = _int, [ctypes.POINTER(args), _vp]
        lib.gdp_group_norm_workspace_bytes.restype = _sz
        lib.gdp_group_norm_workspace_bytes.argtypes = [_i64, _i64, _i64, _int]
        lib.gdp_layer_args_size.restype = _sz
        lib.gdp_layer_args_size.argtypes = [_int]
        for i, args in enumerate((GdpRecurrenceArgs, GdpRecurrenceBackwardArgs, GdpGroupNormArgs,
                                  GdpGroupNormBackwardArgs)):
            if lib.gdp_layer_args_size(i) != ctypes.sizeof(args):
                raise RuntimeError(f"{args.__name__} layout mismatch between the binding and the library")
        _lib = lib
    return _lib


def gdp_group_norm_workspace_bytes(T: int, H: int, D: int, per_head: bool = False) -> int:
    return int(_library().gdp_group_norm_workspace_bytes(T, H, D, int(per_head)))


def _call(name, args, stream):
    lib = _library()
    st = getattr(lib, name)(ctypes.byref(args), ctypes.c_void_p(binding._stream(stream)))
    if st != GDP_OK:
        raise GdpError(st, lib.gdp_last_error().decode())


def _invalid(msg):
    raise GdpError(GDP_ERR_INVALID_ARG, msg)


def _rows(name, t, shape, dtype, dev):
    """A [T, C] or [T, H, D] tensor whose last dimension is contiguous."""
    if t.shape != shape:
        _invalid(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.dtype != dtype:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"{name} must be {dtype} (got {t.dtype})")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        _invalid(f"{name} must be contiguous in its last dimension")
    if t.device != dev:
        _invalid(f"{name} must be on {dev}")


def _dense(name, t, shape, dtype, dev):
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != dev:
        _invalid(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def _device(t):
    if not t.is_cuda:
        _invalid("the tensors must be on a CUDA device")
    return t.device


def _types(x, g):
    if x.dtype not in _TYPES:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"x must be bfloat16, float16 or float32 (got {x.dtype})")
    if g.dtype != x.dtype and g.dtype != torch.float32:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"g must be float32 or of x's type (got {g.dtype})")
    return _TYPES[x.dtype], _TYPES[g.dtype]


def _cu(cu_seqlens, dev):
    if cu_seqlens is None:
        _invalid("cu_seqlens is required (packed input only)")
    if (cu_seqlens.dtype not in (torch.int32, torch.int64) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
            or not cu_seqlens.is_contiguous() or cu_seqlens.device != dev):
        _invalid("cu_seqlens must be a contiguous int32 or int64 vector of N + 1 entries on the tensors' device")
    return cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(cu_seqlens.dtype == torch.int64)


def _status(t, dev):
    if t is None:
        return None
    if t.numel() < 1 or t.element_size() != 4 or t.device != dev:
        _invalid("device_status must be a 32-bit word on the tensors' device")
    return t.data_ptr()


def _workspace(ws, nbytes, dev, stream):
    """The caller's workspace, or a new one (kept from reuse until `stream` has passed the call)."""
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if stream is not None:
            ws.record_stream(torch.cuda.ExternalStream(stream, device=dev))
    elif ws.device != dev or not ws.is_contiguous():
        _invalid("workspace must be contiguous and on the tensors' device")
    return ws, ws.numel() * ws.element_size()


def _gate_code(gate):
    if gate not in _GATES:
        _invalid(f"gate must be one of {sorted(_GATES)} (got {gate!r})")
    return _GATES[gate]


def _state_args(initial_state, output_state, state, state_indices, N, C, dev):
    f32 = torch.float32
    if state is None:
        return (_dense("initial_state", initial_state, (N, C), f32, dev),
                _dense("output_state", output_state, (N, C), f32, dev), None, None, 0)
    if initial_state is not None or output_state is not None:
        _invalid("the state cache excludes initial_state and output_state")
    if state_indices is None or state.dim() != 2:
        _invalid("the state cache is [num_slots, C] and needs state_indices")
    return (None, None, _dense("state", state, (state.shape[0], C), f32, dev),
            _dense("state_indices", state_indices, (N,), torch.int32, dev), state.shape[0])


def gated_linear_recurrence(x, g, cu_seqlens, gate="log", initial_state=None, output_final_state=False, state=None,
                            state_indices=None, output=None, output_state=None, device_status=None, stream=None):
    """h_t = a_t h_{t-1} + b_t along every packed sequence, per channel (gdp_linear_recurrence).

    x [T, C] bf16, f16 or fp32; g [T, C] fp32 or x's type; rows may be strided (slices of a wider
    projection).  ``gate``: "log" a = exp(g), b = x; "alpha" a = g, b = x; "sigmoid" a = sigmoid(g),
    b = (1 - a) x.  cu_seqlens [N + 1] int32 / int64.  initial_state [N, C] fp32 (None: zero), or the
    cache ``state`` [num_slots, C] fp32 read and written in place at ``state_indices`` [N] int32 (-1:
    from zero, nothing written).  Returns ``h`` [T, C] in x's type, or ``(h, final_state)`` when
    output_final_state (dense mode; None in cache mode)."""
    if x.dim() != 2:
        _invalid("x must be [T, C]")
    T, C = x.shape
    dev = _device(x)
    xt, gt = _types(x, g)
    _rows("x", x, x.shape, x.dtype, dev)
    _rows("g", g, x.shape, g.dtype, dev)
    cu, N, cu64 = _cu(cu_seqlens, dev)
    if output is None:
        output = torch.empty((T, C), dtype=x.dtype, device=dev)
    if output_final_state and state is None and output_state is None:
        output_state = torch.empty((N, C), dtype=torch.float32, device=dev)
    init, fin, cache, slots, num = _state_args(initial_state, output_state, state, state_indices, N, C, dev)
    a = GdpRecurrenceArgs(x.data_ptr(), x.stride(0), g.data_ptr(), g.stride(0),
                          _dense("output", output, (T, C), x.dtype, dev), cu, T, N, C, init, fin, cache, slots, num,
                          _status(device_status, dev), cu64, xt, gt, _gate_code(gate))
    _call("gdp_linear_recurrence", a, stream)
    return (output, output_state) if output_final_state else output


def gated_linear_recurrence_decode(x, g, gate="log", initial_state=None, output_final_state=False, state=None,
                                   state_indices=None, output=None, output_state=None, device_status=None,
                                   stream=None):
    """One token per sequence: x, g [N, C]; the state modes, types and gates of gated_linear_recurrence.
    Returns ``h`` [N, C], or ``(h, final_state)`` when output_final_state (dense mode)."""
    if x.dim() != 2:
        _invalid("x must be [N, C]")
    N, C = x.shape
    dev = _device(x)
    xt, gt = _types(x, g)
    _rows("x", x, x.shape, x.dtype, dev)
    _rows("g", g, x.shape, g.dtype, dev)
    if output is None:
        output = torch.empty((N, C), dtype=x.dtype, device=dev)
    if output_final_state and state is None and output_state is None:
        output_state = torch.empty((N, C), dtype=torch.float32, device=dev)
    init, fin, cache, slots, num = _state_args(initial_state, output_state, state, state_indices, N, C, dev)
    a = GdpRecurrenceArgs(x.data_ptr(), x.stride(0), g.data_ptr(), g.stride(0),
                          _dense("output", output, (N, C), x.dtype, dev), None, N, N, C, init, fin, cache, slots, num,
                          _status(device_status, dev), 0, xt, gt, _gate_code(gate))
    _call("gdp_linear_recurrence_decode", a, stream)
    return (output, output_state) if output_final_state else output


def gated_linear_recurrence_backward(g, h, d_output, cu_seqlens, gate="log", x=None, initial_state=None,
                                     d_final_state=None, device_status=None, stream=None):
    """Gradients of gated_linear_recurrence for dL/dh = ``d_output`` [T, C] and dL/dfinal =
    ``d_final_state`` [N, C] fp32 (or None).  ``h``: the forward's output [T, C] in d_output's type, or
    the ActivationCheckpoint of it that gated_group_norm kept ([T, H, D] with H D = C).  ``x`` is needed
    for the sigmoid gate only.  Returns a dict: dx in d_output's type, dg in g's type, d_initial_state
    fp32 (None without an initial state)."""
    if d_output.dim() != 2:
        _invalid("d_output must be [T, C]")
    T, C = d_output.shape
    dev = _device(d_output)
    xt, gt = _types(d_output, g)
    _rows("d_output", d_output, d_output.shape, d_output.dtype, dev)
    _rows("g", g, d_output.shape, g.dtype, dev)
    gate = _gate_code(gate)
    xp = xs = 0
    if gate == GDP_GATE_SIGMOID:
        if x is None:
            _invalid("the sigmoid gate's gradient needs x")
        _rows("x", x, d_output.shape, d_output.dtype, dev)
        xp, xs = x.data_ptr(), x.stride(0)
    hp = hs = codes = scales = group = 0
    if isinstance(h, ActivationCheckpoint):
        if h.codes.dim() != 3 or h.codes.shape[0] != T or h.codes.shape[1] * h.codes.shape[2] != C:
            _invalid("the checkpoint of h must be [T, H, D] with H D = C")
        codes, scales, group = _checkpoint("h", h, h.codes.shape, dev) + (h.codes.shape[2],)
    else:
        _rows("h", h, d_output.shape, d_output.dtype, dev)
        hp, hs = h.data_ptr(), h.stride(0)
    cu, N, cu64 = _cu(cu_seqlens, dev)
    init = _dense("initial_state", initial_state, (N, C), torch.float32, dev)
    dfin = _dense("d_final_state", d_final_state, (N, C), torch.float32, dev)
    out = {"dx": torch.empty((T, C), dtype=d_output.dtype, device=dev),
           "dg": torch.empty((T, C), dtype=g.dtype, device=dev),
           "d_initial_state": (torch.empty((N, C), dtype=torch.float32, device=dev)
                               if initial_state is not None else None)}
    dinit = out["d_initial_state"]
    a = GdpRecurrenceBackwardArgs(
        g.data_ptr(), g.stride(0), xp, xs, hp, hs, codes, scales, group, d_output.data_ptr(), d_output.stride(0), cu,
        T, N, C, init, dfin, out["dx"].data_ptr(), out["dg"].data_ptr(), None if dinit is None else dinit.data_ptr(),
        _status(device_status, dev), cu64, xt, gt, gate)
    _call("gdp_linear_recurrence_backward", a, stream)
    return out


def _checkpoint(name, c, shape, dev):
    """Addresses of a checkpoint's codes and scales for an activation of `shape` [T, H, D]."""
    T, H, D = shape
    return (_dense(f"{name}'s codes", c.codes, (T, H, D), torch.int8, dev),
            _dense(f"{name}'s scales", c.scales, (T, H, -(-D // CHECKPOINT_BLOCK)), torch.float32, dev))


def _new_checkpoint(T, H, D, dev):
    return ActivationCheckpoint(torch.empty((T, H, D), dtype=torch.int8, device=dev),
                                torch.empty((T, H, -(-D // CHECKPOINT_BLOCK)), dtype=torch.float32, device=dev))


def _affine(weight, bias, H, D, dev):
    """(weight, bias, per_head): fp32 [D] or [H, D]."""
    if weight.dim() == 2 and weight.shape == (H, D):
        per_head = 1
    elif weight.shape == (D,):
        per_head = 0
    else:
        _invalid(f"weight must be [{D}] or [{H}, {D}] (got {tuple(weight.shape)})")
    return (_dense("weight", weight, weight.shape, torch.float32, dev),
            _dense("bias", bias, weight.shape, torch.float32, dev), per_head)


def _act_code(activation):
    if activation not in _ACTS:
        _invalid(f"activation must be 'silu', 'sigmoid' or None (got {activation!r})")
    return _ACTS[activation]


def gated_group_norm(o, weight, z=None, bias=None, eps=1e-5, center=False, activation="silu", save_checkpoint=False,
                     output=None, stream=None):
    """y = (n weight + bias) act(z) with n the norm of o [T, H, D] over each (token, head)'s D channels:
    RMS, or mean and variance when ``center`` (gdp_group_norm).  ``activation`` "silu" or "sigmoid" of z
    [T, H, D]; without z, "silu" of the affine norm itself, or None.  o and z bf16, f16 or fp32 (one
    type, token and head strides free); weight and bias fp32, [D] or one row per head [H, D].

    Returns ``y`` [T, H, D] in o's type, or ``(y, checkpoint)`` with the GroupNormCheckpoint (8-bit
    codes of o and z) that gated_group_norm_backward takes when ``save_checkpoint``."""
    if o.dim() != 3:
        _invalid("o must be [T, H, D]")
    T, H, D = o.shape
    dev = _device(o)
    if o.dtype not in _TYPES:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"o must be bfloat16, float16 or float32 (got {o.dtype})")
    _rows("o", o, o.shape, o.dtype, dev)
    zp = zt = zh = 0
    if z is not None:
        _rows("z", z, o.shape, o.dtype, dev)
        zp, zt, zh = z.data_ptr(), z.stride(0), z.stride(1)
    w, b, per_head = _affine(weight, bias, H, D, dev)
    if output is None:
        output = torch.empty((T, H, D), dtype=o.dtype, device=dev)
    kept, ptrs = None, (None, None, None, None)
    if save_checkpoint:
        kept = GroupNormCheckpoint(_new_checkpoint(T, H, D, dev), _new_checkpoint(T, H, D, dev) if z is not None else None)
        ptrs = (kept.o.codes.data_ptr(), kept.o.scales.data_ptr())
        ptrs += (kept.z.codes.data_ptr(), kept.z.scales.data_ptr()) if z is not None else (None, None)
    a = GdpGroupNormArgs(o.data_ptr(), o.stride(0), o.stride(1), zp, zt, zh, w, b,
                         _dense("output", output, (T, H, D), o.dtype, dev), *ptrs, T, H, D, eps, _TYPES[o.dtype],
                         int(bool(center)), per_head, _act_code(activation))
    _call("gdp_group_norm", a, stream)
    return (output, kept) if save_checkpoint else output


def gated_group_norm_backward(d_output, saved, weight, bias=None, eps=1e-5, center=False, activation="silu",
                              workspace=None, stream=None):
    """Gradients of gated_group_norm for dL/dy = ``d_output`` [T, H, D].  ``saved``: the
    GroupNormCheckpoint of the forward call, or the pair ``(o, z)`` of tensors (z None without a gate).
    Returns a dict: do and dz in d_output's type (dz None without z), dweight and dbias fp32 (None
    without a bias)."""
    if d_output.dim() != 3:
        _invalid("d_output must be [T, H, D]")
    T, H, D = d_output.shape
    dev = _device(d_output)
    if d_output.dtype not in _TYPES:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"d_output must be bfloat16, float16 or float32 (got {d_output.dtype})")
    _rows("d_output", d_output, d_output.shape, d_output.dtype, dev)
    o, z = saved
    tensors, codes = [0] * 6, [None] * 4
    if isinstance(saved, GroupNormCheckpoint):
        codes[:2] = _checkpoint("o", o, d_output.shape, dev)
        if z is not None:
            codes[2:] = _checkpoint("z", z, d_output.shape, dev)
    else:
        for i, (name, t) in enumerate((("o", o), ("z", z))):
            if t is not None:
                _rows(name, t, d_output.shape, d_output.dtype, dev)
                tensors[3 * i:3 * i + 3] = t.data_ptr(), t.stride(0), t.stride(1)
    w, b, per_head = _affine(weight, bias, H, D, dev)
    like = dict(dtype=d_output.dtype, device=dev)
    out = {"do": torch.empty((T, H, D), **like), "dz": torch.empty((T, H, D), **like) if z is not None else None,
           "dweight": torch.empty_like(weight), "dbias": torch.empty_like(bias) if bias is not None else None}
    ws, ws_bytes = _workspace(workspace, gdp_group_norm_workspace_bytes(T, H, D, per_head), dev, stream)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    a = GdpGroupNormBackwardArgs(
        d_output.data_ptr(), d_output.stride(0), d_output.stride(1), *tensors, *codes, w, b, ptr(out["do"]),
        ptr(out["dz"]), ptr(out["dweight"]), ptr(out["dbias"]), ws.data_ptr(), ws_bytes, T, H, D, eps,
        _TYPES[d_output.dtype], int(bool(center)), per_head, _act_code(activation))
    _call("gdp_group_norm_backward", a, stream)
    return out
