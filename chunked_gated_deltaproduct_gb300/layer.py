"""The layer operators of ``include/gdp_layer.h`` over torch tensors: the gated linear recurrence
(packed sequences, backward, one-token step) and the grouped norm with an activated gate, with its
8-bit activation checkpoints.  Argument checks and marshalling only; torch supplies device memory and
the current stream, and there is no fallback: without the library every call raises.

``stream``, a raw stream handle, makes a call as under ``torch.cuda.stream`` of it: it runs there and what it
allocates belongs there, so that the caller orders it after the inputs' stream, and other streams after it.
"""
from __future__ import annotations

import ctypes
import struct
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
        ("zero_padding", _int),
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


def _packer(args):
    """The argument struct's bytes from its fields' values in order: a tenth of the time of filling a
    ctypes structure, which a one-token step would notice.  (The fields need no padding between them.)"""
    codes = {_vp: "Q", _i64: "q", _sz: "Q", _int: "i", _f32: "f"}
    return struct.Struct("@" + "".join(codes[t] for _, t in args._fields_) + "0q").pack


_pack_recurrence, _pack_recurrence_backward = _packer(GdpRecurrenceArgs), _packer(GdpRecurrenceBackwardArgs)
_pack_norm, _pack_norm_backward = _packer(GdpGroupNormArgs), _packer(GdpGroupNormBackwardArgs)


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
            fn.restype, fn.argtypes = _int, [_vp, _vp]
        lib.gdp_group_norm_workspace_bytes.restype = _sz
        lib.gdp_group_norm_workspace_bytes.argtypes = [_i64, _i64, _i64, _int]
        lib.gdp_arm_recurrence_wait_test.restype = _int
        lib.gdp_arm_recurrence_wait_test.argtypes = [ctypes.c_uint64]
        lib.gdp_layer_args_size.restype = _sz
        lib.gdp_layer_args_size.argtypes = [_int]
        for i, args in enumerate((GdpRecurrenceArgs, GdpRecurrenceBackwardArgs, GdpGroupNormArgs,
                                  GdpGroupNormBackwardArgs)):
            if not lib.gdp_layer_args_size(i) == ctypes.sizeof(args) == len(_packer(args)(*[0] * len(args._fields_))):
                raise RuntimeError(f"{args.__name__} layout mismatch between the binding and the library")
        _lib = lib
    return _lib


def gdp_group_norm_workspace_bytes(T: int, H: int, D: int, per_head: bool = False) -> int:
    return int(_library().gdp_group_norm_workspace_bytes(T, H, D, int(per_head)))


def gdp_arm_recurrence_wait_test(limit_ns: int) -> None:
    """Arm the calling thread's next packed recurrence (or its backward pass) to exercise the bounded-wait
    failure path; see the header."""
    lib = _library()
    _finish(lib.gdp_arm_recurrence_wait_test(int(limit_ns)), lib)


# ---- checks.  A one-token step costs a few microseconds of host time, so each tensor's are one
# expression, and the wording of a refusal is worked out only once it fails.

def _invalid(msg):
    raise GdpError(GDP_ERR_INVALID_ARG, msg)


def _finish(status, lib):
    if status != GDP_OK:
        raise GdpError(status, lib.gdp_last_error().decode())


def _current(dev):
    """Handle of torch's current stream on the device."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _on(stream, call, *args):
    """The call with that stream as torch's current one, its allocations too: a block of another stream's pool may
    still be in use by work on that one."""
    with torch.cuda.stream(torch.cuda.ExternalStream(stream)):
        return call(*args)


def _current_device():
    return torch._C._cuda_getDevice()


def _first(name, t, dims):
    """(shape, type code, device index) of the tensor that sets them for the call.  The library launches on the
    current device, so the tensors have to be there."""
    if t.dim() != len(dims):
        _invalid(f"{name} must be [{', '.join(dims)}]")
    code = _TYPES.get(t.dtype)
    if code is None:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"{name} must be bfloat16, float16 or float32 (got {t.dtype})")
    if not t.is_cuda:
        _invalid("the tensors must be on a CUDA device")
    shape = t.shape
    if shape[-1] > 1 and t.stride(-1) != 1:
        _invalid(f"{name} must be contiguous in its last dimension")
    dev = t.get_device()
    if dev != _current_device():
        _invalid(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return shape, code, dev


def _rows(name, t, shape, dtype, dev):
    """Address of a tensor of that shape, type and device whose last dimension is contiguous."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or (t.stride(-1) != 1 and shape[-1] > 1):
        if t.shape != shape:
            _invalid(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
        if t.dtype != dtype:
            raise GdpError(GDP_ERR_UNSUPPORTED, f"{name} must be {dtype} (got {t.dtype})")
        if t.get_device() != dev:
            _invalid(f"{name} must be on the device of the other tensors")
        _invalid(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def _dense(name, t, shape, dtype, dev):
    """Address of a contiguous tensor of that shape, type and device (None: 0)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
        _invalid(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the device of the other tensors")
    return t.data_ptr()


def _gate_type(x, g):
    """g's type code: x's or fp32."""
    dtype = g.dtype
    if dtype != x.dtype and dtype != torch.float32:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"g must be float32 or of x's type (got {dtype})")
    return _TYPES[dtype]


def _cu(cu_seqlens, dev):
    if cu_seqlens is None:
        _invalid("cu_seqlens is required (packed input only)")
    wide = cu_seqlens.dtype == torch.int64
    if (not (wide or cu_seqlens.dtype == torch.int32) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
            or not cu_seqlens.is_contiguous() or cu_seqlens.get_device() != dev):
        _invalid("cu_seqlens must be a contiguous int32 or int64 vector of N + 1 entries on the tensors' device")
    return cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(wide)


def _status(t, dev):
    if t is None:
        return 0
    if t.numel() < 1 or t.element_size() != 4 or t.get_device() != dev:
        _invalid("device_status must be a 32-bit word on the tensors' device")
    return t.data_ptr()


def _gate_code(gate):
    code = _GATES.get(gate)
    if code is None:
        _invalid(f"gate must be one of {sorted(_GATES)} (got {gate!r})")
    return code


def _state_args(initial_state, output_state, state, state_indices, N, C, dev):
    if state is None:
        if initial_state is None and output_state is None:
            return 0, 0, 0, 0, 0
        return (_dense("initial_state", initial_state, (N, C), torch.float32, dev),
                _dense("output_state", output_state, (N, C), torch.float32, dev), 0, 0, 0)
    if initial_state is not None or output_state is not None:
        _invalid("the state cache excludes initial_state and output_state")
    if state_indices is None or state.dim() != 2:
        _invalid("the state cache is [num_slots, C] and needs state_indices")
    slots = state.shape[0]
    return (0, 0, _dense("state", state, (slots, C), torch.float32, dev),
            _dense("state_indices", state_indices, (N,), torch.int32, dev), slots)


def _recurrence(x, g, gate, cu, N, cu64, entry, first, initial_state, output_final_state, state, state_indices, output,
                output_state, device_status):
    """The common part of the packed and the one-token call."""
    shape, xt, dev = first
    T, C = shape
    gp, gt = _rows("g", g, shape, g.dtype, dev), _gate_type(x, g)
    own = output is None
    if own:
        output = torch.empty_like(x, memory_format=torch.contiguous_format)
        op = output.data_ptr()
    else:
        op = _dense("output", output, shape, x.dtype, dev)
    if output_final_state and state is None and output_state is None:
        output_state = torch.empty((N, C), dtype=torch.float32, device=x.device)
    lib = _library()
    a = _pack_recurrence(x.data_ptr(), x.stride(0), gp, g.stride(0), op, cu, T, N, C,
                          *_state_args(initial_state, output_state, state, state_indices, N, C, dev),
                          _status(device_status, dev), cu64, xt, gt, _gate_code(gate), own)
    _finish(getattr(lib, entry)(a, _current(dev)), lib)
    return (output, output_state) if output_final_state else output


def gated_linear_recurrence(x, g, cu_seqlens, gate="log", initial_state=None, output_final_state=False, state=None,
                            state_indices=None, output=None, output_state=None, device_status=None, stream=None):
    """h_t = a_t h_{t-1} + b_t along every packed sequence, per channel (gdp_linear_recurrence).

    x [T, C] bf16, f16 or fp32; g [T, C] fp32 or x's type; rows may be strided (slices of a wider
    projection).  ``gate``: "log" a = exp(g), b = x; "alpha" a = g, b = x; "sigmoid" a = sigmoid(g),
    b = (1 - a) x.  cu_seqlens [N + 1] int32 / int64.  initial_state [N, C] fp32 (None: zero), or the
    cache ``state`` [num_slots, C] fp32 read and written in place at ``state_indices`` [N] int32 (-1:
    from zero, nothing written).  Returns ``h`` [T, C] in x's type, or ``(h, final_state)`` when
    output_final_state (dense mode; None in cache mode).  Rows at or past cu_seqlens[N] (padding) are zeros;
    in a buffer given as ``output`` they are left as they are."""
    if stream is not None:
        return _on(stream, gated_linear_recurrence, x, g, cu_seqlens, gate, initial_state, output_final_state, state,
                   state_indices, output, output_state, device_status)
    first = _first("x", x, ("T", "C"))
    cu, N, cu64 = _cu(cu_seqlens, first[2])
    return _recurrence(x, g, gate, cu, N, cu64, "gdp_linear_recurrence", first, initial_state, output_final_state, state,
                       state_indices, output, output_state, device_status)


def gated_linear_recurrence_decode(x, g, gate="log", initial_state=None, output_final_state=False, state=None,
                                   state_indices=None, output=None, output_state=None, device_status=None,
                                   stream=None):
    """One token per sequence: x, g [N, C]; the state modes, types and gates of gated_linear_recurrence.
    Returns ``h`` [N, C], or ``(h, final_state)`` when output_final_state (dense mode)."""
    if stream is not None:
        return _on(stream, gated_linear_recurrence_decode, x, g, gate, initial_state, output_final_state, state, state_indices,
                   output, output_state, device_status)
    first = _first("x", x, ("N", "C"))
    return _recurrence(x, g, gate, 0, first[0][0], 0, "gdp_linear_recurrence_decode", first, initial_state,
                       output_final_state, state, state_indices, output, output_state, device_status)


def gated_linear_recurrence_backward(g, h, d_output, cu_seqlens, gate="log", x=None, initial_state=None,
                                     d_final_state=None, device_status=None, stream=None):
    """Gradients of gated_linear_recurrence for dL/dh = ``d_output`` [T, C] and dL/dfinal =
    ``d_final_state`` [N, C] fp32 (or None).  ``h``: the forward's output [T, C] in d_output's type, or
    the ActivationCheckpoint of it that gated_group_norm kept ([T, H, D] with H D = C).  ``x`` is needed
    for the sigmoid gate only.  Returns a dict: dx in d_output's type, dg in g's type (both zero in rows at or
    past cu_seqlens[N]), d_initial_state fp32 (None without an initial state)."""
    if stream is not None:
        return _on(stream, gated_linear_recurrence_backward, g, h, d_output, cu_seqlens, gate, x, initial_state, d_final_state,
                   device_status)
    shape, xt, dev = _first("d_output", d_output, ("T", "C"))
    T, C = shape
    dtype, where = d_output.dtype, d_output.device
    gp, gt = _rows("g", g, shape, g.dtype, dev), _gate_type(d_output, g)
    gate = _gate_code(gate)
    xp = xs = hp = hs = codes = scales = group = 0
    if gate == GDP_GATE_SIGMOID:
        if x is None:
            _invalid("the sigmoid gate's gradient needs x")
        xp, xs = _rows("x", x, shape, dtype, dev), x.stride(0)
    if isinstance(h, ActivationCheckpoint):
        if h.codes.dim() != 3 or h.codes.shape[0] != T or h.codes.shape[1] * h.codes.shape[2] != C:
            _invalid("the checkpoint of h must be [T, H, D] with H D = C")
        group = h.codes.shape[2]
        codes, scales = _checkpoint("h", h, h.codes.shape, dev)
    else:
        hp, hs = _rows("h", h, shape, dtype, dev), h.stride(0)
    cu, N, cu64 = _cu(cu_seqlens, dev)
    init = _dense("initial_state", initial_state, (N, C), torch.float32, dev)
    dfin = _dense("d_final_state", d_final_state, (N, C), torch.float32, dev)
    dx, dg = torch.empty(shape, dtype=dtype, device=where), torch.empty(shape, dtype=g.dtype, device=where)
    dinit = torch.empty((N, C), dtype=torch.float32, device=where) if initial_state is not None else None
    lib = _library()
    a = _pack_recurrence_backward(
        gp, g.stride(0), xp, xs, hp, hs, codes, scales, group, d_output.data_ptr(), d_output.stride(0), cu, T, N, C, init,
        dfin, dx.data_ptr(), dg.data_ptr(), 0 if dinit is None else dinit.data_ptr(), _status(device_status, dev), cu64,
        xt, gt, gate)
    _finish(lib.gdp_linear_recurrence_backward(a, _current(dev)), lib)
    return {"dx": dx, "dg": dg, "d_initial_state": dinit}


def _checkpoint(name, c, shape, dev):
    """Addresses of a checkpoint's codes and scales for an activation of `shape` [T, H, D]."""
    T, H, D = shape
    return (_dense(name + "'s codes", c.codes, shape, torch.int8, dev),
            _dense(name + "'s scales", c.scales, (T, H, -(-D // CHECKPOINT_BLOCK)), torch.float32, dev))


def _new_checkpoint(T, H, D, where):
    return ActivationCheckpoint(torch.empty((T, H, D), dtype=torch.int8, device=where),
                                torch.empty((T, H, -(-D // CHECKPOINT_BLOCK)), dtype=torch.float32, device=where))


def _affine(weight, bias, H, D, dev):
    """(weight, bias, per_head): fp32 [D] or [H, D]."""
    shape = weight.shape
    per_head = len(shape) == 2 and shape == (H, D)
    if not per_head and shape != (D,):
        _invalid(f"weight must be [{D}] or [{H}, {D}] (got {tuple(shape)})")
    return (_dense("weight", weight, shape, torch.float32, dev), _dense("bias", bias, shape, torch.float32, dev),
            int(per_head))


def _act_code(activation):
    code = _ACTS.get(activation)
    if code is None:
        _invalid(f"activation must be 'silu', 'sigmoid' or None (got {activation!r})")
    return code


def gated_group_norm(o, weight, z=None, bias=None, eps=1e-5, center=False, activation="silu", save_checkpoint=False,
                     output=None, stream=None):
    """y = (n weight + bias) act(z) with n the norm of o [T, H, D] over each (token, head)'s D channels:
    RMS, or mean and variance when ``center`` (gdp_group_norm).  ``activation`` "silu" or "sigmoid" of z
    [T, H, D]; without z, "silu" of the affine norm itself, or None.  o and z bf16, f16 or fp32 (one
    type, token and head strides free); weight and bias fp32, [D] or one row per head [H, D].

    Returns ``y`` [T, H, D] in o's type, or ``(y, checkpoint)`` with the GroupNormCheckpoint (8-bit
    codes of o and z) that gated_group_norm_backward takes when ``save_checkpoint``."""
    if stream is not None:
        return _on(stream, gated_group_norm, o, weight, z, bias, eps, center, activation, save_checkpoint, output)
    shape, dt, dev = _first("o", o, ("T", "H", "D"))
    T, H, D = shape
    where = o.device
    ot, oh, _ = o.stride()
    zp = zt = zh = 0
    if z is not None:
        zp = _rows("z", z, shape, o.dtype, dev)
        zt, zh, _ = z.stride()
    w, b, per_head = _affine(weight, bias, H, D, dev)
    if output is None:
        output = torch.empty_like(o, memory_format=torch.contiguous_format)
        yp = output.data_ptr()
    else:
        yp = _dense("output", output, shape, o.dtype, dev)
    kept, ptrs = None, (0, 0, 0, 0)
    if save_checkpoint:
        ko, kz = _new_checkpoint(T, H, D, where), _new_checkpoint(T, H, D, where) if z is not None else None
        kept = GroupNormCheckpoint(ko, kz)
        ptrs = (ko.codes.data_ptr(), ko.scales.data_ptr(), *((kz.codes.data_ptr(), kz.scales.data_ptr()) if kz is not None
                                                             else (0, 0)))
    lib = _library()
    a = _pack_norm(o.data_ptr(), ot, oh, zp, zt, zh, w, b, yp, *ptrs, T, H, D, eps, dt, int(bool(center)), per_head,
                         _act_code(activation))
    _finish(lib.gdp_group_norm(a, _current(dev)), lib)
    return (output, kept) if save_checkpoint else output


def gated_group_norm_backward(d_output, saved, weight, bias=None, eps=1e-5, center=False, activation="silu",
                              workspace=None, stream=None):
    """Gradients of gated_group_norm for dL/dy = ``d_output`` [T, H, D].  ``saved``: the
    GroupNormCheckpoint of the forward call, or the pair ``(o, z)`` of tensors (z None without a gate).
    Returns a dict: do and dz in d_output's type (dz None without z), dweight and dbias fp32 (None
    without a bias)."""
    if stream is not None:
        return _on(stream, gated_group_norm_backward, d_output, saved, weight, bias, eps, center, activation, workspace)
    shape, dt, dev = _first("d_output", d_output, ("T", "H", "D"))
    T, H, D = shape
    dtype, where = d_output.dtype, d_output.device
    dt_t, dt_h, _ = d_output.stride()
    o, z = saved
    op = ot = oh = zp = zt = zh = 0
    codes = (0, 0, 0, 0)
    if isinstance(saved, GroupNormCheckpoint):
        codes = _checkpoint("o", o, shape, dev) + (_checkpoint("z", z, shape, dev) if z is not None else (0, 0))
    else:
        op = _rows("o", o, shape, dtype, dev)
        ot, oh, _ = o.stride()
        if z is not None:
            zp = _rows("z", z, shape, dtype, dev)
            zt, zh, _ = z.stride()
    w, b, per_head = _affine(weight, bias, H, D, dev)
    do, dz = torch.empty(shape, dtype=dtype, device=where), torch.empty(shape, dtype=dtype, device=where) if z is not None else None
    dw, db = torch.empty_like(weight), torch.empty_like(bias) if bias is not None else None
    lib = _library()
    need = lib.gdp_group_norm_workspace_bytes(T, H, D, per_head)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=where)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _invalid("workspace must be contiguous and on the tensors' device")
    a = _pack_norm_backward(
        d_output.data_ptr(), dt_t, dt_h, op, ot, oh, zp, zt, zh, *codes, w, b, do.data_ptr(),
        0 if dz is None else dz.data_ptr(), dw.data_ptr(), 0 if db is None else db.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), T, H, D, eps, dt, int(bool(center)), per_head, _act_code(activation))
    _finish(lib.gdp_group_norm_backward(a, _current(dev)), lib)
    return {"do": do, "dz": dz, "dweight": dw, "dbias": db}
