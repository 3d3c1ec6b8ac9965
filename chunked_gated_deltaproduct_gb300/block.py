"""The operators of ``include/gdp_block.h`` over torch tensors: the short causal convolution, the selective state
space scan (packed sequences, backward, one-token step of each) and the residual norm with its backward pass.
Argument checks and marshalling only, in the manner of ``layer.py``: torch supplies device memory and the current
stream, there is no fallback, and ``stream`` makes a call as under ``torch.cuda.stream`` of it.
"""
from __future__ import annotations

import ctypes

import torch

from . import layer
from .binding import GDP_ERR_UNSUPPORTED, GdpError
from .layer import (_TYPES, GDP_ACT_NONE, GDP_ACT_SIGMOID, GDP_ACT_SILU, _cu, _current, _dense, _f32, _finish, _first, _i64, _int,
                    _invalid, _on, _packer, _rows, _status, _sz, _vp)

GDP_SCAN_CHUNK = 16  # tokens between the states that selective_scan keeps for its backward pass
_CONV_ACTS = {None: GDP_ACT_NONE, "silu": GDP_ACT_SILU}
_GATE_ACTS = {None: GDP_ACT_NONE, "silu": GDP_ACT_SILU, "sigmoid": GDP_ACT_SIGMOID}


class GdpConvArgs(ctypes.Structure):
    """Mirror of ``gdp_conv_args``."""
    _fields_ = [
        ("x", _vp), ("x_stride_t", _i64), ("weight", _vp), ("bias", _vp), ("output", _vp), ("cu_seqlens", _vp),
        ("T", _i64), ("N", _i64), ("C", _i64), ("width", _i64), ("initial_state", _vp), ("output_state", _vp),
        ("state", _vp), ("state_indices", _vp), ("num_slots", _i64), ("device_status", _vp),
        ("cu_seqlens_int64", _int), ("dtype", _int), ("activation", _int), ("zero_padding", _int),
    ]


class GdpConvBackwardArgs(ctypes.Structure):
    """Mirror of ``gdp_conv_backward_args``."""
    _fields_ = [
        ("x", _vp), ("x_stride_t", _i64), ("weight", _vp), ("bias", _vp), ("d_output", _vp),
        ("d_output_stride_t", _i64), ("cu_seqlens", _vp), ("T", _i64), ("N", _i64), ("C", _i64), ("width", _i64),
        ("initial_state", _vp), ("d_final_state", _vp), ("dx", _vp), ("d_weight", _vp), ("d_bias", _vp),
        ("d_initial_state", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("device_status", _vp),
        ("cu_seqlens_int64", _int), ("dtype", _int), ("activation", _int),
    ]


class GdpScanArgs(ctypes.Structure):
    """Mirror of ``gdp_scan_args``."""
    _fields_ = [
        ("x", _vp), ("x_stride_t", _i64), ("dt", _vp), ("dt_stride_t", _i64), ("A", _vp), ("B", _vp), ("C_in", _vp),
        ("B_stride_t", _i64), ("B_stride_g", _i64), ("C_stride_t", _i64), ("C_stride_g", _i64), ("D", _vp),
        ("z", _vp), ("z_stride_t", _i64), ("dt_bias", _vp), ("output", _vp), ("cu_seqlens", _vp), ("T", _i64),
        ("N", _i64), ("C", _i64), ("S", _i64), ("G", _i64), ("initial_state", _vp), ("output_state", _vp),
        ("state", _vp), ("state_indices", _vp), ("num_slots", _i64), ("chunk_states", _vp), ("workspace", _vp),
        ("workspace_bytes", _sz), ("device_status", _vp), ("cu_seqlens_int64", _int), ("x_dtype", _int),
        ("dt_dtype", _int), ("dt_softplus", _int), ("zero_padding", _int),
    ]


class GdpScanBackwardArgs(ctypes.Structure):
    """Mirror of ``gdp_scan_backward_args``."""
    _fields_ = [
        ("x", _vp), ("x_stride_t", _i64), ("dt", _vp), ("dt_stride_t", _i64), ("A", _vp), ("B", _vp), ("C_in", _vp),
        ("B_stride_t", _i64), ("B_stride_g", _i64), ("C_stride_t", _i64), ("C_stride_g", _i64), ("D", _vp),
        ("z", _vp), ("z_stride_t", _i64), ("dt_bias", _vp), ("d_output", _vp), ("d_output_stride_t", _i64),
        ("cu_seqlens", _vp), ("T", _i64), ("N", _i64), ("C", _i64), ("S", _i64), ("G", _i64), ("chunk_states", _vp),
        ("d_final_state", _vp), ("dx", _vp), ("ddt", _vp), ("dA", _vp), ("dB", _vp), ("dC", _vp), ("dD", _vp),
        ("dz", _vp), ("ddt_bias", _vp), ("d_initial_state", _vp), ("workspace", _vp), ("workspace_bytes", _sz),
        ("device_status", _vp), ("cu_seqlens_int64", _int), ("x_dtype", _int), ("dt_dtype", _int),
        ("dt_softplus", _int),
    ]


class GdpResidualNormArgs(ctypes.Structure):
    """Mirror of ``gdp_residual_norm_args``."""
    _fields_ = [
        ("residual", _vp), ("residual_stride_t", _i64), ("block", _vp), ("block_stride_t", _i64), ("gate", _vp),
        ("gate_stride_t", _i64), ("weight", _vp), ("post_weight", _vp), ("scale", _vp), ("y", _vp),
        ("residual_out", _vp), ("T", _i64), ("C", _i64), ("eps", _f32), ("dtype", _int), ("residual_dtype", _int),
        ("activation", _int),
    ]


class GdpResidualNormBackwardArgs(ctypes.Structure):
    """Mirror of ``gdp_residual_norm_backward_args``."""
    _fields_ = [
        ("d_y", _vp), ("d_y_stride_t", _i64), ("d_residual_out", _vp), ("d_residual_out_stride_t", _i64),
        ("residual_out", _vp), ("residual_out_stride_t", _i64), ("block", _vp), ("block_stride_t", _i64),
        ("gate", _vp), ("gate_stride_t", _i64), ("weight", _vp), ("post_weight", _vp), ("scale", _vp),
        ("d_residual", _vp), ("d_block", _vp), ("d_gate", _vp), ("d_weight", _vp), ("d_post_weight", _vp),
        ("d_scale", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("T", _i64), ("C", _i64), ("eps", _f32),
        ("dtype", _int), ("residual_dtype", _int), ("activation", _int),
    ]


_ARGS = (GdpConvArgs, GdpConvBackwardArgs, GdpScanArgs, GdpScanBackwardArgs, GdpResidualNormArgs, GdpResidualNormBackwardArgs)
(_pack_conv, _pack_conv_backward, _pack_scan, _pack_scan_backward, _pack_residual, _pack_residual_backward) = map(_packer, _ARGS)
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = layer._library()
        for name in ("gdp_short_convolution", "gdp_short_convolution_decode", "gdp_short_convolution_backward", "gdp_selective_scan",
                     "gdp_selective_scan_decode", "gdp_selective_scan_backward", "gdp_residual_norm", "gdp_residual_norm_backward"):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = _int, [_vp, _vp]
        for name, dims, result in (("gdp_conv_workspace_bytes", 3, _sz), ("gdp_scan_workspace_bytes", 5, _sz),
                                   ("gdp_scan_forward_workspace_bytes", 5, _sz),
                                   ("gdp_residual_norm_workspace_bytes", 2, _sz), ("gdp_scan_chunk_rows", 2, _i64)):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = result, [_i64] * dims
        lib.gdp_block_args_size.restype, lib.gdp_block_args_size.argtypes = _sz, [_int]
        for i, args in enumerate(_ARGS):
            if not lib.gdp_block_args_size(i) == ctypes.sizeof(args) == len(_packer(args)(*[0] * len(args._fields_))):
                raise RuntimeError(f"{args.__name__} layout mismatch between the binding and the library")
        _lib = lib
    return _lib


def gdp_conv_workspace_bytes(T: int, C: int, width: int) -> int:
    return int(_library().gdp_conv_workspace_bytes(T, C, width))


def gdp_scan_workspace_bytes(T: int, N: int, C: int, S: int, G: int = 1) -> int:
    return int(_library().gdp_scan_workspace_bytes(T, N, C, S, G))


def gdp_scan_forward_workspace_bytes(T: int, N: int, C: int, S: int, G: int = 1) -> int:
    return int(_library().gdp_scan_forward_workspace_bytes(T, N, C, S, G))


def gdp_scan_chunk_rows(T: int, N: int) -> int:
    return int(_library().gdp_scan_chunk_rows(T, N))


def gdp_residual_norm_workspace_bytes(T: int, C: int) -> int:
    return int(_library().gdp_residual_norm_workspace_bytes(T, C))


# ---- checks ------------------------------------------------------------------------------------------

def _activation(table, name):
    code = table.get(name, -1)
    if code < 0:
        _invalid(f"activation must be one of {list(table)} (got {name!r})")
    return code


def _address(t):
    return 0 if t is None else t.data_ptr()


def _output(output, x, shape, dev):
    """(output, its address, whether the call allocated it)."""
    if output is None:
        output = torch.empty_like(x, memory_format=torch.contiguous_format)
        return output, output.data_ptr(), 1
    return output, _dense("output", output, shape, x.dtype, dev), 0


def _workspace(workspace, need, like, dev):
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _invalid("workspace must be contiguous and on the tensors' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _states(initial_state, output_state, state, state_indices, N, each, dtype, dev):
    """Addresses of the state buffers ([N, *each], or the cache [num_slots, *each] and its indices) and num_slots."""
    if state is None:
        if initial_state is None and output_state is None:
            return 0, 0, 0, 0, 0
        return (_dense("initial_state", initial_state, (N, *each), dtype, dev),
                _dense("output_state", output_state, (N, *each), dtype, dev), 0, 0, 0)
    if initial_state is not None or output_state is not None:
        _invalid("the state cache excludes initial_state and output_state")
    if state_indices is None or state.dim() != 1 + len(each):
        _invalid(f"the state cache is [num_slots, {', '.join(map(str, each))}] and needs state_indices")
    slots = state.shape[0]
    return (0, 0, _dense("state", state, (slots, *each), dtype, dev), _dense("state_indices", state_indices, (N,), torch.int32, dev),
            slots)


# ---- the short convolution ---------------------------------------------------------------------------

def _taps(weight, bias, C, dev):
    """(addresses of weight and bias, width)."""
    if weight.dim() != 2 or weight.shape[0] != C:
        _invalid(f"weight must be [{C}, width] (got {tuple(weight.shape)})")
    return (_dense("weight", weight, weight.shape, torch.float32, dev), _dense("bias", bias, (C,), torch.float32, dev),
            weight.shape[1])


def _convolution(x, weight, bias, activation, first, cu, N, cu64, entry, initial_state, output_final_state, state, state_indices,
                 output, output_state, device_status):
    """The common part of the packed and the one-token call."""
    shape, dtype, dev = first
    T, C = shape
    w, b, width = _taps(weight, bias, C, dev)
    output, op, own = _output(output, x, shape, dev)
    if output_final_state and state is None and output_state is None:
        output_state = torch.empty((N, width - 1, C), dtype=x.dtype, device=x.device)
    lib = _library()
    a = _pack_conv(x.data_ptr(), x.stride(0), w, b, op, cu, T, N, C, width,
                   *_states(initial_state, output_state, state, state_indices, N, (width - 1, C), x.dtype, dev),
                   _status(device_status, dev), cu64, dtype, _activation(_CONV_ACTS, activation), own)
    _finish(getattr(lib, entry)(a, _current(dev)), lib)
    return (output, output_state) if output_final_state else output


def short_convolution(x, weight, cu_seqlens, bias=None, activation="silu", initial_state=None, output_final_state=False, state=None,
                      state_indices=None, output=None, output_state=None, device_status=None, stream=None):
    """y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}) along every packed sequence, per channel
    (gdp_short_convolution).

    x [T, C] bf16, f16 or fp32, rows may be strided; weight [C, W] fp32 with W 2 to 4, bias [C] fp32 or None;
    ``activation`` "silu" or None; cu_seqlens [N + 1] int32 / int64.  A state is the last W - 1 inputs, oldest
    first, in x's type: initial_state [N, W - 1, C] (None: zeros), or the cache ``state`` [num_slots, W - 1, C] read
    and written in place at ``state_indices`` [N] int32 (-1: from zeros, nothing written).  Returns ``y`` [T, C], or
    ``(y, final_state)`` when output_final_state (dense mode; None in cache mode).  Rows at or past
    cu_seqlens[N] (padding) are zeros; in a buffer given as ``output`` they are left as they are."""
    if stream is not None:
        return _on(stream, short_convolution, x, weight, cu_seqlens, bias, activation, initial_state, output_final_state, state,
                   state_indices, output, output_state, device_status)
    first = _first("x", x, ("T", "C"))
    cu, N, cu64 = _cu(cu_seqlens, first[2])
    return _convolution(x, weight, bias, activation, first, cu, N, cu64, "gdp_short_convolution", initial_state, output_final_state,
                        state, state_indices, output, output_state, device_status)


def short_convolution_decode(x, weight, bias=None, activation="silu", initial_state=None, output_final_state=False, state=None,
                             state_indices=None, output=None, output_state=None, device_status=None, stream=None):
    """One token per sequence: x [N, C]; the state modes and types of short_convolution.  Returns ``y`` [N, C], or
    ``(y, final_state)`` when output_final_state (dense mode)."""
    if stream is not None:
        return _on(stream, short_convolution_decode, x, weight, bias, activation, initial_state, output_final_state, state, state_indices,
                   output, output_state, device_status)
    first = _first("x", x, ("N", "C"))
    return _convolution(x, weight, bias, activation, first, 0, first[0][0], 0, "gdp_short_convolution_decode", initial_state,
                        output_final_state, state, state_indices, output, output_state, device_status)


def short_convolution_backward(x, weight, d_output, cu_seqlens, bias=None, activation="silu", initial_state=None, d_final_state=None,
                               workspace=None, device_status=None, stream=None):
    """Gradients of short_convolution for dL/dy = ``d_output`` [T, C] and dL/dfinal = ``d_final_state``
    [N, W - 1, C] (or None), both in x's type.  Returns a dict: dx (zero in rows at or past cu_seqlens[N]) and
    d_initial_state (None without an initial state) in x's type, dweight and dbias fp32 (None without a bias)."""
    if stream is not None:
        return _on(stream, short_convolution_backward, x, weight, d_output, cu_seqlens, bias, activation, initial_state, d_final_state,
                   workspace, device_status)
    shape, dtype, dev = _first("x", x, ("T", "C"))
    T, C = shape
    w, b, width = _taps(weight, bias, C, dev)
    dp = _rows("d_output", d_output, shape, x.dtype, dev)
    cu, N, cu64 = _cu(cu_seqlens, dev)
    each = (N, width - 1, C)
    init, dfin = _dense("initial_state", initial_state, each, x.dtype, dev), _dense("d_final_state", d_final_state, each, x.dtype, dev)
    code = _activation(_CONV_ACTS, activation)
    dx, dw = torch.empty(shape, dtype=x.dtype, device=x.device), torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    dinit = torch.empty(each, dtype=x.dtype, device=x.device) if initial_state is not None else None
    lib = _library()
    workspace, wp, wb = _workspace(workspace, lib.gdp_conv_workspace_bytes(T, C, width), x, dev)
    a = _pack_conv_backward(x.data_ptr(), x.stride(0), w, b, dp, d_output.stride(0), cu, T, N, C, width, init, dfin, dx.data_ptr(),
                            dw.data_ptr(), _address(db), _address(dinit), wp, wb, _status(device_status, dev), cu64, dtype, code)
    _finish(lib.gdp_short_convolution_backward(a, _current(dev)), lib)
    return {"dx": dx, "dweight": dw, "dbias": db, "d_initial_state": dinit}


# ---- the selective scan ------------------------------------------------------------------------------

def _vectors(name, t, T, x, dev):
    """Address, token and group stride, and [G, S] of B or C ([T, S] or [T, G, S])."""
    shape = t.shape
    if len(shape) == 2:
        return _rows(name, t, (T, shape[1]), x.dtype, dev), t.stride(0), 0, 1, shape[1]
    if len(shape) != 3:
        _invalid(f"{name} must be [T, S] or [T, G, S]")
    return _rows(name, t, (T, *shape[1:]), x.dtype, dev), t.stride(0), t.stride(1), shape[1], shape[2]


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, first):
    """The inputs' part of the argument structs, and (S, G, dt's type code)."""
    shape, _, dev = first
    T, channels = shape
    if dt.dtype != x.dtype and dt.dtype != torch.float32:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"dt must be float32 or of x's type (got {dt.dtype})")
    dp = _rows("dt", dt, shape, dt.dtype, dev)
    bp, bt, bg, G, S = _vectors("B", B, T, x, dev)
    cp, ct, cg, cG, cS = _vectors("C", C, T, x, dev)
    if (cG, cS) != (G, S):
        _invalid("B and C must have one shape")
    zp = _rows("z", z, shape, x.dtype, dev) if z is not None else 0
    return ((x.data_ptr(), x.stride(0), dp, dt.stride(0), _dense("A", A, (channels, S), torch.float32, dev), bp, cp, bt, bg, ct, cg,
             _dense("D", D, (channels,), torch.float32, dev), zp, z.stride(0) if z is not None else 0,
             _dense("dt_bias", dt_bias, (channels,), torch.float32, dev)), S, G, _TYPES[dt.dtype])


def _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, first, cu, N, cu64, entry, initial_state, output_final_state, state,
          state_indices, save_states, output, output_state, workspace, device_status):
    """The common part of the packed and the one-token call."""
    shape, dtype, dev = first
    T, channels = shape
    inputs, S, G, dt_type = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, first)
    output, op, own = _output(output, x, shape, dev)
    if output_final_state and state is None and output_state is None:
        output_state = torch.empty((N, channels, S), dtype=torch.float32, device=x.device)
    lib = _library()
    kept = None
    if save_states:
        kept = torch.empty((lib.gdp_scan_chunk_rows(T, N), channels, S), dtype=torch.float32, device=x.device)
    need = lib.gdp_scan_forward_workspace_bytes(T, N, channels, S, G) if cu else 0
    wp = wb = 0
    if need:
        workspace, wp, wb = _workspace(workspace, need, x, dev)
    a = _pack_scan(*inputs, op, cu, T, N, channels, S, G,
                   *_states(initial_state, output_state, state, state_indices, N, (channels, S), torch.float32, dev), _address(kept),
                   wp, wb, _status(device_status, dev), cu64, dtype, dt_type, int(bool(dt_softplus)), own)
    _finish(getattr(lib, entry)(a, _current(dev)), lib)
    if not output_final_state:
        return (output, kept) if save_states else output
    return (output, output_state, kept) if save_states else (output, output_state)


def selective_scan(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                   output_final_state=False, state=None, state_indices=None, save_states=False, output=None, output_state=None,
                   workspace=None, device_status=None, stream=None):
    """h_t = exp(e_t A) h_{t-1} + e_t x_t B_t, y_t = (sum_s C_t h_t + D x_t) silu(z_t) along every packed sequence,
    with e = softplus(dt + dt_bias) (or dt + dt_bias): S states per channel (gdp_selective_scan).

    x, z [T, C] bf16, f16 or fp32; dt [T, C] fp32 or x's type; B, C [T, S] or [T, G, S] in x's type, shared by the
    channels of a group (S up to 64); rows may be strided (slices of wider projections).  A [C, S], D [C],
    dt_bias [C] fp32; D, z and dt_bias may be None.  cu_seqlens [N + 1] int32 / int64.  initial_state [N, C, S] fp32
    (None: zero), or the cache ``state`` [num_slots, C, S] fp32 read and written in place at ``state_indices`` [N] int32
    (-1: from zero, nothing written).

    Returns ``y`` [T, C] in x's type; with output_final_state also the final state (dense mode; None in cache
    mode); with save_states also what selective_scan_backward reads, the states entering every GDP_SCAN_CHUNK
    tokens of a sequence (fp32 [gdp_scan_chunk_rows(T, N), C, S]).  Rows at or past cu_seqlens[N] (padding) are
    zeros; in a buffer given as ``output`` they are left as they are."""
    if stream is not None:
        return _on(stream, selective_scan, x, dt, A, B, C, cu_seqlens, D, z, dt_bias, dt_softplus, initial_state, output_final_state,
                   state, state_indices, save_states, output, output_state, workspace, device_status)
    first = _first("x", x, ("T", "C"))
    cu, N, cu64 = _cu(cu_seqlens, first[2])
    return _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, first, cu, N, cu64, "gdp_selective_scan", initial_state,
                 output_final_state, state, state_indices, save_states, output, output_state, workspace, device_status)


def selective_scan_decode(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                          output_final_state=False, state=None, state_indices=None, output=None, output_state=None,
                          device_status=None, stream=None):
    """One token per sequence: x, dt, z [N, C], B, C [N, S] or [N, G, S]; the state modes and types of
    selective_scan.  Returns ``y`` [N, C], or ``(y, final_state)`` when output_final_state (dense mode)."""
    if stream is not None:
        return _on(stream, selective_scan_decode, x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, output_final_state, state,
                   state_indices, output, output_state, device_status)
    first = _first("x", x, ("N", "C"))
    return _scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, first, 0, first[0][0], 0, "gdp_selective_scan_decode", initial_state,
                 output_final_state, state, state_indices, False, output, output_state, None, device_status)


def selective_scan_backward(x, dt, A, B, C, d_output, cu_seqlens, chunk_states, D=None, z=None, dt_bias=None, dt_softplus=True,
                            d_final_state=None, output_d_initial_state=False, workspace=None, device_status=None, stream=None):
    """Gradients of selective_scan for dL/dy = ``d_output`` [T, C] in x's type and dL/dfinal = ``d_final_state``
    [N, C, S] fp32 (or None).  ``chunk_states``: what selective_scan returned for save_states with the same inputs.
    Returns a dict: dx, dz in x's type, ddt in dt's, dB and dC in x's type and B's shape (all zero in rows at or past
    cu_seqlens[N]); dA, dD, ddt_bias fp32; d_initial_state fp32 with output_d_initial_state.  What the forward call
    did without is None."""
    if stream is not None:
        return _on(stream, selective_scan_backward, x, dt, A, B, C, d_output, cu_seqlens, chunk_states, D, z, dt_bias, dt_softplus,
                   d_final_state, output_d_initial_state, workspace, device_status)
    first = _first("x", x, ("T", "C"))
    shape, dtype, dev = first
    T, channels = shape
    inputs, S, G, dt_type = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, first)
    dyp = _rows("d_output", d_output, shape, x.dtype, dev)
    cu, N, cu64 = _cu(cu_seqlens, dev)
    lib = _library()
    kept = _dense("chunk_states", chunk_states, (lib.gdp_scan_chunk_rows(T, N), channels, S), torch.float32, dev)
    dfin = _dense("d_final_state", d_final_state, (N, channels, S), torch.float32, dev)

    def like(t, dtype=None):
        return None if t is None else torch.empty(t.shape, dtype=dtype or t.dtype, device=x.device)

    dx, ddt, dA, dB, dC, dD, dz, dbias = map(like, (x, dt, A, B, C, D, z, dt_bias))
    dinit = torch.empty((N, channels, S), dtype=torch.float32, device=x.device) if output_d_initial_state else None
    workspace, wp, wb = _workspace(workspace, lib.gdp_scan_workspace_bytes(T, N, channels, S, G), x, dev)
    a = _pack_scan_backward(*inputs, dyp, d_output.stride(0), cu, T, N, channels, S, G, kept, dfin,
                            *map(_address, (dx, ddt, dA, dB, dC, dD, dz, dbias, dinit)), wp, wb, _status(device_status, dev), cu64,
                            dtype, dt_type, int(bool(dt_softplus)))
    _finish(lib.gdp_selective_scan_backward(a, _current(dev)), lib)
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": dD, "dz": dz, "ddt_bias": dbias, "d_initial_state": dinit}


# ---- the residual norm -------------------------------------------------------------------------------

def _stream_type(name, t, x):
    """The residual's type code: the block's or fp32."""
    if t.dtype != x.dtype and t.dtype != torch.float32:
        raise GdpError(GDP_ERR_UNSUPPORTED, f"{name} must be float32 or of the block's type (got {t.dtype})")
    return _TYPES[t.dtype]


def residual_norm(residual, block, weight, post_weight=None, gate=None, activation="sigmoid", scale=None, eps=1e-5, output=None,
                  output_residual=None, stream=None):
    """r = residual + scale act(gate) m, y = r / rms(r) weight, with m = block / rms(block) post_weight (or the block
    itself): the norm behind a block, its gate and scale, the residual sum and the norm before the next block
    (gdp_residual_norm).

    block, gate [T, C] bf16, f16 or fp32; residual [T, C] of that type or fp32; rows may be strided; weight,
    post_weight, scale [C] fp32; post_weight, gate and scale may be None.  ``activation`` "sigmoid" or "silu" of the
    gate, or None: the gate itself.  C up to 8192.  Returns ``(y, r)``, y in the block's type and r in the residual's.
    ``output_residual`` may be the residual itself."""
    if stream is not None:
        return _on(stream, residual_norm, residual, block, weight, post_weight, gate, activation, scale, eps, output, output_residual)
    first = _first("block", block, ("T", "C"))
    shape, dtype, dev = first
    T, C = shape
    rt = _stream_type("residual", residual, block)
    rp = _rows("residual", residual, shape, residual.dtype, dev)
    gp = _rows("gate", gate, shape, block.dtype, dev) if gate is not None else 0
    columns = [_dense(n, t, (C,), torch.float32, dev) for n, t in (("weight", weight), ("post_weight", post_weight), ("scale", scale))]
    code = _activation(_GATE_ACTS, activation)
    output, yp, _ = _output(output, block, shape, dev)
    if output_residual is None:
        output_residual = torch.empty_like(residual, memory_format=torch.contiguous_format)
        op = output_residual.data_ptr()
    else:
        op = _dense("output_residual", output_residual, shape, residual.dtype, dev)
    lib = _library()
    a = _pack_residual(rp, residual.stride(0), block.data_ptr(), block.stride(0), gp, gate.stride(0) if gate is not None else 0, *columns,
                       yp, op, T, C, eps, dtype, rt, code)
    _finish(lib.gdp_residual_norm(a, _current(dev)), lib)
    return output, output_residual


def residual_norm_backward(d_y, d_residual_out, residual_out, block, weight, post_weight=None, gate=None, activation="sigmoid",
                           scale=None, eps=1e-5, workspace=None, stream=None):
    """Gradients of residual_norm for dL/dy = ``d_y`` and dL/dr = ``d_residual_out`` (or None), from the forward's
    ``residual_out`` (its second result), block and gate.  Returns a dict: d_residual in the residual's type,
    d_block and d_gate in the block's, dweight, dpost_weight and dscale fp32; None for what the forward call did
    without."""
    if stream is not None:
        return _on(stream, residual_norm_backward, d_y, d_residual_out, residual_out, block, weight, post_weight, gate, activation, scale,
                   eps, workspace)
    first = _first("block", block, ("T", "C"))
    shape, dtype, dev = first
    T, C = shape
    rt = _stream_type("residual_out", residual_out, block)
    rp = _rows("residual_out", residual_out, shape, residual_out.dtype, dev)
    dyp = _rows("d_y", d_y, shape, block.dtype, dev)
    drp, drs = 0, 0
    if d_residual_out is not None:
        drp, drs = _rows("d_residual_out", d_residual_out, shape, residual_out.dtype, dev), d_residual_out.stride(0)
    gp, gs = (_rows("gate", gate, shape, block.dtype, dev), gate.stride(0)) if gate is not None else (0, 0)
    columns = [_dense(n, t, (C,), torch.float32, dev) for n, t in (("weight", weight), ("post_weight", post_weight), ("scale", scale))]
    code = _activation(_GATE_ACTS, activation)
    dres = torch.empty(shape, dtype=residual_out.dtype, device=block.device)
    dblock = torch.empty(shape, dtype=block.dtype, device=block.device)
    dgate = torch.empty(shape, dtype=block.dtype, device=block.device) if gate is not None else None
    dw, dpost, dscale = (None if t is None else torch.empty_like(t) for t in (weight, post_weight, scale))
    lib = _library()
    workspace, wp, wb = _workspace(workspace, lib.gdp_residual_norm_workspace_bytes(T, C), block, dev)
    a = _pack_residual_backward(dyp, d_y.stride(0), drp, drs, rp, residual_out.stride(0), block.data_ptr(), block.stride(0), gp, gs,
                                *columns, *map(_address, (dres, dblock, dgate, dw, dpost, dscale)), wp, wb, T, C, eps, dtype, rt, code)
    _finish(lib.gdp_residual_norm_backward(a, _current(dev)), lib)
    return {"d_residual": dres, "d_block": dblock, "d_gate": dgate, "dweight": dw, "dpost_weight": dpost, "dscale": dscale}
