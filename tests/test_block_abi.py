"""Host-side checks of the block operators (no GPU needed): struct layouts, shape-only queries, and the refusal of
bad arguments before any launch, through the C ABI and the torch wrappers."""
import ctypes

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from chunked_gated_deltaproduct_gb300 import block, layer
from chunked_gated_deltaproduct_gb300 import build as libbuild
from tests.test_layer_abi import _Elsewhere

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced on these paths
INVALID, UNSUPPORTED, ALIAS, WORKSPACE = (pkg.GDP_ERR_INVALID_ARG, pkg.GDP_ERR_UNSUPPORTED, pkg.GDP_ERR_ALIAS, pkg.GDP_ERR_WORKSPACE)
BF16, F16, F32 = pkg.GDP_DTYPE_BF16, pkg.GDP_DTYPE_F16, pkg.GDP_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return block._library()


def _refused(lib, name, a, status):
    assert getattr(lib, name)(ctypes.byref(a), None) == status, pkg.gdp_last_error()
    assert pkg.gdp_last_error() != ""


def _with(a, over):
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_layouts_and_queries(lib):
    for i, s in enumerate(block._ARGS):
        assert lib.gdp_block_args_size(i) == ctypes.sizeof(s)
    assert lib.gdp_block_args_size(6) == 0
    assert pkg.gdp_scan_chunk_rows(100, 3) == 6 + 3 and pkg.gdp_scan_chunk_rows(-1, 3) == 0
    assert pkg.gdp_conv_workspace_bytes(100, 8, 4) > 0 and pkg.gdp_conv_workspace_bytes(100, 8, 5) == 0
    assert pkg.gdp_scan_workspace_bytes(100, 2, 8, 16, 2) > 0
    for bad in ((100, 2, 8, 16, 3), (100, 2, 8, 65, 1), (100, 2, 8, 0, 1), (-1, 2, 8, 16, 1)):
        assert pkg.gdp_scan_workspace_bytes(*bad) == 0
    assert pkg.gdp_residual_norm_workspace_bytes(10, 8192) > 0 and pkg.gdp_residual_norm_workspace_bytes(10, 8193) == 0


@pytest.mark.parametrize("T,lengths", [(100, [100]), (64, [16, 0, 1, 47]), (5, [1, 1, 1, 1, 1]), (31, [15, 16]), (48, [0, 48, 0])])
def test_chunk_rows_are_apart(T, lengths):
    """Rows cu[i] / chunk + i + j of every sequence's chunks are different ones of gdp_scan_chunk_rows(T, N)."""
    seen, at = set(), 0
    for i, n in enumerate(lengths):
        for j in range(-(-n // pkg.GDP_SCAN_CHUNK)):
            row = at // pkg.GDP_SCAN_CHUNK + i + j
            assert row not in seen and 0 <= row < T // pkg.GDP_SCAN_CHUNK + len(lengths)
            seen.add(row)
        at += n


def _conv(**over):
    T, C = 8, 16
    return _with(pkg.GdpConvArgs(x=FAKE, x_stride_t=C, weight=FAKE, output=FAKE, cu_seqlens=FAKE, T=T, N=2, C=C, width=4,
                                 dtype=BF16, activation=1), over)


STATE = dict(state=1 << 22, state_indices=1 << 23, num_slots=4)
MODES = [(dict(initial_state=FAKE + 1), INVALID), (dict(state=1 << 22), INVALID), (dict(STATE, num_slots=0), INVALID),
         (dict(STATE, initial_state=1 << 24), INVALID), (dict(STATE, output_state=1 << 24), INVALID),
         (dict(initial_state=1 << 24, output_state=(1 << 24) + 64), ALIAS), (dict(cu_seqlens=None), INVALID),
         (dict(output=None), INVALID), (dict(output=FAKE + 1), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 1), INVALID),
         (dict(x_stride_t=15), INVALID), (dict(x_stride_t=-16), INVALID), (dict(T=-1), INVALID), (dict(N=-1), INVALID),
         (dict(C=0), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(C=(1 << 20) + 16), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", MODES + [
    (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(activation=2), INVALID),
    (dict(weight=None), INVALID), (dict(weight=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID)])
def test_convolution_refusals(lib, over, status):
    _refused(lib, "gdp_short_convolution", _conv(**over), status)


def _conv_back(**over):
    T, C = 8, 16
    return _with(pkg.GdpConvBackwardArgs(x=FAKE, x_stride_t=C, weight=FAKE, d_output=FAKE, d_output_stride_t=C, cu_seqlens=FAKE,
                                         T=T, N=2, C=C, width=4, dx=FAKE, d_weight=FAKE, workspace=FAKE, workspace_bytes=1 << 30,
                                         dtype=BF16, activation=1), over)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(d_output=None), INVALID), (dict(dx=None), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(d_weight=None), INVALID), (dict(bias=FAKE), INVALID), (dict(d_bias=FAKE), INVALID), (dict(d_output_stride_t=8), INVALID),
    (dict(width=5), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED), (dict(activation=2), INVALID),
    (dict(initial_state=FAKE + 1), INVALID), (dict(initial_state=1 << 24, d_initial_state=1 << 24), ALIAS),
    (dict(d_final_state=1 << 24, d_initial_state=(1 << 24) + 32), ALIAS), (dict(workspace=None), WORKSPACE),
    (dict(workspace=FAKE + 16), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE)])
def test_convolution_backward_refusals(lib, over, status):
    _refused(lib, "gdp_short_convolution_backward", _conv_back(**over), status)


def _scan(**over):
    T, C, S = 8, 16, 4
    return _with(pkg.GdpScanArgs(x=FAKE, x_stride_t=C, dt=FAKE, dt_stride_t=C, A=FAKE, B=FAKE, C_in=FAKE, B_stride_t=S, C_stride_t=S,
                                 output=FAKE, cu_seqlens=FAKE, T=T, N=2, C=C, S=S, G=1, x_dtype=BF16, dt_dtype=BF16), over)


VECTORS = [(dict(S=0), INVALID), (dict(S=65, B_stride_t=65, C_stride_t=65), UNSUPPORTED), (dict(G=0), INVALID), (dict(G=3), INVALID),
           (dict(G=2, B_stride_t=8, C_stride_t=8, B_stride_g=4, C_stride_g=3), INVALID), (dict(B=None), INVALID),
           (dict(C_in=None), INVALID), (dict(A=None), INVALID), (dict(A=FAKE + 2), INVALID), (dict(D=FAKE + 2), INVALID),
           (dict(dt_bias=FAKE + 2), INVALID), (dict(dt=None), INVALID), (dict(dt_stride_t=8), INVALID), (dict(B_stride_t=2), INVALID),
           (dict(z=FAKE, z_stride_t=8), INVALID), (dict(z=FAKE + 1, z_stride_t=16), INVALID), (dict(x_dtype=9), UNSUPPORTED),
           (dict(dt_dtype=F16), UNSUPPORTED), (dict(C=1 << 20, G=1 << 17, x_stride_t=1 << 20, dt_stride_t=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", MODES + VECTORS + [(dict(chunk_states=FAKE + 2), INVALID)])
def test_scan_refusals(lib, over, status):
    _refused(lib, "gdp_selective_scan", _scan(**over), status)


def _scan_back(**over):
    T, C, S = 8, 16, 4
    return _with(pkg.GdpScanBackwardArgs(
        x=FAKE, x_stride_t=C, dt=FAKE, dt_stride_t=C, A=FAKE, B=FAKE, C_in=FAKE, B_stride_t=S, C_stride_t=S, d_output=FAKE,
        d_output_stride_t=C, cu_seqlens=FAKE, T=T, N=2, C=C, S=S, G=1, chunk_states=FAKE, dx=FAKE, ddt=FAKE, dA=FAKE, dB=FAKE,
        dC=FAKE, workspace=FAKE, workspace_bytes=1 << 30, x_dtype=BF16, dt_dtype=F32), over)


@pytest.mark.parametrize("over,status", VECTORS + [
    (dict(d_output=None), INVALID), (dict(d_output_stride_t=8), INVALID), (dict(dx=None), INVALID), (dict(ddt=None), INVALID),
    (dict(ddt=FAKE + 2), INVALID), (dict(dA=None), INVALID), (dict(dB=None), INVALID), (dict(dC=FAKE + 1), INVALID),
    (dict(D=FAKE), INVALID), (dict(dD=FAKE), INVALID), (dict(dt_bias=FAKE), INVALID), (dict(ddt_bias=FAKE), INVALID),
    (dict(z=FAKE, z_stride_t=16), INVALID), (dict(chunk_states=None), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(d_final_state=1 << 24, d_initial_state=(1 << 24) + 64), ALIAS), (dict(workspace=None), WORKSPACE),
    (dict(workspace=FAKE + 16), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE)])
def test_scan_backward_refusals(lib, over, status):
    _refused(lib, "gdp_selective_scan_backward", _scan_back(**over), status)


def _norm(**over):
    T, C = 8, 16
    return _with(pkg.GdpResidualNormArgs(residual=FAKE, residual_stride_t=C, block=FAKE, block_stride_t=C, weight=FAKE, y=FAKE,
                                         residual_out=1 << 24, T=T, C=C, eps=1e-5, dtype=BF16, residual_dtype=F32, activation=2), over)


NORM = [(dict(T=-1), INVALID), (dict(C=0), INVALID), (dict(C=8193), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
        (dict(dtype=0), UNSUPPORTED), (dict(residual_dtype=F16), UNSUPPORTED), (dict(eps=-1.0), INVALID),
        (dict(eps=float("nan")), INVALID), (dict(activation=3), INVALID), (dict(weight=None), INVALID), (dict(block=None), INVALID),
        (dict(block=FAKE + 1), INVALID), (dict(block_stride_t=8), INVALID), (dict(gate=FAKE, gate_stride_t=8), INVALID),
        (dict(post_weight=FAKE + 2), INVALID), (dict(scale=FAKE + 2), INVALID)]


@pytest.mark.parametrize("over,status", NORM + [
    (dict(residual=None), INVALID), (dict(residual=FAKE + 2), INVALID), (dict(y=None), INVALID), (dict(residual_out=None), INVALID),
    (dict(residual_out=FAKE + 64), ALIAS), (dict(residual_out=FAKE, residual_stride_t=32), ALIAS)])
def test_residual_norm_refusals(lib, over, status):
    _refused(lib, "gdp_residual_norm", _norm(**over), status)


def _norm_back(**over):
    T, C = 8, 16
    return _with(pkg.GdpResidualNormBackwardArgs(
        d_y=FAKE, d_y_stride_t=C, residual_out=FAKE, residual_out_stride_t=C, block=FAKE, block_stride_t=C, weight=FAKE,
        d_residual=1 << 24, d_block=FAKE, d_weight=FAKE, workspace=FAKE, workspace_bytes=1 << 30, T=T, C=C, eps=1e-5, dtype=BF16,
        residual_dtype=F32, activation=2), over)


@pytest.mark.parametrize("over,status", NORM + [
    (dict(d_y=None), INVALID), (dict(residual_out=None), INVALID), (dict(d_residual=None), INVALID), (dict(d_block=None), INVALID),
    (dict(gate=FAKE, gate_stride_t=16), INVALID), (dict(d_weight=None), INVALID), (dict(post_weight=FAKE), INVALID),
    (dict(d_scale=FAKE), INVALID), (dict(d_residual_out=FAKE, d_residual_out_stride_t=8), INVALID),
    (dict(d_residual_out=(1 << 24) + 64, d_residual_out_stride_t=16), ALIAS), (dict(workspace=None), WORKSPACE),
    (dict(workspace=FAKE + 64), WORKSPACE), (dict(workspace_bytes=8), WORKSPACE)])
def test_residual_norm_backward_refusals(lib, over, status):
    _refused(lib, "gdp_residual_norm_backward", _norm_back(**over), status)


def test_null_and_nothing_to_do(lib):
    for name in ("gdp_short_convolution", "gdp_short_convolution_decode", "gdp_short_convolution_backward", "gdp_selective_scan",
                 "gdp_selective_scan_decode", "gdp_selective_scan_backward", "gdp_residual_norm", "gdp_residual_norm_backward"):
        assert getattr(lib, name)(None, None) == INVALID
    for a, names in ((_conv(T=0, N=0, x=None, output=None), ("gdp_short_convolution", "gdp_short_convolution_decode")),
                     (_scan(T=0, N=0, x=None, dt=None, B=None, C_in=None, output=None), ("gdp_selective_scan", "gdp_selective_scan_decode")),
                     (_norm(T=0, block=None, residual=None, y=None, residual_out=None), ("gdp_residual_norm",))):
        for name in names:
            assert getattr(lib, name)(ctypes.byref(a), None) == pkg.GDP_OK, pkg.gdp_last_error()
    for a, name in ((_conv(), "gdp_short_convolution_decode"), (_scan(), "gdp_selective_scan_decode")):
        _refused(lib, name, a, INVALID)  # T != N


def test_wrappers_refuse(lib, monkeypatch):
    x, cu = torch.zeros(4, 8, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    w, A, v = torch.zeros(8, 4), torch.zeros(8, 2), torch.zeros(4, 2, dtype=torch.bfloat16)
    calls = (lambda x: pkg.short_convolution(x, w, cu), lambda x: pkg.short_convolution_decode(x, w),
             lambda x: pkg.short_convolution_backward(x, w, x, cu), lambda x: pkg.selective_scan(x, x, A, v, v, cu),
             lambda x: pkg.selective_scan_decode(x, x, A, v, v), lambda x: pkg.selective_scan_backward(x, x, A, v, v, x, cu, None),
             lambda x: pkg.residual_norm(x, x, w[:, 0]), lambda x: pkg.residual_norm_backward(x, None, x, x, w[:, 0]))
    for call in calls:
        with pytest.raises(pkg.GdpError, match="CUDA device"):
            call(x)
        with pytest.raises(pkg.GdpError, match="must be bfloat16"):
            call(x.long())
    monkeypatch.setattr(layer, "_current_device", lambda: 0)
    for call in calls:
        with pytest.raises(pkg.GdpError, match="is on cuda:1, the current device is cuda:0"):
            call(_Elsewhere(4, 8))


@pytest.mark.parametrize("table,name", [(block._CONV_ACTS, "sigmoid"), (block._GATE_ACTS, "tanh"), (block._CONV_ACTS, 1)])
def test_activations(table, name):
    with pytest.raises(pkg.GdpError, match="activation must be one of"):
        block._activation(table, name)


def test_refusals_of_range(lib):
    """What is documented as out of range or as overlapping is refused before any launch."""
    far = 1 << 31
    for name in ("residual", "block", "gate"):
        a = _norm(gate=FAKE, gate_stride_t=16)
        _refused(lib, "gdp_residual_norm", _with(a, {name + "_stride_t": far}), UNSUPPORTED)
    for name in ("d_y", "d_residual_out", "residual_out", "block", "gate"):
        a = _norm_back(gate=FAKE, gate_stride_t=16, d_gate=FAKE, d_residual_out=1 << 26, d_residual_out_stride_t=16)
        _refused(lib, "gdp_residual_norm_backward", _with(a, {name + "_stride_t": far}), UNSUPPORTED)
    for at in (FAKE, FAKE + 2, FAKE + 16 * 8 * 2 - 2, FAKE - 16 * 8 * 2 + 2):
        _refused(lib, "gdp_short_convolution", _conv(output=at), ALIAS)
        _refused(lib, "gdp_short_convolution_decode", _conv(output=at, N=8), ALIAS)


def test_scan_in_pieces_needs_its_workspace(lib):
    need = pkg.gdp_scan_forward_workspace_bytes(4096, 1, 64, 16)
    assert need > 0 and pkg.gdp_scan_forward_workspace_bytes(4096, 1, 64, 16, 3) == 0
    assert pkg.gdp_scan_forward_workspace_bytes(100, 1, 64, 16) == 0  # (too short for pieces)
    one = dict(T=4096, N=1, C=64, S=16, x_stride_t=64, dt_stride_t=64, B_stride_t=16, C_stride_t=16, output=1 << 24)
    for over in (dict(workspace=None), dict(workspace=FAKE + 16, workspace_bytes=need), dict(workspace=FAKE, workspace_bytes=need - 1)):
        _refused(lib, "gdp_selective_scan", _scan(**one, **over), WORKSPACE)
