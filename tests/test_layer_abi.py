"""Host-side checks of the layer operators (no GPU needed): struct layouts, shape-only queries, and the
refusal of bad arguments before any launch, through the C ABI and the torch wrappers."""
import ctypes

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from chunked_gated_deltaproduct_gb300 import build as libbuild
from chunked_gated_deltaproduct_gb300 import layer

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return layer._library()


def test_layouts_and_queries(lib):
    for i, s in enumerate((pkg.GdpRecurrenceArgs, pkg.GdpRecurrenceBackwardArgs, pkg.GdpGroupNormArgs,
                           pkg.GdpGroupNormBackwardArgs)):
        assert lib.gdp_layer_args_size(i) == ctypes.sizeof(s)
    assert lib.gdp_layer_args_size(4) == 0
    nw = pkg.gdp_group_norm_workspace_bytes
    assert nw(100, 4, 128) > 0 and nw(100, 4, 0) == 0 and nw(100, 4, 8193) == 0


@pytest.mark.parametrize("limit", [0, 99_999, 1_000_000_001])
def test_wait_test_limits(lib, limit):
    assert lib.gdp_arm_recurrence_wait_test(limit) == pkg.GDP_ERR_INVALID_ARG and pkg.gdp_last_error() != ""


def _rec(**over):
    T, C = 8, 16
    a = pkg.GdpRecurrenceArgs(x=FAKE, x_stride_t=C, g=FAKE, g_stride_t=C, output=FAKE, cu_seqlens=FAKE, T=T, N=2, C=C,
                              x_dtype=pkg.GDP_DTYPE_BF16, g_dtype=pkg.GDP_DTYPE_BF16, gate=0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


STATE = dict(state=1 << 22, state_indices=1 << 23, num_slots=4)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), pkg.GDP_ERR_INVALID_ARG), (dict(N=-1), pkg.GDP_ERR_INVALID_ARG), (dict(C=0), pkg.GDP_ERR_INVALID_ARG),
    (dict(C=(1 << 20) + 1), pkg.GDP_ERR_UNSUPPORTED), (dict(T=1 << 31), pkg.GDP_ERR_UNSUPPORTED),
    (dict(x_dtype=0), pkg.GDP_ERR_UNSUPPORTED), (dict(x_dtype=9), pkg.GDP_ERR_UNSUPPORTED),
    (dict(g_dtype=pkg.GDP_DTYPE_F16), pkg.GDP_ERR_UNSUPPORTED),  # neither x's type nor fp32
    (dict(gate=3), pkg.GDP_ERR_INVALID_ARG), (dict(gate=-1), pkg.GDP_ERR_INVALID_ARG),
    (dict(x=None), pkg.GDP_ERR_INVALID_ARG), (dict(g=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(output=None), pkg.GDP_ERR_INVALID_ARG), (dict(cu_seqlens=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(x=FAKE + 1), pkg.GDP_ERR_INVALID_ARG), (dict(x_stride_t=15), pkg.GDP_ERR_INVALID_ARG),
    (dict(g_stride_t=0), pkg.GDP_ERR_INVALID_ARG), (dict(g_stride_t=-16), pkg.GDP_ERR_INVALID_ARG),
    (dict(initial_state=FAKE + 2), pkg.GDP_ERR_INVALID_ARG),
    (dict(state=1 << 22), pkg.GDP_ERR_INVALID_ARG), (dict(STATE, num_slots=0), pkg.GDP_ERR_INVALID_ARG),
    (dict(STATE, initial_state=1 << 24), pkg.GDP_ERR_INVALID_ARG),
    (dict(STATE, output_state=1 << 24), pkg.GDP_ERR_INVALID_ARG),
    (dict(initial_state=1 << 24, output_state=(1 << 24) + 64), pkg.GDP_ERR_ALIAS),
])
def test_recurrence_refusals(lib, over, status):
    a = _rec(**over)
    assert lib.gdp_linear_recurrence(ctypes.byref(a), None) == status, pkg.gdp_last_error()
    assert pkg.gdp_last_error() != ""


def test_recurrence_null_and_nothing_to_do(lib):
    for name in ("gdp_linear_recurrence", "gdp_linear_recurrence_decode", "gdp_linear_recurrence_backward",
                 "gdp_group_norm", "gdp_group_norm_backward"):
        assert getattr(lib, name)(None, None) == pkg.GDP_ERR_INVALID_ARG
    a = _rec(T=0, N=0, x=None, g=None, output=None)
    assert lib.gdp_linear_recurrence(ctypes.byref(a), None) == pkg.GDP_OK
    assert lib.gdp_linear_recurrence_decode(ctypes.byref(a), None) == pkg.GDP_OK
    a = _rec()  # T != N
    assert lib.gdp_linear_recurrence_decode(ctypes.byref(a), None) == pkg.GDP_ERR_INVALID_ARG


def _bwd(**over):
    T, C = 8, 16
    a = pkg.GdpRecurrenceBackwardArgs(
        g=FAKE, g_stride_t=C, h=FAKE, h_stride_t=C, d_output=FAKE, d_output_stride_t=C, cu_seqlens=FAKE, T=T, N=2, C=C,
        dx=FAKE, dg=FAKE, x_dtype=pkg.GDP_DTYPE_BF16,
        g_dtype=pkg.GDP_DTYPE_F32, gate=0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(h=None), pkg.GDP_ERR_INVALID_ARG), (dict(h_codes=FAKE, h_scales=FAKE, h_group=16), pkg.GDP_ERR_INVALID_ARG),
    (dict(h=None, h_codes=FAKE, h_group=16), pkg.GDP_ERR_INVALID_ARG),
    (dict(h=None, h_codes=FAKE, h_scales=FAKE, h_group=5), pkg.GDP_ERR_INVALID_ARG),
    (dict(gate=2), pkg.GDP_ERR_INVALID_ARG),  # the sigmoid gate needs x
    (dict(dx=None), pkg.GDP_ERR_INVALID_ARG), (dict(dg=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(d_output=None), pkg.GDP_ERR_INVALID_ARG), (dict(cu_seqlens=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(dg=FAKE + 2), pkg.GDP_ERR_INVALID_ARG), (dict(h_stride_t=8), pkg.GDP_ERR_INVALID_ARG),
    (dict(initial_state=1 << 24, d_initial_state=1 << 24), pkg.GDP_ERR_ALIAS),
    (dict(d_final_state=1 << 24, d_initial_state=(1 << 24) + 64), pkg.GDP_ERR_ALIAS),
])
def test_recurrence_backward_refusals(lib, over, status):
    a = _bwd(**over)
    assert lib.gdp_linear_recurrence_backward(ctypes.byref(a), None) == status, pkg.gdp_last_error()
    assert pkg.gdp_last_error() != ""


def _norm(**over):
    T, H, D = 8, 2, 16
    a = pkg.GdpGroupNormArgs(o=FAKE, o_stride_t=H * D, o_stride_h=D, z=FAKE, z_stride_t=H * D, z_stride_h=D, weight=FAKE,
                             y=FAKE, T=T, H=H, D=D, eps=1e-5, dtype=pkg.GDP_DTYPE_BF16, activation=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), pkg.GDP_ERR_INVALID_ARG), (dict(D=0), pkg.GDP_ERR_INVALID_ARG), (dict(H=0), pkg.GDP_ERR_INVALID_ARG),
    (dict(D=8193, o_stride_h=8193, z_stride_h=8193), pkg.GDP_ERR_UNSUPPORTED), (dict(dtype=0), pkg.GDP_ERR_UNSUPPORTED),
    (dict(eps=-1.0), pkg.GDP_ERR_INVALID_ARG), (dict(eps=float("nan")), pkg.GDP_ERR_INVALID_ARG),
    (dict(activation=3), pkg.GDP_ERR_INVALID_ARG), (dict(activation=0), pkg.GDP_ERR_INVALID_ARG),
    (dict(z=None, activation=2), pkg.GDP_ERR_INVALID_ARG), (dict(weight=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(o=None), pkg.GDP_ERR_INVALID_ARG), (dict(y=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(o=FAKE + 1), pkg.GDP_ERR_INVALID_ARG), (dict(o_stride_h=8), pkg.GDP_ERR_INVALID_ARG),
    (dict(z_stride_t=0), pkg.GDP_ERR_INVALID_ARG), (dict(weight=FAKE + 2), pkg.GDP_ERR_INVALID_ARG),
    (dict(o_codes=FAKE), pkg.GDP_ERR_INVALID_ARG), (dict(z_scales=FAKE), pkg.GDP_ERR_INVALID_ARG),
    (dict(z=None, z_codes=FAKE, z_scales=FAKE), pkg.GDP_ERR_INVALID_ARG),
])
def test_group_norm_refusals(lib, over, status):
    a = _norm(**over)
    assert lib.gdp_group_norm(ctypes.byref(a), None) == status, pkg.gdp_last_error()
    assert pkg.gdp_last_error() != ""


def _norm_bwd(**over):
    T, H, D = 8, 2, 16
    a = pkg.GdpGroupNormBackwardArgs(
        d_y=FAKE, d_y_stride_t=H * D, d_y_stride_h=D, o_codes=FAKE, o_scales=FAKE, z_codes=FAKE, z_scales=FAKE,
        weight=FAKE, d_o=FAKE, d_z=FAKE, d_weight=FAKE, workspace=FAKE, workspace_bytes=1 << 30, T=T, H=H, D=D, eps=1e-5,
        dtype=pkg.GDP_DTYPE_BF16, activation=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(o_codes=None), pkg.GDP_ERR_INVALID_ARG), (dict(o=FAKE, o_stride_t=32, o_stride_h=16), pkg.GDP_ERR_INVALID_ARG),
    (dict(o_scales=None), pkg.GDP_ERR_INVALID_ARG), (dict(z_scales=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(z=FAKE, z_stride_t=32, z_stride_h=16), pkg.GDP_ERR_INVALID_ARG),
    (dict(z=FAKE, z_stride_t=32, z_stride_h=16, z_codes=None), pkg.GDP_ERR_INVALID_ARG),  # o in codes, z a tensor
    (dict(d_z=None), pkg.GDP_ERR_INVALID_ARG), (dict(d_o=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(d_weight=None), pkg.GDP_ERR_INVALID_ARG), (dict(bias=FAKE), pkg.GDP_ERR_INVALID_ARG),
    (dict(d_bias=FAKE), pkg.GDP_ERR_INVALID_ARG), (dict(d_y=None), pkg.GDP_ERR_INVALID_ARG),
    (dict(workspace=None), pkg.GDP_ERR_WORKSPACE), (dict(workspace_bytes=4), pkg.GDP_ERR_WORKSPACE),
    (dict(workspace=FAKE + 64), pkg.GDP_ERR_WORKSPACE),
])
def test_group_norm_backward_refusals(lib, over, status):
    a = _norm_bwd(**over)
    assert lib.gdp_group_norm_backward(ctypes.byref(a), None) == status, pkg.gdp_last_error()
    assert pkg.gdp_last_error() != ""


def test_wrappers_refuse_host_tensors(lib):
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(pkg.GdpError, match="CUDA device"):
        pkg.gated_linear_recurrence(x, x, torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(pkg.GdpError, match="CUDA device"):
        pkg.gated_linear_recurrence_decode(x, x)
    with pytest.raises(pkg.GdpError, match="CUDA device"):
        pkg.gated_group_norm(x.view(4, 2, 4), torch.ones(4))
    with pytest.raises(pkg.GdpError, match=r"\[T, C\]"):
        pkg.gated_linear_recurrence(x[0], x[0], torch.tensor([0, 4], dtype=torch.int32))


def test_checkpoint_dequantizes_by_blocks():
    c = pkg.ActivationCheckpoint(torch.full((1, 1, 130), 2, dtype=torch.int8), torch.tensor([[[0.5, 3.0]]]))
    v = c.dequantize()
    assert v.shape == (1, 1, 130) and float(v[0, 0, 127]) == 1.0 and float(v[0, 0, 128]) == 6.0


@pytest.mark.parametrize("activation", [0, 1, 2])
def test_group_norm_of_an_empty_batch(lib, activation):
    """Its tensors, the gate among them, may have no address."""
    a = _norm(T=0, o=None, z=None, y=None, activation=activation)
    assert lib.gdp_group_norm(ctypes.byref(a), None) == pkg.GDP_OK, pkg.gdp_last_error()


class _Elsewhere:
    """What the checks ask of a CUDA tensor, without one."""
    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return 1

    def get_device(self):
        return 1


def test_wrappers_refuse_tensors_off_the_current_device(lib, monkeypatch):
    """The library launches on the current device; nothing is launched here."""
    monkeypatch.setattr(layer, "_current_device", lambda: 0, raising=False)
    x, o = _Elsewhere(4, 8), _Elsewhere(4, 2, 4)
    for call in (lambda: pkg.gated_linear_recurrence(x, x, None), lambda: pkg.gated_linear_recurrence_decode(x, x),
                 lambda: pkg.gated_linear_recurrence_backward(x, x, x, None), lambda: pkg.gated_group_norm(o, None),
                 lambda: pkg.gated_group_norm_backward(o, (o, None), None)):
        with pytest.raises(pkg.GdpError, match="is on cuda:1, the current device is cuda:0"):
            call()
