"""Outputs of the block operators that share memory with an input, or with one another, are refused before any launch
(no GPU needed: nothing here is launched)."""
import pytest

import chunked_gated_deltaproduct_gb300 as pkg
from chunked_gated_deltaproduct_gb300 import block
from chunked_gated_deltaproduct_gb300 import build as libbuild
from tests.test_block_abi import ALIAS, _conv_back, _norm, _norm_back, _refused, _scan, _scan_back

T, C, S = 8, 16, 4
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return block._library()


def _places(at, stride, cols, in_size, out_bytes):
    """Addresses of an output of `out_bytes` that share bytes with T rows of `cols` elements at `at`: the first and last of
    them, and within."""
    last = at + ((T - 1) * stride + cols) * in_size
    return {at, last - 2, at - out_bytes + 2, at + stride * in_size}


def _apart(fields, first=2 * MB):
    """Every tensor in a megabyte of its own."""
    return {name: first + i * MB for i, name in enumerate(fields)}


SCAN_IN = {"x": (C, 2), "dt": (C, 2), "z": (C, 2), "B": (S, 2), "C_in": (S, 2)}


@pytest.mark.parametrize("entry", ["gdp_selective_scan", "gdp_selective_scan_decode"])
@pytest.mark.parametrize("over", SCAN_IN)
def test_scan(lib, entry, over):
    cols, size = SCAN_IN[over]
    at = _apart(SCAN_IN)
    for stride in (cols, cols + 24):
        strides = {("C" if n == "C_in" else n) + "_stride_t": stride if n == over else SCAN_IN[n][0] for n in SCAN_IN}
        for out in _places(at[over], stride, cols, size, T * C * 2):
            _refused(lib, entry, _scan(**at, **strides, output=out, N=T), ALIAS)
            assert "output overlaps" in pkg.gdp_last_error()


def test_scan_over_a_group(lib):
    """The second group of B lies elsewhere; the output shares bytes with its last rows only."""
    at = _apart(SCAN_IN)
    for out in (at["B"] + 4096, at["B"] + 4096 + ((T - 1) * 8 + S) * 2 - 2):
        a = _scan(**{**at, "z": None}, G=2, B_stride_t=8, B_stride_g=2048, C_stride_t=8, C_stride_g=4, output=out)
        _refused(lib, "gdp_selective_scan", a, ALIAS)


def test_scan_backward(lib):
    ins = {**SCAN_IN, "d_output": (C, 2)}
    outs = {"dx": (C, 2), "ddt": (C, 4), "dz": (C, 2), "dB": (S, 2), "dC": (S, 2)}
    at = _apart([*ins, *outs])
    for out, (cols, size) in outs.items():
        for name, (in_cols, in_size) in {**ins, **{k: v for k, v in outs.items() if k != out}}.items():
            in_size = 4 if name == "dt" else in_size
            for place in _places(at[name], in_cols, in_cols, in_size, T * cols * size):
                place = place // size * size
                if place + T * cols * size <= at[name] or place >= at[name] + T * in_cols * in_size:
                    continue
                a = _scan_back(**{**at, out: place}, z_stride_t=C, D=None)
                _refused(lib, "gdp_selective_scan_backward", a, ALIAS)


def test_convolution_backward(lib):
    for name in ("x", "d_output"):
        at = _apart(["x", "d_output"])
        for place in _places(at[name], C + 8, C, 2, T * C * 2):
            _refused(lib, "gdp_short_convolution_backward", _conv_back(**at, **{name + "_stride_t": C + 8}, dx=place), ALIAS)


def test_residual_norm(lib):
    ins = {"residual": (C, 4), "block": (C, 2), "gate": (C, 2)}
    at = _apart([*ins, "y", "residual_out"])
    for out, size in (("y", 2), ("residual_out", 4)):
        other = {"residual_out": (C, 4)} if out == "y" else {"y": (C, 2)}
        for name, (cols, in_size) in {**ins, **other}.items():
            for place in _places(at[name], cols, cols, in_size, T * C * size):
                place = place // size * size
                if (out, name, place) == ("residual_out", "residual", at["residual"]):
                    continue  # (the stream's own buffer may be written)
                if place + T * C * size <= at[name] or place >= at[name] + T * cols * in_size:
                    continue
                _refused(lib, "gdp_residual_norm", _norm(**{**at, out: place}, gate_stride_t=C), ALIAS)


def test_residual_norm_backward(lib):
    ins = {"d_y": (C, 2), "d_residual_out": (C, 4), "residual_out": (C, 4), "block": (C, 2), "gate": (C, 2)}
    outs = {"d_residual": (C, 4), "d_block": (C, 2), "d_gate": (C, 2)}
    at = _apart([*ins, *outs])
    for out, (cols, size) in outs.items():
        for name, (in_cols, in_size) in {**ins, **{k: v for k, v in outs.items() if k != out}}.items():
            for place in _places(at[name], in_cols, in_cols, in_size, T * cols * size):
                place = place // size * size
                if (out, name, place) == ("d_residual", "d_residual_out", at["d_residual_out"]):
                    continue
                if place + T * cols * size <= at[name] or place >= at[name] + T * in_cols * in_size:
                    continue
                a = _norm_back(**{**at, out: place}, d_residual_out_stride_t=C, gate_stride_t=C)
                _refused(lib, "gdp_residual_norm_backward", a, ALIAS)


def test_strides_of_no_size(lib):
    """Strides that no memory has do not stop the check."""
    for stride in (1 << 61, 1 << 62, (1 << 63) - 1):
        a = _scan(**{**_apart(SCAN_IN), "z": None}, x_stride_t=stride, output=2 * MB)
        _refused(lib, "gdp_selective_scan", a, ALIAS)
