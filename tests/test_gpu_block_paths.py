"""The block operators' paths that only some shapes take, against the float64 references or against the same calls on
another path: padded states, several sequences per CTA, longest-first order, long runs of rows, pieces in graphs, on
given streams, in given workspaces and beside one another, calls from two host threads."""
import ctypes
import math
import threading

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from chunked_gated_deltaproduct_gb300 import block
from tests import _block_ref as R
from tests._layer_ref import TINY, UNIT, check
from tests.test_gpu_block import _as_laid_out, _close, _cu, _on, _rand
from tests.test_gpu_block_edges import Block

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _sms(dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count


def _tiles(C, S, G):
    """CTAs that share the channels: 128 threads, four states a lane."""
    lanes = 4 if S <= 16 else 8 if S <= 32 else 16
    return G * -(-(C // G) * lanes // 128)


# ---- padded states -----------------------------------------------------------------------------------

@pytest.mark.parametrize("lengths,C", [([40, 0, 9], 24), ([600], 20), ([129, 127, 128, 640], 9)])
@pytest.mark.parametrize("S", [3, 16, 20, 33])
def test_large_negative_steps(cuda_device, lengths, C, S):
    """Steps without softplus may be far below zero: states of slow channels grow by a finite factor, whatever number of
    states the lanes are padded to, forward and backward, whole and in pieces, and token by token."""
    dev, T, N = cuda_device, sum(lengths), len(lengths)
    whole = T < 96 * N
    assert (pkg.gdp_scan_forward_workspace_bytes(T, N, C, S) == 0) == whole
    x, B, Cm, dy = (_rand(s, i) for i, s in enumerate(((T, C), (T, S), (T, S), (T, C))))
    dt, A = _rand((T, C), 4).abs() * 0.5, -0.005 * torch.rand((C, S), generator=torch.Generator().manual_seed(5)) - 0.005
    dt[5::60], dt[36::120] = -200.0, -1000.0   # factors of up to e^2 and e^10
    dt[6::60], dt[37::120] = 150.0, 900.0      # and most of the way back
    D, h0, dfin = _rand((C,), 6), _rand((N, C, S), 7), _rand((N, C, S), 8)
    ins, (gD, gh0, gdy, gdfin), cu = [t.to(dev) for t in (x, dt, A, B, Cm)], _on(dev, D, h0, dy, dfin), _cu(lengths, dev)
    y, fin, kept = pkg.selective_scan(*ins, cu, D=gD, dt_softplus=False, initial_state=gh0, output_final_state=True, save_states=True)
    want = R.scan(x, dt, A, B, Cm, lengths, D=D, softplus=False, init=h0)
    check(y, *want["y"], "y")
    check(fin, *want["final"], "final state")
    got = pkg.selective_scan_backward(*ins, gdy, cu, kept, D=gD, dt_softplus=False, d_final_state=gdfin, output_d_initial_state=True)
    _close(got, R.scan_backward(x, dt, A, B, Cm, dy, lengths, D=D, softplus=False, init=h0, dfin=dfin))
    at = torch.tensor([5, 36] if T > 36 else [5])
    few = [t[at] if t.shape[0] == T else t for t in (x, dt, A, B, Cm)]
    start = _rand((len(at), C, S), 9)
    y, fin = pkg.selective_scan_decode(*(t.to(dev) for t in few), D=gD, dt_softplus=False, initial_state=start.to(dev), output_final_state=True)
    want = R.scan(*few, [1] * len(at), D=D, softplus=False, init=start)
    check(y, *want["y"], "step")
    check(fin, *want["final"], "state after the step")


# ---- decays ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("k", range(-14, -2))
def test_decays_next_to_one(cuda_device, k):
    """What a state forgets per token has next to no bias: the error of long memory is that times the tokens.  (The hardware's
    exponential alone is low by up to 0.44 2^-24 here; 0.3 is left, and the mean over 32768 states of 90 tokens' other
    roundings, each below 2^-24, is below 3 2^-24 / sqrt(90 x 32768) a token.)"""
    dev, N, n, C, S = cuda_device, 64, 90, 32, 16
    T, g = N * n, torch.Generator().manual_seed(k + 100)
    dt = 2.0 ** k * math.log(2) * (1 + torch.rand((T, C), generator=g))  # exponents in base 2 from -2^(k + 1) to -2^k
    A, h0 = -torch.ones(C, S), 1 + torch.rand((N, C, S), generator=g)
    zero, cu = torch.zeros((T, C), device=dev), _cu([n] * N, dev)
    rows = torch.zeros((T, S), device=dev)
    fin = pkg.selective_scan(zero, dt.to(dev), A.to(dev), rows, rows, cu, dt_softplus=False, initial_state=h0.to(dev), output_final_state=True)[1]
    want = h0.double() * torch.exp(-dt.double().view(N, n, C).sum(1))[..., None]
    bias = float((fin.cpu().double() / want - 1).mean()) / n * 2 ** 24
    assert abs(bias) <= 0.3 + 0.01, bias
    step = pkg.selective_scan_decode(zero, dt.to(dev), A.to(dev), rows, rows, dt_softplus=False, initial_state=torch.ones((T, C, S), device=dev),
                                     output_final_state=True)[1]
    bias = float((step.cpu().double() / torch.exp(-dt.double())[..., None] - 1).mean()) * 2 ** 24
    assert abs(bias) <= 0.3 + 0.01, bias


@pytest.mark.parametrize("S", [5, 16])
def test_a_step_of_zero_keeps_the_state(cuda_device, S):
    """To the bit: a step of zero (softplus of the lowest value, too) takes nothing in and forgets nothing."""
    dev, C, lengths = cuda_device, 24, [70, 0, 33]
    b, cu = Block(103, C, S, 3, dev, F32), _cu(lengths, dev)
    for dt, softplus in ((torch.zeros_like(b.dt), False), (torch.full_like(b.dt, torch.finfo(F32).min), True)):
        y, fin, kept = pkg.selective_scan(b.x, dt, b.A, b.B, b.Cm, cu, dt_softplus=softplus, initial_state=b.h0, output_final_state=True, save_states=True)
        assert torch.equal(fin, b.h0)
        d = pkg.selective_scan_backward(b.x, dt, b.A, b.B, b.Cm, torch.zeros_like(b.x), cu, kept, dt_softplus=softplus, d_final_state=b.h0,
                                        output_d_initial_state=True)
        assert torch.equal(d["d_initial_state"], b.h0)
        step = pkg.selective_scan_decode(b.x[:3], dt[:3], b.A, b.B[:3], b.Cm[:3], dt_softplus=softplus, initial_state=b.h0, output_final_state=True)[1]
        assert torch.equal(step, b.h0)


# ---- the gate's slope --------------------------------------------------------------------------------

@pytest.mark.parametrize("C", [64, 61, 520])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_slope_of_an_open_gate(cuda_device, dtype, C):
    """The gradient of a sigmoid gate keeps its relative precision where the gate is all but open or closed."""
    dev, most = cuda_device, 80.0 if dtype != F16 else 15.0
    T = 41
    gate = torch.linspace(-most, most, T * C).view(T, C).to(dtype)
    rows, dr, w = _rand((T, C), 1).sign().mul(1024.0).to(dtype), 1 + _rand((T, C), 2).abs(), torch.ones(C)
    r = _rand((T, C), 3)
    zero = torch.zeros((T, C), dtype=dtype, device=dev)
    got = pkg.residual_norm_backward(zero, dr.to(dev), r.to(dev), rows.to(dev), w.to(dev), gate=gate.to(dev), activation="sigmoid")["d_gate"]
    v = gate.double()
    want = dr.double() * rows.double() * torch.sigmoid(v) * torch.sigmoid(-v)
    # (d_gate = dr rows q (1 - q): each half off by act_error, three products, one rounding to the type)
    assert bool((want.abs() > 64 * TINY[dtype]).all())
    error = (got.cpu().double() - want).abs() / want.abs()
    bound = 2 * R.act_error(v) + 4 * R.U + UNIT[dtype] + TINY[dtype] / want.abs()
    assert bool((error <= bound).all()), float((error - bound).max())


# ---- bounds of no rows -------------------------------------------------------------------------------

def test_bounds_of_no_rows_backward(cuda_device):
    """The backward passes check bounds where there are no rows too; empty sequences pass the states' gradients on."""
    dev = cuda_device
    b = Block(0, 24, 16, 2, dev)
    kept = torch.empty((2, 24, 16), device=dev)
    for bounds, bad in (([0, 0, 0], False), ([0, 3, 3], True), ([0, 0, 1], True), ([-1, 0, 0], True)):
        cu = torch.tensor(bounds, dtype=torch.int32, device=dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        d = b.conv_backward(cu, initial_state=b.c0, d_final_state=b.c0, device_status=status)
        assert bool(int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS) == bad, bounds
        assert torch.equal(d["d_initial_state"], b.c0) and not d["dweight"].any() and not d["dbias"].any()
        status.zero_()
        d = b.conv_backward(cu, device_status=status)
        assert bool(int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS) == bad and not d["dweight"].any() and not d["dbias"].any()
        status.zero_()
        assert not b.conv_backward(cu, initial_state=b.c0, device_status=status)["d_initial_state"].any()
        assert bool(int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS) == bad
        status.zero_()
        d = b.scan_backward(cu, kept, d_final_state=b.h0, output_d_initial_state=True, device_status=status)
        assert bool(int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS) == bad, bounds
        assert torch.equal(d["d_initial_state"], b.h0) and not d["dA"].any() and not d["dD"].any()


# ---- two host threads --------------------------------------------------------------------------------

def _from_two_threads(calls, times):
    """Every call `times` times from a host thread of its own, all at once, each thread on its own stream."""
    failures, start = [], threading.Barrier(len(calls))

    def work(call):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            try:
                for _ in range(times):
                    call()
            except Exception as e:  # noqa: BLE001 (what it was is shown below)
                failures.append(repr(e))
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


def _same(got, want):
    for name, v in want.items():
        assert (v is None and got[name] is None) or torch.equal(got[name], v), name


def _norm_call(name, args, fields):
    """The C entry with arguments that are filled in once, so that a thread does little else than launch."""
    lib, a = block._library(), args(**{k: v.data_ptr() if isinstance(v, torch.Tensor) else v for k, v in fields.items()})

    def call():
        if getattr(lib, name)(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) != pkg.GDP_OK:
            raise RuntimeError(pkg.gdp_last_error())

    return call


def test_residual_norm_from_two_threads(cuda_device):
    """Calls of one kernel that ask for different amounts of shared memory (with and without a gate), from two host threads
    at once."""
    dev, T, C = cuda_device, 6, 4096
    blocks = [Block(T, C, 1, 1, dev, seed=s) for s in (0, 50)]
    calls, outs, want = [], [], []
    for b, gate in zip(blocks, (True, False)):
        how = dict(post_weight=b.post, gate=b.gate if gate else None, activation="silu")
        y, r = pkg.residual_norm(b.res, b.x, b.weight, **how)
        want.append({"y": y, "r": r, **pkg.residual_norm_backward(b.dy, b.dr if gate else None, b.res, b.x, b.weight, **how)})
        out = {k: None if v is None else torch.empty_like(v) for k, v in want[-1].items()}
        room = torch.empty(pkg.gdp_residual_norm_workspace_bytes(T, C), dtype=torch.uint8, device=dev)
        outs.append(out)
        common = dict(block=b.x, block_stride_t=C, gate=b.gate if gate else 0, gate_stride_t=C, weight=b.weight, post_weight=b.post, T=T,
                      C=C, eps=1e-5, dtype=pkg.GDP_DTYPE_BF16, residual_dtype=pkg.GDP_DTYPE_F32, activation=block.GDP_ACT_SILU)
        forward = _norm_call("gdp_residual_norm", pkg.GdpResidualNormArgs,
                             dict(common, residual=b.res, residual_stride_t=C, y=out["y"], residual_out=out["r"]))
        backward = _norm_call("gdp_residual_norm_backward", pkg.GdpResidualNormBackwardArgs,
                              dict(common, d_y=b.dy, d_y_stride_t=C, d_residual_out=b.dr if gate else 0, d_residual_out_stride_t=C,
                                   residual_out=b.res, residual_out_stride_t=C, d_residual=out["d_residual"], d_block=out["d_block"],
                                   d_gate=out["d_gate"] if gate else 0, d_weight=out["dweight"], d_post_weight=out["dpost_weight"],
                                   workspace=room, workspace_bytes=room.numel()))
        calls.append((forward, backward))
    for k in range(2):
        _from_two_threads([c[k] for c in calls], 20000)
    for got, w in zip(outs, want):
        _same(got, w)


# ---- outputs between strided rows --------------------------------------------------------------------

def test_outputs_in_the_gaps_of_strided_rows(cuda_device):
    """An output may lie where a strided input has a gap: no byte is shared, and the call is served."""
    dev, T, C = cuda_device, 3, 8
    room = _rand((2, 400), 1).to(dev)
    x, z = (r[:T * 100].view(T, 100)[:, 4:4 + C] for r in room)
    gap = lambda r: r[20:20 + T * C].view(T, C)  # noqa: E731
    B, w, cu = _rand((T, 4), 2).to(dev), _rand((C, 3), 3).to(dev), _cu([T], dev)
    A, ones = -torch.rand((C, 4), device=dev), torch.ones(C, device=dev)
    for call in (lambda **k: pkg.short_convolution(x, w, cu, **k), lambda **k: pkg.short_convolution_decode(x, w, **k),
                 lambda **k: pkg.selective_scan(x, x, A, B, B, cu, z=z, **k), lambda **k: pkg.selective_scan_decode(x, x, A, B, B, z=z, **k),
                 lambda **k: pkg.residual_norm(x, z, ones, ones, z, **k)[0]):
        want = call()
        assert torch.equal(call(output=gap(room[0])), want) and torch.equal(call(output=gap(room[1])), want)
        for out in (x, z):  # (one row further: an input's)
            with pytest.raises(pkg.GdpError):
                call(output=out.as_strided((T, C), (C, 1)))
            if out is x and "convolution" in str(call.__code__.co_names):
                break
    r = pkg.residual_norm(x, z, ones, output_residual=gap(room[0]))[1]
    assert torch.equal(r, x + z)
