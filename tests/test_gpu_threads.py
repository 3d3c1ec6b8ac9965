"""Calls from host threads of their own: the first call of a thread, whichever it is, and two threads at once that run the
same kernels with different amounts of shared memory."""
import ctypes
import threading

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from chunked_gated_deltaproduct_gb300 import binding, layer
from gdp_workloads import make_custom
from tests.gpu_helpers import to_dev
from tests.test_gpu_block import _cu, _rand
from tests.test_gpu_block_edges import Block
from tests.test_gpu_block_paths import _from_two_threads, _same

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _calls(dev):
    """One call of every kind into buffers that are there, by name: (call, the buffers it writes)."""
    T, C = 40, 64
    b, cu = Block(T, C, 16, 1, dev), _cu([T], dev)
    g, s0 = -b.dt.abs(), torch.zeros((1, C), device=dev)
    h, y, r = torch.empty_like(b.x), torch.empty_like(b.x), torch.empty_like(b.res)
    w = make_custom([130, 70], 2, 128, 2, seed=1, init_sigma=0.1, decay=0.05)
    d = to_dev(w, dev)
    room = pkg.alloc_workspace(w.T, 2, 2, 128, 128, 2, dev)
    o = torch.empty((w.T, 2, 128), dtype=BF16, device=dev)
    args = (d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], 2, w.scale)
    heads = b.x.view(T, 1, C)
    return {
        "recurrence": (lambda: pkg.gated_linear_recurrence(b.x, g, cu, output=h, initial_state=s0), (h,)),
        "recurrence step": (lambda: pkg.gated_linear_recurrence_decode(b.x, g, output=h), (h,)),
        "recurrence backward": (lambda: pkg.gated_linear_recurrence_backward(g, b.x, b.dy, cu), ()),
        "group norm": (lambda: pkg.gated_group_norm(heads, b.weight, b.z.view(T, 1, C)), ()),
        "convolution": (lambda: pkg.short_convolution(b.x, b.w, cu, output=y), (y,)),
        "convolution step": (lambda: pkg.short_convolution_decode(b.x, b.w, output=y), (y,)),
        "convolution backward": (lambda: pkg.short_convolution_backward(b.x, b.w, b.dy, cu), ()),
        "scan": (lambda: b.scan(cu, output=y), (y,)),
        "scan step": (lambda: pkg.selective_scan_decode(b.x, b.dt, b.A, b.B, b.Cm, output=y), (y,)),
        "residual norm": (lambda: b.norm(output=y, output_residual=r), (y, r)),
        "residual norm backward": (lambda: b.norm_backward(b.res), ()),
        "prefill": (lambda: pkg.chunk_gated_delta_product(*args, initial_state=d["init"], output=o, workspace=room), (o,)),
        "fused prefill": (lambda: pkg.chunk_gated_delta_product(*args, initial_state=d["init"], output=o, workspace=room, fused=True), (o,)),
    }


NAMES = ["recurrence", "recurrence step", "recurrence backward", "group norm", "convolution", "convolution step", "convolution backward", "scan",
         "scan step", "residual norm", "residual norm backward", "prefill", "fused prefill"]


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_thread(cuda_device, name):
    """A thread that has made no call to CUDA yet."""
    call, outs = _calls(cuda_device)[name]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    failures = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001 (what it was is shown below)
            failures.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failures, failures
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def _entry(lib, name, a):
    def call():
        if getattr(lib, name)(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) != pkg.GDP_OK:
            raise RuntimeError(pkg.gdp_last_error())
    return call


def test_recurrence_from_two_threads(cuda_device):
    """One CTA and several to a cluster."""
    dev, lib, C = cuda_device, layer._library(), 64
    calls, outs, want, held = [], [], [], []
    for i, T in enumerate((20, 600)):
        x, g, dy, s0 = (_rand(s, 10 * i + k).to(dev) for k, s in enumerate(((T, C), (T, C), (T, C), (1, C))))
        x, dy, g, cu = x.to(BF16), dy.to(BF16), -g.abs().to(BF16), _cu([T], dev)
        h, fin = pkg.gated_linear_recurrence(x, g, cu, gate="log", initial_state=s0, output_final_state=True)
        d = pkg.gated_linear_recurrence_backward(g, h, dy, cu, gate="log", initial_state=s0)
        want.append({"h": h, "fin": fin, "dx": d["dx"], "dg": d["dg"]})
        out = {k: torch.empty_like(v) for k, v in want[-1].items()}
        outs.append(out)
        at = lambda t: t.data_ptr()  # noqa: E731
        common = dict(g=at(g), g_stride_t=C, cu_seqlens=at(cu), T=T, N=1, C=C, initial_state=at(s0), x_dtype=pkg.GDP_DTYPE_BF16,
                      g_dtype=pkg.GDP_DTYPE_BF16, gate=layer.GDP_GATE_LOG)
        f = pkg.GdpRecurrenceArgs(x=at(x), x_stride_t=C, output=at(out["h"]), output_state=at(out["fin"]), **common)
        b = pkg.GdpRecurrenceBackwardArgs(h=at(h), h_stride_t=C, d_output=at(dy), d_output_stride_t=C, dx=at(out["dx"]), dg=at(out["dg"]), **common)
        calls.append((_entry(lib, "gdp_linear_recurrence", f), _entry(lib, "gdp_linear_recurrence_backward", b)))
        held += [x, g, dy, s0, cu, h]
    for k in range(2):
        _from_two_threads([c[k] for c in calls], 30000)
    for got, w in zip(outs, want):
        _same(got, w)


@pytest.mark.parametrize("kind", ["prefill", "fused", "backward"])
def test_prefill_from_two_threads(cuda_device, kind):
    """Two householder counts: the stages of the scans and of the chunk kernels differ in size."""
    dev, lib = cuda_device, binding.load_library()
    calls, outs, want, held = [], [], [], []
    for M in (2, 5) if kind != "fused" else (2, 4):
        w = make_custom([130, 70], 2, 128, M, seed=M, init_sigma=0.1, decay=0.05)
        d = to_dev(w, dev)
        args = (d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], M)
        if kind == "backward":
            do = _rand((w.T, 2, 128), 3, BF16).to(dev)
            call = lambda a=args, s=w.scale, x=do, i=d["init"]: pkg.chunk_gated_delta_product_backward(*a, x, scale=s, initial_state=i)  # noqa: E731
        else:
            def call(a=args, s=w.scale, i=d["init"]):
                o, fin = pkg.chunk_gated_delta_product(*a, s, initial_state=i, output_final_state=True, fused=kind == "fused")
                return {"o": o, "fin": fin}
        first = call()
        want.append(first)
        outs.append([None])
        held += [d, args]

        def work(call=call, out=outs[-1]):
            out[0] = call()
        calls.append(work)
    _from_two_threads(calls, 400)
    for got, w in zip(outs, want):
        got = got[0]
        assert got.keys() == w.keys()
        _same(got, w)
    if kind != "prefill":
        return
    # the launches alone, as close to one another as can be
    entries, rooms = [], []
    for M in (2, 5):
        w = make_custom([130, 70], 2, 128, M, seed=M, init_sigma=0.1, decay=0.05)
        d = to_dev(w, dev)
        o, room = torch.empty((w.T, 2, 128), dtype=BF16, device=dev), pkg.alloc_workspace(w.T, 2, 2, 128, 128, M, dev)
        a = binding.make_args(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], M, w.scale, d["init"], None, None, o, None, None, None, None,
                              None, None, None, False, room, None)
        entries.append(_entry(lib, "gdp_prefill_varlen", a))
        rooms += [d, o, room, a]
    _from_two_threads(entries, 2000)
    for o, w in zip(rooms[1::4], want):
        assert torch.equal(o, w["o"])
