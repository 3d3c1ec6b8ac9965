"""Calls from host threads of their own: the first call of a thread, whichever it is, and two threads at once that run the
same kernels with different amounts of shared memory."""
import threading

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from gdp_workloads import make_custom
from tests.gpu_helpers import to_dev
from tests.test_gpu_block import _cu, _rand
from tests.test_gpu_block_edges import Block

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
