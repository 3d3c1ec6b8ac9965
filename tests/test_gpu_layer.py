"""The layer operators on the GPU against the float64 references, each element within the derived
bounds of ``tests/_layer_ref.py``."""
import math

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from tests import _layer_ref as R

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(shape, seed, dtype=F32, sigma=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * sigma).to(dtype)


def _gates(kind, shape, seed, dtype):
    if kind == "sigmoid":
        return (torch.randn(shape, generator=_gen(seed)) * 2 + 1).to(dtype)
    g = -torch.rand(shape, generator=_gen(seed)) * 0.1
    g[torch.rand(shape, generator=_gen(seed + 1)) < 0.02] = -20.0  # a few that forget everything
    return (g if kind == "log" else g.exp()).to(dtype)


def _cu(lengths, dev, dtype=torch.int32):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=dtype, device=dev)


def _as_laid_out(t, how, dev):
    """The tensor on the GPU as a contiguous one, as a slice of wider rows, or as a slice whose rows
    start off every vector boundary."""
    t = t.to(dev)
    if how == "dense":
        return t
    pad = 16 if how == "slice" else 3
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + 2 * pad,), math.nan, dtype=t.dtype, device=dev)
    wide[..., pad:pad + t.shape[-1]] = t
    return wide[..., pad:pad + t.shape[-1]]


RAGGED = [100, 257, 0, 64, 1, 1000, 0]
SHAPES = [
    (RAGGED, 128, BF16, BF16, "log", "dense"),
    (RAGGED, 96, BF16, F32, "sigmoid", "slice"),
    (RAGGED, 61, F16, F16, "sigmoid", "odd"),
    (RAGGED, 66, BF16, BF16, "log", "odd"),
    (RAGGED, 33, F32, F32, "log", "odd"),
    (RAGGED, 64, F32, F32, "sigmoid", "dense"),
    ([1], 1, BF16, BF16, "log", "dense"),
    ([1], 200, F16, F32, "alpha", "dense"),
    ([2, 3], 7, BF16, F32, "alpha", "odd"),
    ([127], 64, BF16, BF16, "log", "dense"), ([128], 64, BF16, BF16, "log", "dense"),
    ([129], 64, BF16, BF16, "sigmoid", "dense"), ([64, 64, 64], 8, F16, F16, "log", "dense"),
    ([15, 1, 16, 17, 31, 33], 130, BF16, BF16, "log", "slice"),
    ([1] * 300, 72, BF16, F32, "sigmoid", "dense"),
    ([5000], 40, BF16, BF16, "log", "dense"),
    ([3000, 2999], 65, F16, F32, "alpha", "dense"),
]


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("lengths,C,xt,gt,kind,layout", SHAPES)
def test_recurrence(cuda_device, lengths, C, xt, gt, kind, layout, init):
    T, N, dev = sum(lengths), len(lengths), cuda_device
    x, g = _rand((T, C), 1, xt), _gates(kind, (T, C), 2, gt)
    s0 = _rand((N, C), 3) if init else None
    h, fin = pkg.gated_linear_recurrence(
        _as_laid_out(x, layout, dev), _as_laid_out(g, layout, dev),
        _cu(lengths, dev, torch.int64 if init else torch.int32), gate=kind,
        initial_state=s0.to(dev) if init else None, output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, g, lengths, kind, s0)
    R.check(h, rh, eh, "h")
    R.check(fin, rfin, efin, "final state")


@pytest.mark.parametrize("saved", ["h", "codes"])
@pytest.mark.parametrize("lengths,C,xt,gt,kind,layout", SHAPES)
def test_recurrence_backward(cuda_device, lengths, C, xt, gt, kind, layout, saved):
    T, N, dev = sum(lengths), len(lengths), cuda_device
    x, g, h, dh = (_rand((T, C), i, xt) for i in (1, 2, 3, 4))
    g = _gates(kind, (T, C), 2, gt)
    s0, dfin = (_rand((N, C), 5), _rand((N, C), 6)) if C % 2 == 0 else (None, None)
    if saved == "codes":
        H = 2 if C % 2 == 0 else 1
        kept = h.view(T, H, C // H)
        codes, scales, values = R.quantize(kept)
        h_in, href = pkg.ActivationCheckpoint(codes.to(dev), scales.float().to(dev)), values.view(T, C)
    else:
        h_in, href = _as_laid_out(h, layout, dev), h
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    got = pkg.gated_linear_recurrence_backward(
        _as_laid_out(g, layout, dev), h_in, _as_laid_out(dh, layout, dev), _cu(lengths, dev), gate=kind,
        x=_as_laid_out(x, layout, dev) if kind == "sigmoid" else None, initial_state=on(s0), d_final_state=on(dfin))
    dx, dg, dinit, ex, eg, einit = R.recurrence_backward(g, href, dh, lengths, kind, x, s0, dfin)
    R.check(got["dx"], dx, ex, "dx")
    R.check(got["dg"], dg, eg + 2.0 ** -23 * dg.abs(), "dg")
    if s0 is None:
        assert got["d_initial_state"] is None
    else:
        R.check(got["d_initial_state"], dinit, einit, "d_initial_state")


def test_recurrence_gradient_against_differences(cuda_device):
    """The GPU's own forward, moved by a step in fp32, against its gradients."""
    lengths, C, dev = [70, 0, 130], 8, cuda_device
    T = sum(lengths)
    x, g, s0 = _rand((T, C), 1).to(dev), _gates("sigmoid", (T, C), 2, F32).to(dev), _rand((3, C), 3).to(dev)
    dh, dfin, cu = _rand((T, C), 4).to(dev), _rand((3, C), 5).to(dev), _cu(lengths, dev)

    def loss(x, g, s0):
        h, fin = pkg.gated_linear_recurrence(x, g, cu, gate="sigmoid", initial_state=s0, output_final_state=True)
        return float((h.double() * dh).sum() + (fin.double() * dfin).sum())

    h = pkg.gated_linear_recurrence(x, g, cu, gate="sigmoid", initial_state=s0)
    d = pkg.gated_linear_recurrence_backward(g, h, dh, cu, gate="sigmoid", x=x, initial_state=s0, d_final_state=dfin)
    step = 2.0 ** -6
    for i, (name, at) in enumerate((("dx", (10, 3)), ("dx", (199, 0)), ("dg", (69, 5)), ("dg", (70, 1)),
                                    ("d_initial_state", (0, 2)), ("d_initial_state", (1, 4)))):
        vals = []
        for s in (step, -step):
            moved = {"dx": x.clone(), "dg": g.clone(), "d_initial_state": s0.clone()}
            moved[name][at] += s
            vals.append(loss(moved["dx"], moved["dg"], moved["d_initial_state"]))
        # central difference: step^2 / 6 of a third derivative of order one, and fp32 noise of about
        # 2^-22 times the sums of |h| over the affected tokens (under 100), over 2 step
        assert abs((vals[0] - vals[1]) / (2 * step) - float(d[name][at])) < 2e-3 * max(1.0, abs(float(d[name][at]))), (name, at)


@pytest.mark.parametrize("kind,xt,gt,C,N", [("log", BF16, F32, 128, 9), ("sigmoid", F16, F16, 33, 4), ("alpha", F32, F32, 8, 1),
                                            ("sigmoid", BF16, BF16, 2050, 70)])
@pytest.mark.parametrize("mode", ["dense", "in place", "cache", "zero"])
def test_decode(cuda_device, kind, xt, gt, C, N, mode):
    dev = cuda_device
    x, g, s0 = _rand((N, C), 1, xt), _gates(kind, (N, C), 2, gt), _rand((N, C), 3)
    ref_init = s0.clone()
    if mode == "cache":
        slots = torch.randperm(N + 5, generator=_gen(4))[:N].to(torch.int32)
        slots[N // 2] = -1
        ref_init[N // 2] = 0
        cache = _rand((N + 5, C), 5)
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                cache[s] = s0[i]
        got = cache.to(dev)
        h = pkg.gated_linear_recurrence_decode(x.to(dev), g.to(dev), gate=kind, state=got, state_indices=slots.to(dev))
        fin = got.cpu()[slots.long().clamp(min=0)]
        used = [s for s in slots.tolist() if s >= 0]
        rest = [i for i in range(N + 5) if i not in used]
        assert torch.equal(got.cpu()[rest], cache[rest])
    else:
        init = None if mode == "zero" else s0.to(dev)
        h, fin = pkg.gated_linear_recurrence_decode(x.to(dev), g.to(dev), gate=kind, initial_state=init,
                                                    output_final_state=True, output_state=init if mode == "in place" else None)
        if mode == "zero":
            ref_init.zero_()
    rh, rfin, eh, efin = R.recurrence(x, g, [1] * N, kind, ref_init)
    live = [i for i in range(N) if not (mode == "cache" and i == N // 2)]
    R.check(h, rh, eh, "h")
    R.check(fin.cpu()[live], rfin[live], efin[live], "state")


def test_prefill_cache_then_decode_equals_whole(cuda_device):
    """A prefill over the cache, cut at any token, and decode steps continue to the same states."""
    lengths, C, dev = [300, 40, 129], 72, cuda_device
    x, g = _rand((sum(lengths), C), 1, BF16).to(dev), _gates("log", (sum(lengths), C), 2, F32).to(dev)
    cache, slots = _rand((5, C), 3).to(dev), torch.tensor([4, 0, 2], dtype=torch.int32, device=dev)
    whole = cache.clone()
    h = pkg.gated_linear_recurrence(x, g, _cu(lengths, dev), state=whole, state_indices=slots)
    starts = [0, 300, 340]
    keep = torch.cat([torch.arange(s, s + n - 2) for s, n in zip(starts, lengths)]).to(dev)
    h2 = torch.empty_like(h)
    h2[keep] = pkg.gated_linear_recurrence(x[keep], g[keep], _cu([n - 2 for n in lengths], dev), state=cache,
                                           state_indices=slots)
    for back in (2, 1):
        at = torch.tensor([s + n - back for s, n in zip(starts, lengths)], device=dev)
        h2[at] = pkg.gated_linear_recurrence_decode(x[at], g[at], state=cache, state_indices=slots)
    rh, rfin, eh, efin = R.recurrence(x.cpu(), g.cpu(), lengths, "log", _rand((5, C), 3)[[4, 0, 2]])
    R.check(h, rh, eh, "whole")
    R.check(h2, rh, eh, "cut")
    R.check(cache[slots.long()], rfin, efin, "cut state")
    R.check(whole[slots.long()], rfin, efin, "whole state")
    assert torch.equal(cache[[1, 3]].cpu(), _rand((5, C), 3)[[1, 3]])


def test_sequences_do_not_touch_each_other(cuda_device):
    """Infinities and NaN in one sequence (states, inputs, gates) leave its neighbours' bits alone."""
    lengths, C, dev = [200, 50, 130, 9], 64, cuda_device
    cu = _cu(lengths, dev)
    x, g, s0 = _rand((sum(lengths), C), 1, BF16).to(dev), _gates("log", (sum(lengths), C), 2, BF16).to(dev), _rand((4, C), 3).to(dev)
    dh = _rand((sum(lengths), C), 4, BF16).to(dev)

    def both(x, g, s0, dh):
        h, fin = pkg.gated_linear_recurrence(x, g, cu, initial_state=s0, output_final_state=True)
        d = pkg.gated_linear_recurrence_backward(g, h, dh, cu, initial_state=s0)
        return h, fin, d["dx"], d["dg"], d["d_initial_state"]

    clean = both(x, g, s0, dh)
    x2, g2, s2, dh2 = x.clone(), g.clone(), s0.clone(), dh.clone()
    x2[210], g2[215], s2[1], dh2[240] = math.inf, math.nan, -math.inf, math.nan
    for a, b in zip(clean, both(x2, g2, s2, dh2)):
        rows = [slice(0, 200), slice(250, 389)] if a.shape[0] == 389 else [slice(0, 1), slice(2, 4)]
        for r in rows:
            assert torch.equal(a[r], b[r])


def test_special_gates_and_states(cuda_device):
    """A decay of exactly zero drops a finite state; an infinite state decays to infinity, as the
    definition has it."""
    dev = cuda_device
    x = torch.ones((4, 8), dtype=F32, device=dev)
    g = torch.zeros((4, 8), dtype=F32, device=dev)
    g[1] = -math.inf
    s0 = torch.full((1, 8), 5.0, device=dev)
    h = pkg.gated_linear_recurrence(x, g, _cu([4], dev), initial_state=s0)
    assert h[:, 0].tolist() == [6.0, 1.0, 2.0, 3.0]
    s0[0, 3] = math.inf
    h = pkg.gated_linear_recurrence(x, torch.zeros_like(g), _cu([4], dev), initial_state=s0)
    assert bool(torch.isinf(h[:, 3]).all()) and h[:, 4].tolist() == [6.0, 7.0, 8.0, 9.0]
    g = torch.tensor([[-200.0, 200.0, -math.inf, math.inf, 0.0]], device=dev)
    h = pkg.gated_linear_recurrence(torch.full((1, 5), 3.0, device=dev), g, _cu([1], dev), gate="sigmoid",
                                    initial_state=torch.full((1, 5), 7.0, device=dev))
    assert h[0].tolist() == [3.0, 7.0, 3.0, 7.0, 5.0]


def test_empty_calls(cuda_device):
    dev = cuda_device
    none = torch.empty((0, 24), dtype=BF16, device=dev)
    s0 = _rand((3, 24), 1).to(dev)
    h, fin = pkg.gated_linear_recurrence(none, none, _cu([0, 0, 0], dev), initial_state=s0, output_final_state=True)
    assert h.shape == (0, 24) and torch.equal(fin, s0)
    _, fin = pkg.gated_linear_recurrence(none, none, _cu([0, 0, 0], dev), output_final_state=True)
    assert not bool(fin.any())
    d = pkg.gated_linear_recurrence_backward(none, none, none, _cu([0, 0, 0], dev), initial_state=s0, d_final_state=s0 * 2)
    assert torch.equal(d["d_initial_state"], s0 * 2)
    h = pkg.gated_linear_recurrence(none, none, _cu([], dev))
    assert h.shape == (0, 24)
    assert pkg.gated_linear_recurrence_decode(none, none).shape == (0, 24)
    w = torch.ones(8, device=dev)
    y, kept = pkg.gated_group_norm(none.view(0, 3, 8), w, none.view(0, 3, 8), save_checkpoint=True)
    d = pkg.gated_group_norm_backward(y, kept, w)
    assert y.shape == (0, 3, 8) and not bool(d["dweight"].any())


def test_rows_past_the_sequences_stay(cuda_device):
    """Rows at or past cu_seqlens[N] (a captured batch's padding) are not written, and what lies in
    them is not read into any result."""
    dev, C = cuda_device, 80
    lengths = [130, 77]
    x, g = _rand((400, C), 1, BF16).to(dev), _gates("log", (400, C), 2, BF16).to(dev)
    x[207:], g[207:] = math.nan, math.nan
    out = torch.full((400, C), 9.0, dtype=BF16, device=dev)
    h, fin = pkg.gated_linear_recurrence(x, g, _cu(lengths, dev), output=out, output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x.cpu()[:207], g.cpu()[:207], lengths, "log")
    R.check(h[:207], rh, eh, "h")
    R.check(fin, rfin, efin, "final")
    assert bool((h[207:] == 9.0).all())
    dh = _rand((400, C), 3, BF16).to(dev)
    dh[207:] = math.nan
    d = pkg.gated_linear_recurrence_backward(g, h, dh, _cu(lengths, dev), initial_state=torch.zeros((2, C), device=dev))
    dx, dg, dinit, ex, eg, einit = R.recurrence_backward(g.cpu()[:207], h.cpu()[:207], dh.cpu()[:207], lengths, "log")
    R.check(d["dx"][:207], dx, ex, "dx")
    R.check(d["dg"][:207], dg, eg, "dg")
    R.check(d["d_initial_state"], dinit, einit, "d_initial_state")


def test_device_status(cuda_device):
    dev = cuda_device
    x = _rand((10, 16), 1, BF16).to(dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for cu in ([0, 7, 5, 10], [0, 4, 12], [2, 10], [-1, 10]):
        st.zero_()
        pkg.gated_linear_recurrence(x, x, torch.tensor(cu, dtype=torch.int32, device=dev), device_status=st)
        assert int(st) == pkg.GDP_DEV_ERR_CU_SEQLENS, cu
        st.zero_()
        pkg.gated_linear_recurrence_backward(x, x, x, torch.tensor(cu, dtype=torch.int32, device=dev), device_status=st)
        assert int(st) == pkg.GDP_DEV_ERR_CU_SEQLENS, cu
    st.zero_()
    cache = _rand((3, 16), 2).to(dev)
    before = cache.clone()
    slots = torch.tensor([1, 3, -2], dtype=torch.int32, device=dev)
    pkg.gated_linear_recurrence(x, x, _cu([4, 4, 2], dev), state=cache, state_indices=slots, device_status=st)
    assert int(st) == pkg.GDP_DEV_ERR_SLOT
    assert torch.equal(cache[[0, 2]], before[[0, 2]]) and not torch.equal(cache[1], before[1])
    st.zero_()
    pkg.gated_linear_recurrence_decode(x[:3], x[:3], state=cache, state_indices=slots, device_status=st)
    assert int(st) == pkg.GDP_DEV_ERR_SLOT
    st.zero_()
    pkg.gated_linear_recurrence(x, x, _cu([4, 4, 2], dev), device_status=st)
    assert int(st) == 0


def test_recurrence_same_bits_every_time(cuda_device):
    """Whatever the order in which the parts of a long sequence get done."""
    dev = cuda_device
    lengths = [20000, 0, 777, 12000]
    T = sum(lengths)
    x, g = _rand((T, 192), 1, BF16).to(dev), _gates("log", (T, 192), 2, BF16).to(dev)
    cu, s0 = _cu(lengths, dev), _rand((4, 192), 3).to(dev)
    first = None
    for _ in range(20):
        h, fin = pkg.gated_linear_recurrence(x, g, cu, initial_state=s0, output_final_state=True)
        d = pkg.gated_linear_recurrence_backward(g, h, x, cu, initial_state=s0)
        now = (h, fin, d["dx"], d["dg"], d["d_initial_state"])
        if first is None:
            first = [t.clone() for t in now]
        for a, b in zip(first, now):
            assert torch.equal(a, b)


def test_recurrence_long(cuda_device):
    """Long memory over many parts: 70000 tokens, decays near one."""
    dev, T, C = cuda_device, 70000, 24
    x, g = _rand((T, C), 1, BF16), -torch.rand((T, C), generator=_gen(2)) * 2e-3
    h, fin = pkg.gated_linear_recurrence(x.to(dev), g.to(dev), _cu([T], dev), output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, g, [T], "log")
    R.check(h, rh, eh, "h")
    R.check(fin, rfin, efin, "final")


def test_recurrence_past_32_bit_offsets(cuda_device):
    """More than 2^31 elements: decays of zero make h equal x, of one keep the first row."""
    dev, T, C = cuda_device, 530000, 4096
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.empty((T, C), dtype=BF16, device=dev).normal_(generator=torch.Generator(device=dev).manual_seed(1))
    g = torch.zeros((T, C), dtype=BF16, device=dev)
    g[T - 1] = 1.0
    h, fin = pkg.gated_linear_recurrence(x, g, _cu([T], dev), gate="alpha", output_final_state=True)
    assert torch.equal(h[:T - 1], x[:T - 1])
    assert torch.equal(fin[0], x[T - 1].float() + x[T - 2].float())
    d = pkg.gated_linear_recurrence_backward(g, h, x, _cu([T], dev), gate="alpha")
    assert torch.equal(d["dx"][:T - 2], x[:T - 2]) and torch.equal(d["dx"][T - 1], x[T - 1])
    assert torch.equal(d["dg"][T - 1], (x[T - 1].float() * x[T - 2].float()).to(BF16))
    assert torch.equal(d["dg"][1], (x[1].float() * x[0].float()).to(BF16))


@pytest.mark.parametrize("backward", [False, True])
def test_expired_wait_is_reported(cuda_device, backward):
    """A wait that runs out sets the status bit and ends the call; the next call is unaffected."""
    dev, T, C = cuda_device, 5000, 192
    x, g = _rand((T, C), 1, BF16).to(dev), _gates("log", (T, C), 2, BF16).to(dev)
    cu, st = _cu([T], dev), torch.zeros(1, dtype=torch.int32, device=dev)

    def call():
        if backward:
            return pkg.gated_linear_recurrence_backward(g, x, x, cu, device_status=st)["dx"]
        return pkg.gated_linear_recurrence(x, g, cu, device_status=st)

    want = call().clone()
    pkg.gdp_arm_recurrence_wait_test(1_000_000)
    call()
    torch.cuda.synchronize()
    assert int(st) == pkg.GDP_DEV_ERR_TIMEOUT
    st.zero_()
    assert torch.equal(call(), want) and int(st) == 0


def test_on_another_stream_and_in_a_graph(cuda_device):
    dev = cuda_device
    lengths, C = [3000, 2000], 128
    T = sum(lengths)
    x, g, cu = _rand((T, C), 1, BF16).to(dev), _gates("log", (T, C), 2, BF16).to(dev), _cu(lengths, dev)
    w = torch.ones(64, device=dev)

    def step():
        h = pkg.gated_linear_recurrence(x, g, cu)
        y, kept = pkg.gated_group_norm(h.view(T, 2, 64), w, x.view(T, 2, 64), save_checkpoint=True)
        d = pkg.gated_group_norm_backward(y, kept, w)
        r = pkg.gated_linear_recurrence_backward(g, kept.o, d["do"].view(T, C), cu)
        return h, y, d["do"], d["dz"], d["dweight"], r["dx"], r["dg"]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    h = pkg.gated_linear_recurrence(x, g, cu, stream=side.cuda_stream)  # a raw stream handle
    side.synchronize()
    assert torch.equal(h, want[0])


NORMS = [
    # T, H, D, type, gated, act, center, bias, per_head, layout
    (37, 4, 128, BF16, True, "silu", False, False, False, "dense"),
    (37, 4, 128, BF16, True, "silu", False, False, False, "slice"),
    (20, 5, 64, F16, False, "silu", True, True, True, "dense"),
    (20, 3, 64, BF16, True, "sigmoid", True, False, True, "odd"),
    (1, 1, 1, BF16, True, "silu", False, True, False, "dense"),
    (3, 1, 8, F32, False, None, False, False, False, "dense"),
    (50, 7, 17, F16, True, "silu", True, True, False, "odd"),
    (9, 2, 127, BF16, True, "silu", False, False, True, "odd"),
    (9, 2, 129, F32, True, "sigmoid", True, True, False, "odd"),
    (11, 3, 200, BF16, True, "silu", False, False, False, "dense"),
    (11, 3, 256, F32, False, None, True, True, True, "slice"),
    (300, 2, 96, BF16, True, "silu", False, False, False, "dense"),
    (7, 1, 1000, F16, True, "silu", True, True, True, "odd"),
    (7, 1, 1024, BF16, True, "silu", False, False, False, "dense"),
    (7, 2, 1032, BF16, True, "silu", True, True, True, "slice"),
    (5, 1, 2500, BF16, False, "silu", True, True, False, "odd"),
    (5, 1, 4096, BF16, True, "sigmoid", True, True, True, "dense"),
    (3, 1, 8191, F16, True, "silu", False, False, False, "dense"),
    (3, 1, 8192, F32, True, "silu", False, True, False, "dense"),
    (700, 32, 32, BF16, True, "silu", False, False, False, "dense"),
    (701, 31, 40, BF16, True, "silu", False, True, True, "dense"),
    (5000, 1, 16, F16, False, None, True, True, False, "dense"),
]


def _norm_inputs(case):
    T, H, D, dt, gated, act, center, bias, per_head, layout = case
    o = _rand((T, H, D), 1, sigma=2.0)
    if center:
        o += 3.0
    o[0, 0] *= 1e-3
    shape = (H, D) if per_head else (D,)
    return (o.to(dt), _rand((T, H, D), 2, dt, 2.0) if gated else None, 1 + _rand(shape, 3, sigma=0.3),
            _rand(shape, 4, sigma=0.3) if bias else None, _rand((T, H, D), 5, dt))


@pytest.mark.parametrize("case", NORMS)
def test_group_norm(cuda_device, case):
    T, H, D, dt, gated, act, center, bias, per_head, layout = case
    o, z, w, b, _ = _norm_inputs(case)
    dev = cuda_device
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    od, zd = _as_laid_out(o, layout, dev), None if z is None else _as_laid_out(z, layout, dev)
    how = dict(eps=1e-5, center=center, activation=act)
    y, kept = pkg.gated_group_norm(od, on(w), zd, on(b), save_checkpoint=True, **how)
    R.check(y, *R.group_norm(o, w, z, b, 1e-5, center, act), "y")
    assert torch.equal(pkg.gated_group_norm(od, on(w), zd, on(b), **how), y)
    for name, c, v in (("o", kept.o, o), ("z", kept.z, z)):
        assert (c is None) == (v is None)
        if c is not None:
            codes, scales, values = R.quantize(v)
            if dt != F32:  # an fp32 value times the inverse scale is rounded: a code next to a tie may move
                assert torch.equal(c.codes.cpu(), codes), name
            assert int((c.codes.cpu().int() - codes.int()).abs().max()) <= (0 if dt != F32 else 1), name
            assert torch.equal(c.scales.cpu(), scales.float()), name


def test_checkpoint_codes_of_fp32_values(cuda_device):
    """fp32 values: the codes of plain fp32 arithmetic, product rounded first, bit for bit (a value next to a
    tie may differ from the 64-bit code)."""
    for shape in ((3000, 8, 128), (400, 1, 4096), (500, 3, 100)):
        v = _rand(shape, 1).to(cuda_device)
        kept = pkg.gated_group_norm(v, torch.ones(shape[-1], device=cuda_device), activation=None, save_checkpoint=True)[1]
        pad = -shape[-1] % 128
        amax = torch.nn.functional.pad(v, (0, pad)).view(*shape[:2], -1, 128).abs().amax(-1)
        inv = ((127.0 / amax).view(torch.int32) & -0x100000).view(torch.float32)
        codes = torch.round(v * inv.repeat_interleave(128, -1)[..., :shape[-1]])
        assert torch.equal(kept.o.codes, codes.to(torch.int8)) and torch.equal(kept.o.scales, 1.0 / inv)


@pytest.mark.parametrize("saved", ["checkpoint", "tensors"])
@pytest.mark.parametrize("case", NORMS)
def test_group_norm_backward(cuda_device, case, saved):
    T, H, D, dt, gated, act, center, bias, per_head, layout = case
    o, z, w, b, dy = _norm_inputs(case)
    dev = cuda_device
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    how = dict(eps=1e-5, center=center, activation=act)
    if saved == "checkpoint":
        co, cz = R.quantize(o), R.quantize(z) if z is not None else None
        pack = lambda q: pkg.ActivationCheckpoint(q[0].to(dev), q[1].float().to(dev))  # noqa: E731
        kept = pkg.GroupNormCheckpoint(pack(co), pack(cz) if cz is not None else None)
        o, z = co[0].double() * co[1].float().double().repeat_interleave(128, -1)[..., :D], z
        if cz is not None:
            z = cz[0].double() * cz[1].float().double().repeat_interleave(128, -1)[..., :D]
    else:
        kept = (_as_laid_out(o, layout, dev), _as_laid_out(z, layout, dev) if z is not None else None)
    got = pkg.gated_group_norm_backward(_as_laid_out(dy, layout, dev), kept, on(w), on(b), **how)
    ref = R.group_norm_backward(dy, o, w, z, b, 1e-5, center, act)
    for name in ("do", "dz", "dweight", "dbias"):
        if got[name] is None:
            assert (name == "dz" and z is None) or (name == "dbias" and b is None)
            continue
        R.check(got[name], *ref[name], name)


def test_group_norm_special_rows(cuda_device):
    """A row of zeros, infinities and NaN stay in their own rows; their checkpoint blocks too."""
    dev, D = cuda_device, 256
    o = _rand((6, 1, D), 1, BF16)
    z = _rand((6, 1, D), 2, BF16)
    w = torch.ones(D, device=dev)
    y0, k0 = pkg.gated_group_norm(o.to(dev), w, z.to(dev), save_checkpoint=True)
    o[1] = 0
    o[2, 0, 3], o[3, 0, 200], z[4, 0, 5] = math.inf, math.nan, math.nan
    y, k = pkg.gated_group_norm(o.to(dev), w, z.to(dev), save_checkpoint=True)
    for a, b in ((y0, y), (k0.o.codes, k.o.codes), (k0.z.scales, k.z.scales)):
        assert torch.equal(a[[0, 5]], b[[0, 5]])
    assert not bool(y[1].any()) and not bool(k.o.codes[1].any()) and float(k.o.scales[1].abs().sum()) == 0.0
    assert bool(torch.isnan(k.o.scales[2, 0, 0])) and bool(torch.isfinite(k.o.scales[2, 0, 1]))
    assert bool(torch.isnan(k.o.scales[3, 0, 1])) and bool(torch.isfinite(k.o.scales[3, 0, 0]))
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4, 0, 5])) and bool(torch.isfinite(y[4, 0, 6]))
    dy = _rand((6, 1, D), 3, BF16).to(dev)
    d = pkg.gated_group_norm_backward(dy, k, w)
    assert bool(torch.isfinite(d["do"][[0, 1, 5]].float()).all()) and bool(torch.isnan(d["do"][3]).all())
    assert bool(torch.isnan(d["dz"][4, 0, :128]).all())
    big = torch.full((1, 1, D), 3e38, dtype=BF16)
    kept = pkg.gated_group_norm(big.to(dev), w, activation=None, save_checkpoint=True)[1]
    assert torch.equal(kept.o.codes.cpu(), R.quantize(big)[0])


def test_group_norm_same_bits_every_time(cuda_device):
    dev = cuda_device
    o, z, dy = (_rand((3000, 8, 128), i, BF16).to(dev) for i in (1, 2, 3))
    for w in (torch.ones(128, device=dev), torch.ones((8, 128), device=dev)):
        kept = pkg.gated_group_norm(o, w, z, save_checkpoint=True)[1]
        first = pkg.gated_group_norm_backward(dy, kept, w)
        for _ in range(10):
            again = pkg.gated_group_norm_backward(dy, kept, w)
            assert all(torch.equal(first[n], again[n]) for n in ("do", "dz", "dweight"))


def test_group_norm_behind_the_delta_product(cuda_device):
    """The norm as the output stage of the Gated DeltaProduct: its o is normed and gated, and the norm's
    gradient is the delta product's upstream gradient."""
    from gdp_workloads import make_custom
    dev = cuda_device
    w = make_custom([100, 37], 2, 128, 2, seed=5, init_sigma=0.1)
    q, k, v, g, b, cu = (t.to(dev) for t in (w.q, w.k, w.v, w.g, w.beta, w.cu_seqlens))
    o = pkg.chunk_gated_delta_product(q, k, v, g, b, cu, 2, w.scale)
    z, weight = _rand(tuple(o.shape), 1, BF16).to(dev), torch.ones(128, device=dev)
    y, kept = pkg.gated_group_norm(o, weight, z, save_checkpoint=True)
    R.check(y, *R.group_norm(o.cpu(), weight.cpu(), z.cpu()), "y")
    d = pkg.gated_group_norm_backward(y, kept, weight)
    grads = pkg.chunk_gated_delta_product_backward(q, k, v, g, b, cu, 2, d["do"], w.scale)
    assert bool(torch.isfinite(grads["dq"]).all()) and bool(grads["dk"].any())


def test_wrapper_refusals(cuda_device):
    dev = cuda_device
    x = torch.zeros((8, 16), dtype=BF16, device=dev)
    cu = _cu([8], dev)
    f32 = torch.zeros((1, 16), device=dev)
    for call, words in (
            (lambda: pkg.gated_linear_recurrence(x, x[:4], cu), "g must have shape"),
            (lambda: pkg.gated_linear_recurrence(x, x.half(), cu), "g must be float32 or of x's type"),
            (lambda: pkg.gated_linear_recurrence(x.long(), x, cu), "x must be"),
            (lambda: pkg.gated_linear_recurrence(x, x, None), "cu_seqlens"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu.cpu()), "cu_seqlens"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu.float()), "cu_seqlens"),
            (lambda: pkg.gated_linear_recurrence(x.t().contiguous().t(), x, cu), "contiguous in its last"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, gate="tanh"), "gate must be"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, initial_state=f32[:, :8]), "initial_state"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, initial_state=f32.bfloat16()), "initial_state"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, state=f32), "state_indices"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, state=f32, initial_state=f32, state_indices=cu[:1]), "excludes"),
            (lambda: pkg.gated_linear_recurrence(x, x, cu, output=x.float()), "output"),
            (lambda: pkg.gated_linear_recurrence(x.expand(8, 16)[:1].expand(8, 16), x, cu), "rows at least C"),
            (lambda: pkg.gated_linear_recurrence_decode(x, x, state=f32, state_indices=cu), "state_indices"),
            (lambda: pkg.gated_linear_recurrence_backward(x, x, x, cu, gate="sigmoid"), "needs x"),
            (lambda: pkg.gated_linear_recurrence_backward(x, x[:4], x, cu), "h must have shape"),
            (lambda: pkg.gated_linear_recurrence_backward(
                x, pkg.ActivationCheckpoint(x.view(8, 1, 16).to(torch.int8), f32), x, cu), "scales"),
            (lambda: pkg.gated_group_norm(x, f32[0]), r"\[T, H, D\]"),
            (lambda: pkg.gated_group_norm(x.view(8, 2, 8), f32[0]), "weight must be"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0].bfloat16()), "weight"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0], x.view(8, 2, 8)), "z must have shape"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0], x.view(8, 1, 16), activation=None), "z needs"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0], activation="sigmoid"), "gates with z"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0], activation="gelu"), "activation"),
            (lambda: pkg.gated_group_norm(x.view(8, 1, 16), f32[0], bias=f32), "bias"),
            (lambda: pkg.gated_group_norm_backward(x.view(8, 1, 16), (x.view(8, 2, 8), None), f32[0]), "o must have shape"),
    ):
        with pytest.raises(pkg.GdpError, match=words):
            call()
