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


# ---- nothing but padding, and long caches -------------------------------------------------------------

@pytest.mark.parametrize("N,T,C", [(1, 1000, 40), (3, 1000, 40), (2, 30, 2200)])
def test_nothing_but_padding(cuda_device, N, T, C):
    """Empty sequences before rows that belong to none, in pieces and not: zeros, states as they came, sums of nothing."""
    dev = cuda_device
    assert (pkg.gdp_scan_forward_workspace_bytes(T, N, C, 16) > 0) == (C == 40)
    b, cu = Block(T, C, 16, N, dev), _cu([0] * N, dev)
    for t in (b.x, b.z, b.dy, b.dt, b.B, b.Cm):
        t.fill_(math.nan)
    y, fin = b.conv(cu, initial_state=b.c0, output_final_state=True)
    assert not y.any() and torch.equal(fin, b.c0)
    y, fin, kept = b.scan(cu, initial_state=b.h0, output_final_state=True, save_states=True)
    assert not y.any() and torch.equal(fin, b.h0)
    d = b.conv_backward(cu, initial_state=b.c0, d_final_state=b.c0)
    assert torch.equal(d.pop("d_initial_state"), b.c0) and not any(v.any() for v in d.values())
    d = b.scan_backward(cu, kept, d_final_state=b.h0, output_d_initial_state=True)
    assert torch.equal(d.pop("d_initial_state"), b.h0) and not any(v.any() for v in d.values())


def test_caches_beyond_32_bits(cuda_device):
    """State caches of more than 2^31 elements, their last slots among those in use."""
    dev, C, S = cuda_device, 4096, 16
    for each, lengths in (((C, S), [40, 0, 9]), ((3, C), [5, 2, 70])):
        elems = each[0] * each[1]
        many = (1 << 31) // elems + 5
        b, cu = Block(sum(lengths), C, S, 3, dev), _cu(lengths, dev)
        cache = torch.empty((many, *each), dtype=F32 if each == (C, S) else BF16, device=dev)
        slots = torch.tensor([many - 1, 1, many - 3], dtype=torch.int32, device=dev)
        init = b.h0 if each == (C, S) else b.c0
        call = b.scan if each == (C, S) else b.conv
        cache[many - 2] = 7.0
        cache[slots.long()] = init
        want, fin = call(cu, initial_state=init, output_final_state=True)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        assert torch.equal(call(cu, state=cache, state_indices=slots, device_status=status), want)
        assert torch.equal(cache[slots.long()], fin)
        if each == (C, S):
            step = lambda **k: pkg.selective_scan_decode(b.x[:3], b.dt[:3], b.A, b.B[:3], b.Cm[:3], **k)  # noqa: E731
        else:
            step = lambda **k: pkg.short_convolution_decode(b.x[:3], b.w, b.b, **k)  # noqa: E731
        want, fin = step(initial_state=fin, output_final_state=True)
        assert torch.equal(step(state=cache, state_indices=slots, device_status=status), want)
        assert torch.equal(cache[slots.long()], fin) and bool((cache[many - 2] == 7.0).all()) and int(status) == 0
        del cache


# ---- one token, two sequences a CTA ------------------------------------------------------------------
# sequences, channels, states, groups, x's type, dt's type, layout: 16 CTAs per SM and more, odd numbers of sequences
STEPS = [(21, 4096, 16, 1, BF16, BF16, "dense"), (39, 2048, 16, 1, F32, F32, "slice"), (23, 2048, 64, 2, F16, F32, "dense"),
         (41, 2048, 18, 1, BF16, F32, "odd"), (153, 1000, 5, 2, F16, F16, "odd"), (512, 200, 16, 1, BF16, BF16, "dense"),
         (2433, 24, 8, 1, BF16, BF16, "dense")]


@pytest.mark.parametrize("N,C,S,G,xt,dtt,layout", STEPS)
def test_steps_of_many_sequences(cuda_device, N, C, S, G, xt, dtt, layout):
    dev = cuda_device
    assert N * _tiles(C, S, G) >= 16 * _sms(dev)
    x, z, dt = _rand((N, C), 1, xt), _rand((N, C), 2, xt), _rand((N, C), 3, dtt, 0.5)
    A, B, Cm = -torch.exp(_rand((C, S), 4)), _rand((N, G, S), 5, xt), _rand((N, G, S), 6, xt)
    D, bias, init = _rand((C,), 7), _rand((C,), 8) - 2.0, _rand((N, C, S), 9)
    lay = lambda t: _as_laid_out(t, layout, dev)  # noqa: E731
    ins = (lay(x), lay(dt), A.to(dev), lay(B), lay(Cm))
    how = {"D": D.to(dev), "z": lay(z), "dt_bias": bias.to(dev)}
    want = R.scan(x, dt, A, B, Cm, [1] * N, D=D, z=z, dt_bias=bias, init=init)
    y, fin = pkg.selective_scan_decode(*ins, initial_state=init.to(dev), output_final_state=True, **how)
    check(y, *want["y"], "y")
    check(fin, *want["final"], "final state")
    # the cache: slots in another order, one that nobody has, entries of padding, one outside
    order = torch.randperm(N + 1, generator=torch.Generator().manual_seed(10))[:N].to(torch.int32)
    off = list(range(3, N, 7)) + [N - 1]
    cache = torch.empty((N + 1, C, S)).fill_(3.0)
    cache[order.long()] = init
    order[off] = -1
    order[off[0]] = N + 1
    state, status = cache.to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    got = pkg.selective_scan_decode(*ins, state=state, state_indices=order.to(dev), device_status=status, **how)
    assert int(status) == pkg.GDP_DEV_ERR_SLOT
    live = [i for i in range(N) if i not in off]
    assert torch.equal(got[live], y[live]) and torch.equal(state[order[live].long()], fin[live])
    rest = sorted(set(range(N + 1)) - set(order[live].tolist()))
    assert torch.equal(state[rest].cpu(), cache[rest])
    zero = R.scan(*(t[off] if t.shape[0] == N else t for t in (x, dt, A, B, Cm)), [1] * len(off), D=D, z=z[off], dt_bias=bias)
    check(got[off], *zero["y"], "padding entries")


# ---- several sequences per CTA, and the longest first ------------------------------------------------

def _mixed(n, most, seed):
    """n lengths, short ones in the main, some of them zero, one of `most`."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, max(2, most // 8), (n,), generator=g).tolist()
    lengths[n // 3], lengths[n // 2], lengths[-1] = most, 0, 0
    return lengths


# lengths, channels, states, groups, x's type, dt's type, gated, workers' loops, ranked
MANY = [
    (_mixed(90, 30, 1), 2080, 16, 1, BF16, BF16, True, True, False), (_mixed(90, 41, 2), 130, 33, 65, F16, F32, False, True, False),
    (_mixed(40, 600, 3), 130, 5, 130, F32, F32, True, True, True), (_mixed(12, 200, 4), 832, 16, 1, BF16, F32, True, False, True),
    (_mixed(200, 60, 5), 96, 64, 8, F32, F32, True, True, False), ([700, 3] * 20, 130, 20, 130, BF16, BF16, True, True, True),
]


@pytest.mark.parametrize("lengths,C,S,G,xt,dtt,gated,loops,ranked", MANY)
def test_many_sequences(cuda_device, lengths, C, S, G, xt, dtt, gated, loops, ranked):
    """More sequences than the backward pass has CTAs for, so that each takes several in turn, and sequences that are run by
    length, against the reference, with rows behind the last one."""
    dev, N, T, sms = cuda_device, len(lengths), sum(lengths), _sms(cuda_device)
    tiles, rows = _tiles(C, S, G), sum(lengths) + 5
    assert loops == (N > -(-16 * sms // tiles)) and ranked == (rows >= N * N and N * tiles > 2 * sms)
    assert pkg.gdp_scan_forward_workspace_bytes(rows, N, C, S, G) == 0
    start = torch.exp(_rand((C,), 20) - 3.0)
    x, z, dy, dt = _rand((T, C), 1, xt), _rand((T, C), 2, xt), _rand((T, C), 3, xt), _rand((T, C), 4, dtt, 0.5)
    A, B, Cm = -torch.exp(_rand((C, S), 5)) * 2.0, _rand((T, G, S), 6, xt), _rand((T, G, S), 7, xt)
    D, bias, h0, dfin = _rand((C,), 8), torch.log(torch.expm1(start)), _rand((N, C, S), 9), _rand((N, C, S), 10)
    z = z if gated else None

    def padded(t):
        return None if t is None else torch.cat([t, torch.full((5, *t.shape[1:]), math.nan, dtype=t.dtype)]).to(dev)

    ins, how = (padded(x), padded(dt), A.to(dev), padded(B), padded(Cm)), {"D": D.to(dev), "z": padded(z), "dt_bias": bias.to(dev)}
    cu = _cu(lengths, dev)
    y, fin, kept = pkg.selective_scan(*ins, cu, initial_state=h0.to(dev), output_final_state=True, save_states=True, **how)
    want = R.scan(x, dt, A, B, Cm, lengths, D=D, z=z, dt_bias=bias, init=h0)
    check(y[:T], *want["y"], "y")
    check(fin, *want["final"], "final state")
    got = pkg.selective_scan_backward(*ins, padded(dy), cu, kept, d_final_state=dfin.to(dev), output_d_initial_state=True, **how)
    for name in ("dx", "ddt", "dB", "dC") + (("dz",) if gated else ()):
        assert not got[name][T:].any(), name
        got[name] = got[name][:T]
    assert not y[T:].any()
    _close(got, R.scan_backward(x, dt, A, B, Cm, dy, lengths, D=D, z=z, dt_bias=bias, init=h0, dfin=dfin))


# ---- the convolution's long runs ---------------------------------------------------------------------

@pytest.mark.parametrize("C,W,dtype,bias", [(1024, 4, BF16, True), (127, 3, F16, False), (512, 2, F32, True), (254, 4, BF16, False)])
def test_convolution_of_many_rows(cuda_device, C, W, dtype, bias):
    """Rows enough for 64 a thread, bounds on and off the runs' borders; some channels against the reference (channels do not
    mix), rows behind the last sequence."""
    dev = cuda_device
    lengths = [1, 63, 64, 65, 0, 2, 127, 128, 129, 3, 0, 4093, 1, 1, 1, 30000, 61, 60003]
    T, N = sum(lengths), len(lengths)
    vecs = C // 8 if C % 8 == 0 and dtype != F32 else C // 4 if C % 4 == 0 and dtype == F32 else C // 2 if C % 2 == 0 else C
    assert vecs in (127, 128) and T >= 64 * 8 * _sms(dev)  # (128 vectors of channels a CTA, one run of rows)
    g = torch.Generator(dev).manual_seed(1)
    x, dy = (torch.randn((T + 70, C), generator=g, device=dev).to(dtype) for _ in range(2))
    x[T:], dy[T:] = math.nan, math.nan
    w, b = _rand((C, W), 2, sigma=0.5), _rand((C,), 3) if bias else None
    s0, dfin = _rand((N, W - 1, C), 4, dtype), _rand((N, W - 1, C), 5, dtype)
    gw, gb, gs0, gdfin = _on(dev, w, b, s0, dfin)
    cu = _cu(lengths, dev)
    y, fin = pkg.short_convolution(x, gw, cu, gb, initial_state=gs0, output_final_state=True)
    got = pkg.short_convolution_backward(x, gw, dy, cu, gb, initial_state=gs0, d_final_state=gdfin)
    at = torch.tensor([0, 1, 7, C // 2, C - 2, C - 1])
    part = lambda t: t[..., at.to(t.device)].cpu()  # noqa: E731
    args = (part(x[:T]), w[at]), dict(b=None if b is None else b[at], init=s0[..., at])
    want, err, wfin = R.convolution(*args[0], lengths, act="silu", **args[1])
    check(part(y[:T]), want, err, "y")
    assert torch.equal(part(fin).double(), wfin) and not y[T:].any() and bool(torch.isfinite(y).all())
    back = R.convolution_backward(*args[0], part(dy[:T]), lengths, act="silu", dfin=dfin[..., at], **args[1])
    check(part(got["dx"][:T]), *back["dx"], "dx")
    assert not got["dx"][T:].any() and all(bool(torch.isfinite(v).all()) for v in got.values() if v is not None)
    check(got["dweight"][at.to(dev)], *back["dweight"], "dweight")
    if bias:
        check(part(got["dbias"]), *back["dbias"], "dbias")
    check(part(got["d_initial_state"]), *back["d_initial_state"], "d_initial_state")


# ---- pieces ------------------------------------------------------------------------------------------

PIECES = [([1200], 40), ([129, 127, 128, 640], 40)]


def _in_pieces(lengths, C, S=16):
    """Both passes run these sequences in pieces: they need what joins them beside the sums that whole sequences need."""
    T, N = sum(lengths), len(lengths)
    lanes = {16: 4}[S]
    sums = -(-N * 4 * (-(-C * (S + 2) // 4) * 4) // 256) * 256
    whole = sums + _tiles(C, S, 1) * T * 8 * 4 * lanes
    return pkg.gdp_scan_forward_workspace_bytes(T, N, C, S) > 0 and pkg.gdp_scan_workspace_bytes(T, N, C, S) > whole + N * C * S * 4


@pytest.mark.parametrize("lengths,C", PIECES)
def test_pieces_captured_and_replayed(cuda_device, lengths, C):
    """Two graphs of all calls, pieces among them, replayed in turn with other inputs in the same buffers."""
    dev = cuda_device
    assert _in_pieces(lengths, C)
    cu, b, other = _cu(lengths, dev), *(Block(sum(lengths), C, 16, len(lengths), dev, seed=s) for s in (0, 100))
    want_other, want = other.everything(cu), b.everything(cu)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.everything(cu))
        graphs.append(g)
    for g in graphs:
        g.replay()
    for o in outs:
        _same(o, want)
    for k, v in vars(other).items():
        getattr(b, k).copy_(v)
    for g in (*graphs, graphs[0]):
        g.replay()
    for o in outs:
        _same(o, want_other)


@pytest.mark.parametrize("lengths,C", PIECES)
def test_pieces_on_a_given_stream(cuda_device, lengths, C):
    dev = cuda_device
    assert _in_pieces(lengths, C)
    b, cu = Block(sum(lengths), C, 16, len(lengths), dev), _cu(lengths, dev)
    y, fin, kept = b.scan(cu, initial_state=b.h0, output_final_state=True, save_states=True)
    want = {"y": y, "fin": fin, **b.scan_backward(cu, kept, d_final_state=b.h0, output_d_initial_state=True)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the side stream is busy for a while
    h = side.cuda_stream
    y, fin, kept = b.scan(cu, initial_state=b.h0, output_final_state=True, save_states=True, stream=h)
    got = {"y": y, "fin": fin, **b.scan_backward(cu, kept, d_final_state=b.h0, output_d_initial_state=True, stream=h)}
    assert not side.query()
    side.synchronize()
    _same(got, want)


@pytest.mark.parametrize("lengths,C", PIECES)
def test_pieces_in_given_workspaces(cuda_device, lengths, C):
    """Workspaces of the stated size, with anything in them; a byte less, or off 256 bytes, is refused."""
    dev, T, N = cuda_device, sum(lengths), len(lengths)
    assert _in_pieces(lengths, C)
    b, cu = Block(T, C, 16, N, dev), _cu(lengths, dev)
    kept = b.scan(cu, initial_state=b.h0, save_states=True)[1]

    def forward(**k):
        y, fin, states = b.scan(cu, initial_state=b.h0, output_final_state=True, save_states=True, **k)
        rows = torch.cat([torch.arange(-(-n // 16)) + sum(lengths[:i]) // 16 + i for i, n in enumerate(lengths)])
        return {"y": y, "fin": fin, "states": states[rows.to(dev)]}

    def backward(**k):
        return b.scan_backward(cu, kept, d_final_state=b.h0, output_d_initial_state=True, **k)

    for need, call in ((pkg.gdp_scan_forward_workspace_bytes(T, N, C, 16), forward), (pkg.gdp_scan_workspace_bytes(T, N, C, 16), backward)):
        assert need > 0
        want = call()
        for stale in (255, 127, 0):  # NaN, large and zero values
            room = torch.full((need + 512,), stale, dtype=torch.uint8, device=dev)
            _same(call(workspace=room[:need]), want)
            assert bool((room[need:] == stale).all())
        with pytest.raises(pkg.GdpError):
            call(workspace=room[:need - 1])
        with pytest.raises(pkg.GdpError):
            call(workspace=room[16:16 + need])


def test_pieces_on_two_streams_at_once(cuda_device):
    """Both streams run pieces, each in workspaces of its own, beside one another."""
    dev = cuda_device
    assert all(_in_pieces(*p) for p in PIECES)
    blocks = [Block(sum(n), c, 16, len(n), dev, seed=i) for i, (n, c) in enumerate(PIECES)]
    cus = [_cu(n, dev) for n, _ in PIECES]
    alone = [b.everything(cu) for b, cu in zip(blocks, cus)]
    streams = [torch.cuda.Stream(dev) for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(6):
        got = []
        for b, cu, s in zip(blocks, cus, streams):
            with torch.cuda.stream(s):
                got.append(b.everything(cu))
        torch.cuda.synchronize()
        for mine, want in zip(got, alone):
            _same(mine, want)


def test_pieces_from_two_threads(cuda_device):
    """The scan in pieces and a wide one that is not, forward and backward, from two host threads at once."""
    dev = cuda_device
    blocks = [(Block(1200, 40, 16, 1, dev), _cu([1200], dev)), (Block(230, 2200, 16, 3, dev), _cu([30, 0, 200], dev))]
    got = [None, None]

    def one(i):
        b, cu = blocks[i]
        y, kept = b.scan(cu, save_states=True)
        return {"y": y, **b.scan_backward(cu, kept)}

    def call(i):
        def work():
            got[i] = one(i)
        return work

    want = [one(0), one(1)]
    _from_two_threads([call(0), call(1)], 200)
    for g, w in zip(got, want):
        _same(g, w)


# ---- sums over many rows -----------------------------------------------------------------------------

@pytest.mark.parametrize("C", [1025, 4095, 4096])
def test_convolution_sums_of_many_rows(cuda_device, C):
    """The weights' gradients are sums of exact products over all rows (no activation).  A running sum of n random terms is off by
    2^-24 sqrt(n / 6) of its size (a rounding's root mean square is 2^-24 / sqrt(3) of what the sum is by then); here 64 rows' are
    summed, these sums over a part, and P parts' by 32 warps and then over the warps.  (One running sum over a part: 2.7e-7 and
    5.6e-7 at the odd widths.)"""
    dev, T = cuda_device, 65536
    g = torch.Generator(dev).manual_seed(1)
    x, dy = (torch.randn((T, C), generator=g, device=dev).bfloat16() for _ in range(2))
    w, b, cu = _rand((C, 4), 2).to(dev), _rand((C,), 3).to(dev), _cu([T], dev)
    got = pkg.short_convolution_backward(x, w, dy, cu, b, None)
    xd, dyd = x.double(), dy.double()
    want = torch.stack([(dyd[3 - j:] * xd[:T - 3 + j]).sum(0) for j in range(4)], 1)
    parts = 4 * _sms(dev) // -(-(C // 4 if C % 4 == 0 else C) // 128)  # CTAs of 128 vectors of channels, four per SM
    bound = R.U * math.sqrt((64 + T / parts / 64 + parts / 32 + 32) / 6)
    for name, ref in (("dweight", want), ("dbias", dyd.sum(0))):
        error = float((got[name].double() - ref).norm() / ref.norm())
        assert error <= bound, (name, error, bound)


@pytest.mark.parametrize("lengths", [[65536], [2000] * 32])
def test_scan_sums_of_many_rows(cuda_device, lengths):
    """dD is the sum of products over all rows.  A thread takes every eighth row: 32 products, these sums over its sequences, then
    eight threads' and the workers' (bound as above; one running sum over the thread's rows: 1.6e-6 and 4.7e-7)."""
    dev, T, C, S = cuda_device, 65536, 160, 4  # (a group per channel: CTAs enough for whole sequences)
    N = len(lengths)
    assert pkg.gdp_scan_forward_workspace_bytes(sum(lengths), N, C, S, C) == 0
    T = sum(lengths)
    g = torch.Generator(dev).manual_seed(1)
    x, dy, dt, B, Cm = (torch.randn(s, generator=g, device=dev) for s in ((T, C), (T, C), (T, C), (T, C, S), (T, C, S)))
    A, D, cu = -torch.ones((C, S), device=dev), torch.ones(C, device=dev), _cu(lengths, dev)
    kept = pkg.selective_scan(x, dt, A, B, Cm, cu, D=D, save_states=True)[1]
    got = pkg.selective_scan_backward(x, dt, A, B, Cm, dy, cu, kept, D=D)["dD"]
    want = (x.double() * dy.double()).sum(0)
    each = -(-N // -(-16 * _sms(dev) // C))  # sequences of a worker
    bound = R.U * math.sqrt((32 + each * max(lengths) / 256 + each + 8 + N) / 6)
    error = float((got.double() - want).norm() / want.norm())
    assert error <= bound, (error, bound)
