"""The block operators at the edges of calls and types: padding rows, wild bounds and slots, given buffers, other streams,
captured graphs, repeats to the bit, more than 2^31 elements, infinities and NaN, empty batches, a whole block."""
import math

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from tests import _block_ref as R
from tests._layer_ref import check
from tests.test_gpu_block import _cu, _rand

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Block:
    """Inputs of the three operators over packed rows, and calls of them by name."""

    def __init__(self, T, C, S, N, dev, dtype=BF16, seed=0, G=1):
        r = lambda shape, i, t=F32, sigma=1.0: _rand(shape, seed + i, t, sigma).to(dev)  # noqa: E731
        self.x, self.z, self.dy, self.gate = (r((T, C), i, dtype) for i in range(4))
        self.dt, self.B, self.Cm = r((T, C), 5, dtype, 0.5), r((T, G, S), 6, dtype), r((T, G, S), 7, dtype)
        self.A, self.D, self.bias = -torch.exp(r((C, S), 8)), r((C,), 9), r((C,), 10) - 2.0
        self.w, self.b = r((C, 4), 11), r((C,), 12)
        self.h0, self.c0 = r((N, C, S), 13), r((N, 3, C), 14, dtype)
        self.res, self.dr = r((T, C), 15), r((T, C), 16)
        self.weight, self.post, self.scale = (1 + 0.1 * r((C,), i) for i in (17, 18, 19))

    def scan_in(self):
        return (self.x, self.dt, self.A, self.B, self.Cm), {"D": self.D, "z": self.z, "dt_bias": self.bias}

    def conv(self, cu, **kw):
        return pkg.short_convolution(self.x, self.w, cu, self.b, **kw)

    def conv_backward(self, cu, **kw):
        return pkg.short_convolution_backward(self.x, self.w, self.dy, cu, self.b, **kw)

    def scan(self, cu, **kw):
        ins, how = self.scan_in()
        return pkg.selective_scan(*ins, cu, **how, **kw)

    def scan_backward(self, cu, kept, **kw):
        ins, how = self.scan_in()
        return pkg.selective_scan_backward(*ins, self.dy, cu, kept, **how, **kw)

    def norm(self, **kw):
        return pkg.residual_norm(self.res, self.x, self.weight, self.post, self.gate, "silu", self.scale, **kw)

    def norm_backward(self, r, **kw):
        return pkg.residual_norm_backward(self.dy, self.dr, r, self.x, self.weight, self.post, self.gate, "silu", self.scale, **kw)

    def everything(self, cu):
        """All outputs of all calls, by name."""
        out = {}
        out["conv"], out["conv state"] = self.conv(cu, initial_state=self.c0, output_final_state=True)
        out["scan"], out["scan state"], kept = self.scan(cu, initial_state=self.h0, output_final_state=True, save_states=True)
        out["y"], out["r"] = self.norm()
        n = cu.numel() - 1
        for name, d in (("conv", self.conv_backward(cu, initial_state=self.c0, d_final_state=self.c0)),
                        ("scan", self.scan_backward(cu, kept, d_final_state=self.h0, output_d_initial_state=True)),
                        ("norm", self.norm_backward(out["r"]))):
            out.update({f"{name} {k}": v for k, v in d.items()})
        out["conv step"], out["conv step state"] = pkg.short_convolution_decode(self.x[:n], self.w, self.b, initial_state=self.c0,
                                                                                output_final_state=True)
        (x, dt, A, B, Cm), how = self.scan_in()
        how["z"] = how["z"][:n]
        out["scan step"], out["scan step state"] = pkg.selective_scan_decode(x[:n], dt[:n], A, B[:n], Cm[:n], initial_state=self.h0,
                                                                             output_final_state=True, **how)
        return out


LENGTHS = [40, 0, 300, 1, 77]


@pytest.mark.parametrize("lengths,C", [([40, 0, 9, 1, 77], 70), (LENGTHS, 48), ([700], 33)])
def test_padding_rows(cuda_device, lengths, C):
    """Rows behind the last sequence: zeros in what a call allocates, untouched in what it is given, and nothing of them in
    any sum."""
    real, T = sum(lengths), sum(lengths) + 21
    b, cu = Block(T, C, 16, len(lengths), cuda_device), _cu(lengths, cuda_device)
    for t in (b.x, b.z, b.dy, b.dt, b.B, b.Cm):
        t[real:] = math.nan
    y, (s, kept) = b.conv(cu), b.scan(cu, save_states=True)
    assert not y[real:].any() and not s[real:].any()
    for call in (b.conv, b.scan):
        given = torch.full_like(b.x, 7.0)
        out = call(cu, output=given)
        assert out is given and bool((given[real:] == 7.0).all()) and torch.isfinite(given).all()
    for d, rows in ((b.conv_backward(cu), ("dx",)), (b.scan_backward(cu, kept), ("dx", "ddt", "dz", "dB", "dC"))):
        for name, v in d.items():
            if v is not None:
                assert torch.isfinite(v).all(), name
                if name in rows:
                    assert not v[real:].any(), name


def test_no_sequences(cuda_device):
    """N = 0: every row is padding; T = 0: empty sequences pass their states on."""
    b, none = Block(20, 24, 16, 0, cuda_device), _cu([], cuda_device)
    assert not b.conv(none).any()
    y, kept = b.scan(none, save_states=True)
    assert not y.any()
    for d in (b.conv_backward(none), b.scan_backward(none, kept, output_d_initial_state=True)):
        for name, v in d.items():
            assert v is None or not v.any(), name
    e, cu = Block(0, 24, 16, 3, cuda_device), _cu([0, 0, 0], cuda_device)
    y, fin = e.conv(cu, initial_state=e.c0, output_final_state=True)
    assert y.shape == (0, 24) and torch.equal(fin, e.c0)
    y, fin, kept = e.scan(cu, initial_state=e.h0, output_final_state=True, save_states=True)
    assert torch.equal(fin, e.h0)
    d = e.conv_backward(cu, initial_state=e.c0, d_final_state=e.c0)
    assert torch.equal(d["d_initial_state"], e.c0) and not d["dweight"].any() and not d["dbias"].any()
    d = e.scan_backward(cu, kept, d_final_state=e.h0, output_d_initial_state=True)
    assert torch.equal(d["d_initial_state"], e.h0) and not d["dA"].any() and not d["dD"].any()
    y, r = e.norm()
    assert y.shape == r.shape == (0, 24)
    d = e.norm_backward(r)
    assert not d["dweight"].any() and not d["dpost_weight"].any() and not d["dscale"].any()


BAD_BOUNDS = [[0, 50, 40, 100], [5, 50, 60, 100], [0, 50, 60, 200], [0, -3, 60, 100], [0, 1 << 62, -(1 << 62), 100], [-(1 << 62)] * 4,
              [1 << 62] * 4]


@pytest.mark.parametrize("T,C", [(100, 40), (100, 2200)])
@pytest.mark.parametrize("bounds", BAD_BOUNDS)
def test_wild_bounds(cuda_device, bounds, T, C):
    """Bounds that do not ascend from 0 to at most T are reported; nothing outside the buffers is touched."""
    _wild(cuda_device, bounds, T, C)


@pytest.mark.parametrize("bounds", [[0, 500, 400, 1000], [0, 500, 600, 1 << 40], [-7, 1 << 62, -(1 << 62), 5]])
def test_wild_bounds_in_pieces(cuda_device, bounds):
    assert pkg.gdp_scan_forward_workspace_bytes(1000, 3, 40, 16) > 0
    _wild(cuda_device, bounds, 1000, 40)


def _wild(dev, bounds, T, C):
    b = Block(T, C, 16, 3, dev)
    cu, good = torch.tensor(bounds, dtype=torch.int64, device=dev), _cu([T // 2, T // 5, T // 10], dev)
    before = {k: v.clone() for k, v in vars(b).items()}
    kept = b.scan(good, save_states=True)[1]
    canary = torch.full((3, T * C), 7.0, device=dev, dtype=BF16)
    for call in (lambda st: b.conv(cu, device_status=st, output=canary[1].view(T, C)), lambda st: b.scan(cu, device_status=st, output=canary[1].view(T, C)),
                 lambda st: b.conv_backward(cu, device_status=st), lambda st: b.scan_backward(cu, kept, device_status=st)):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        call(status)
        assert int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS
        assert bool((canary[0] == 7).all()) and bool((canary[2] == 7).all())
    for k, v in before.items():
        assert torch.equal(getattr(b, k), v), k


def test_wild_slots(cuda_device):
    """Slots outside the cache are reported and treated as none, those of empty sequences too."""
    lengths, C, dev = [9, 0, 300, 3], 24, cuda_device
    b, cu = Block(sum(lengths), C, 16, 4, dev), _cu(lengths, dev)
    for slots, bad in (([0, 1, 2, 3], False), ([0, -1, 2, 3], False), ([0, 7, 2, 3], True), ([0, 1, 4, 3], True), ([0, 1, -2, 3], True),
                       ([0, 1, 2, -(2 ** 31)], True)):
        idx = torch.tensor(slots, dtype=torch.int32, device=dev)
        for call, cache in ((b.conv, b.c0), (b.scan, b.h0)):
            status, state = torch.zeros(1, dtype=torch.int32, device=dev), cache.clone()
            y = call(cu, state=state, state_indices=idx, device_status=status)
            assert bool(int(status) & pkg.GDP_DEV_ERR_SLOT) == bad, slots
            init = torch.stack([cache[s] if 0 <= s < 4 else torch.zeros_like(cache[0]) for s in slots])
            want, fin = call(cu, initial_state=init, output_final_state=True)
            assert torch.equal(y, want)
            for s in range(4):
                assert torch.equal(state[s], fin[slots.index(s)] if s in slots else cache[s])
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.short_convolution_decode(b.x[:4], b.w, state=b.c0.clone(), state_indices=idx, device_status=status)
        assert bool(int(status)) == bad
        status.zero_()
        pkg.selective_scan_decode(b.x[:4], b.dt[:4], b.A, b.B[:4], b.Cm[:4], state=b.h0.clone(), state_indices=idx, device_status=status)
        assert bool(int(status)) == bad


@pytest.mark.parametrize("lengths,C", [(LENGTHS, 70), ([40, 0, 9, 1, 77], 2200), ([700], 33)])
def test_repeats_to_the_bit(cuda_device, lengths, C):
    b, cu = Block(sum(lengths), C, 16, len(lengths), cuda_device), _cu(lengths, cuda_device)
    first = b.everything(cu)
    torch.empty(1 << 28, dtype=torch.uint8, device=cuda_device).fill_(255)  # workspaces come with something else in them
    for name, v in b.everything(cu).items():
        assert (v is None and first[name] is None) or torch.equal(v, first[name]), name


@pytest.mark.parametrize("lengths,C", [(LENGTHS, 70), ([40, 0, 9, 1, 77], 2200)])
def test_captured_and_replayed(cuda_device, lengths, C):
    """Two graphs of all calls, replayed in turn with other inputs in the same buffers, against eager calls."""
    b, cu = Block(sum(lengths), C, 16, len(lengths), cuda_device), _cu(lengths, cuda_device)
    other = Block(sum(lengths), C, 16, len(lengths), cuda_device, seed=100)
    want_other, want = other.everything(cu), b.everything(cu)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.everything(cu))
        graphs.append(g)
    for g, o in zip(graphs, outs):
        g.replay()
    for o in outs:
        for name, v in o.items():
            assert torch.equal(v, want[name]), name
    for k, v in vars(other).items():
        getattr(b, k).copy_(v)
    for g in graphs:
        g.replay()
    graphs[0].replay()
    for o in outs:
        for name, v in o.items():
            assert torch.equal(v, want_other[name]), name


def test_given_stream(cuda_device):
    """A call on a given stream runs there and allocates there."""
    lengths = [40, 0, 300, 1, 77]
    b, cu = Block(sum(lengths), 64, 16, 5, cuda_device), _cu(lengths, cuda_device)
    y, (s, kept), (n, r) = b.conv(cu), b.scan(cu, save_states=True), b.norm()
    want = [y, s, n, b.conv_backward(cu)["dweight"], b.scan_backward(cu, kept)["dA"], b.norm_backward(r)["dweight"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the side stream is busy for a while
    h = side.cuda_stream
    got_s, got_kept = b.scan(cu, save_states=True, stream=h)
    got = [b.conv(cu, stream=h), got_s, b.norm(stream=h)[0], b.conv_backward(cu, stream=h)["dweight"],
           b.scan_backward(cu, got_kept, stream=h)["dA"], b.norm_backward(r, stream=h)["dweight"]]
    assert not side.query()
    side.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_given_workspaces(cuda_device):
    """Workspaces of the stated size, with anything in them, and one byte less is refused."""
    lengths, C = [40, 0, 300, 1, 77], 64
    T, N = sum(lengths), len(lengths)
    b, cu = Block(T, C, 16, N, cuda_device), _cu(lengths, cuda_device)
    kept, r = b.scan(cu, save_states=True)[1], b.norm()[1]
    calls = [(pkg.gdp_conv_workspace_bytes(T, C, 4), lambda **k: b.conv_backward(cu, **k)["dweight"]),
             (pkg.gdp_scan_workspace_bytes(T, N, C, 16), lambda **k: b.scan_backward(cu, kept, **k)["dA"]),
             (pkg.gdp_scan_forward_workspace_bytes(T, N, C, 16), lambda **k: b.scan(cu, **k)),
             (pkg.gdp_residual_norm_workspace_bytes(T, C), lambda **k: b.norm_backward(r, **k)["dweight"])]
    for need, call in calls:
        if need == 0:
            continue
        want = call()
        room = torch.full((need + 512,), 255, dtype=torch.uint8, device=cuda_device)
        assert torch.equal(call(workspace=room[:need]), want) and bool((room[need:] == 255).all())
        with pytest.raises(pkg.GdpError):
            call(workspace=room[:need - 1])
        with pytest.raises(pkg.GdpError):
            call(workspace=room[16:16 + need])


@pytest.mark.parametrize("lengths,C", [([40, 0, 9, 30], 70), ([100, 0, 290, 400], 33)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinities_stay_in_their_sequence(cuda_device, lengths, C, bad):
    """What is not a number in one sequence (its inputs, its states) changes no bit of another one's rows and states."""
    b, cu = Block(sum(lengths), C, 16, 4, cuda_device), _cu(lengths, cuda_device)
    clean = b.everything(cu)
    last = sum(lengths[:3])
    for t in (b.x, b.z, b.dt, b.dy):
        t[last + 3::7] = bad
    b.B[last + 5] = bad
    b.h0[3], b.c0[3] = bad, bad
    got = b.everything(cu)
    for name in ("conv", "scan", "conv dx", "scan dx", "scan ddt", "scan dz", "scan dB", "scan dC", "y", "r", "norm d_block", "norm d_gate"):
        assert torch.equal(got[name][:last], clean[name][:last]), name
    for name in ("conv state", "scan state", "conv d_initial_state", "scan d_initial_state"):
        assert torch.equal(got[name][:3], clean[name][:3]), name
    y, _, _ = R.convolution(b.x.cpu(), b.w.cpu(), lengths, b.b.cpu(), "silu", b.c0.cpu())
    assert torch.equal(torch.isfinite(got["conv"].cpu()), torch.isfinite(y.to(F32)))


def test_pieces_far_from_fp32(cuda_device):
    """Few channels, so the scan runs in pieces: growing and dying states whose decays over a piece leave fp32, next to zero
    and infinite ones."""
    T, C, S, dev = 1024, 4, 4, cuda_device
    assert pkg.gdp_scan_forward_workspace_bytes(T, 1, C, S) > 0
    x, B = torch.zeros(T, C), torch.ones(T, S)
    dt, A = torch.ones(T, C), torch.zeros(C, S)
    A[0], A[1], A[2], A[3] = 1.0, -1.0, -0.25, 0.05   # factors of e^128, e^-128, e^-32, e^6.4 over 128 tokens
    x[900, 1] = 1.0
    h0 = torch.zeros(1, C, S)
    h0[0, 2], h0[0, 3, :2] = 3.0, 1e-30
    dt[:, 3] = torch.where(torch.arange(T) < 512, 1.0, -1.0)  # up by e^25.6 and down again
    h0[0, 2, 3] = math.inf
    on = [t.to(dev) for t in (x, dt, A, B, B)]
    cu = _cu([T], dev)
    y, fin, kept = pkg.selective_scan(*on, cu, dt_softplus=False, initial_state=h0.to(dev), output_final_state=True, save_states=True)
    want = R.scan(x, dt, A, B, B, [T], softplus=False, init=h0)
    wy, wf = want["y"][0], want["final"][0]
    got = y.cpu().double()
    assert bool((got[:, 0] == 0).all()) and torch.isfinite(got[:, 1]).all()
    check(y[:, 1], wy[:, 1], want["y"][1][:, 1] + 1e-37, "dying")
    check(y[:, 3], wy[:, 3], want["y"][1][:, 3], "there and back")
    assert bool((fin[0, 2, :3].cpu().double() - wf[0, 2, :3]).abs().max() <= 1e-6) and float(fin[0, 2, 3]) == math.inf
    back = pkg.selective_scan_backward(*on, torch.zeros_like(on[0]), cu, kept, dt_softplus=False, d_final_state=torch.zeros_like(fin),
                                       output_d_initial_state=True)
    assert not back["d_initial_state"].any()


def test_many_elements(cuda_device):
    """More than 2^31 elements, and offsets beyond 32 bits: first and last rows against a call on those rows alone."""
    dev, C = cuda_device, 4096
    T = (1 << 31) // C + 4096
    x = torch.empty((T, C), dtype=BF16, device=dev).normal_()
    w = _rand((C, 4), 1).to(dev)
    cut = T - 300
    cu, tail = _cu([cut, 300], dev, torch.int64), _cu([300], dev)
    y = pkg.short_convolution(x, w, cu)
    assert torch.equal(y[cut:], pkg.short_convolution(x[cut:], w, tail))
    d = pkg.short_convolution_backward(x, w, x, cu)["dx"]
    assert torch.equal(d[cut:], pkg.short_convolution_backward(x[cut:], w, x[cut:], tail)["dx"])
    del d, y
    weight = torch.ones(C, device=dev)
    y, r = pkg.residual_norm(x, x, weight, weight, x, "silu")
    y2, r2 = pkg.residual_norm(x[cut:], x[cut:], weight, weight, x[cut:], "silu")
    assert torch.equal(y[cut:], y2) and torch.equal(r[cut:], r2)
    g = pkg.residual_norm_backward(x, None, r, x, weight, weight, x, "silu")
    g2 = pkg.residual_norm_backward(x[cut:], None, r2, x[cut:], weight, weight, x[cut:], "silu")
    for name in ("d_residual", "d_block", "d_gate"):
        assert torch.equal(g[name][cut:], g2[name]), name
    del g, y, r
    A, B = -torch.rand(C, 2, device=dev), torch.empty((T, 2), dtype=BF16, device=dev).normal_()
    s, fin, kept = pkg.selective_scan(x, x, A, B, B, cu, output_final_state=True, save_states=True)
    s2, fin2, kept2 = pkg.selective_scan(x[cut:], x[cut:], A, B[cut:], B[cut:], tail, output_final_state=True, save_states=True)
    check(s[cut:], s2.cpu().double(), s2.cpu().double().abs() * 2.0 ** -8 + 1e-4, "scan")
    b1 = pkg.selective_scan_backward(x, x, A, B, B, x, cu, kept)
    b2 = pkg.selective_scan_backward(x[cut:], x[cut:], A, B[cut:], B[cut:], x[cut:], tail, kept2)
    check(b1["dx"][cut:], b2["dx"].cpu().double(), b2["dx"].cpu().double().abs() * 2.0 ** -8 + 1e-3, "scan dx")


def test_scan_of_many_groups_and_channels(cuda_device):
    """One channel per group, and a width that is no multiple of anything."""
    for C, G, S in ((37, 37, 16), (1000, 8, 20), (130, 2, 8)):
        lengths = [33, 20]
        T = 53
        v = {"x": _rand((T, C), 1), "dt": _rand((T, C), 2, sigma=0.5), "A": -torch.exp(_rand((C, S), 3)), "B": _rand((T, G, S), 4),
             "Cm": _rand((T, G, S), 5), "z": _rand((T, C), 6)}
        on = {k: t.to(cuda_device) for k, t in v.items()}
        ins, cu = (on["x"], on["dt"], on["A"], on["B"], on["Cm"]), _cu(lengths, cuda_device)
        y, kept = pkg.selective_scan(*ins, cu, z=on["z"], save_states=True)
        check(y, *R.scan(v["x"], v["dt"], v["A"], v["B"], v["Cm"], lengths, z=v["z"])["y"], "y")
        d = pkg.selective_scan_backward(*ins, on["x"], cu, kept, z=on["z"])
        want = R.scan_backward(v["x"], v["dt"], v["A"], v["B"], v["Cm"], v["x"], lengths, z=v["z"])
        for name in ("dx", "ddt", "dA", "dB", "dC", "dz"):
            check(d[name], *want[name], name)


def test_types_lowest_values(cuda_device):
    """Gates and steps at their type's lowest and largest values are finite where the formula is."""
    dev, C = cuda_device, 32
    for dt in (BF16, F16, F32):
        low, high = torch.finfo(dt).min, torch.finfo(dt).max
        z = torch.tensor([low, -100.0, -20.0, 0.0, 20.0, high], dtype=dt, device=dev)[:, None].expand(6, C).contiguous()
        x, B = torch.ones((6, C), dtype=dt, device=dev), torch.ones((6, 4), dtype=dt, device=dev)
        A, cu = -torch.ones(C, 4, device=dev), _cu([1] * 6, dev)
        y = pkg.selective_scan(x, z.clamp(max=20.0), A, B, B, cu)  # softplus of the lowest step is zero
        assert torch.isfinite(y).all() and not y[0].any()
        y = pkg.selective_scan(x, x, A, B, B, cu, z=z)
        assert not y[0].any() and torch.isfinite(y[:5]).all()
        w = torch.ones(C, device=dev)
        for act in ("sigmoid", "silu"):
            y, r = pkg.residual_norm(x, x, w, w, z, act)
            assert torch.isfinite(r[:5]).all() and torch.allclose(r[0].float(), x[0].float())
            d = pkg.residual_norm_backward(x, None, r, x, w, w, z, act)
            assert torch.isfinite(d["d_gate"][:5]).all() and torch.isfinite(d["d_block"][:5]).all()


@pytest.mark.parametrize("T", [1, 40])
def test_residual_rows_do_not_mix(cuda_device, T):
    """A row of NaN or infinities leaves the others alone, widths of one warp and of many."""
    for C in (48, 1000, 4104):
        b = Block(T + 1, C, 4, 1, cuda_device)
        (y, r), row = b.norm(), T // 2
        d = b.norm_backward(r)
        b.x[row], b.res[row], b.gate[row] = math.nan, math.inf, -math.inf
        y2, r2 = b.norm()
        d2 = b.norm_backward(r2)
        keep = [i for i in range(T + 1) if i != row]
        assert torch.equal(y[keep], y2[keep]) and torch.equal(r[keep], r2[keep])
        for name in ("d_residual", "d_block", "d_gate"):
            assert torch.equal(d[name][keep], d2[name][keep]), name


def test_a_block_trained_and_served(cuda_device):
    """The operators as one block: gradients of the whole against differences along a direction, and a prompt followed by
    single tokens against one pass over everything."""
    dev, C, S, lengths = cuda_device, 48, 16, [60, 0, 37]
    T, N = sum(lengths), len(lengths)
    b, cu = Block(T, C, S, N, dev, F32), _cu(lengths, dev)
    P = {"w": b.w * 0.5, "b": b.b * 0.1, "A": b.A, "D": b.D, "bias": b.bias, "weight": b.weight, "post": b.post, "scale": b.scale}

    def forward(P, keep=False):
        c = pkg.short_convolution(b.x, P["w"], cu, P["b"])
        s, kept = pkg.selective_scan(c, b.dt, P["A"], b.B, b.Cm, cu, D=P["D"], z=b.z, dt_bias=P["bias"], save_states=True)
        y, r = pkg.residual_norm(b.res, s, P["weight"], P["post"], b.gate, "sigmoid", P["scale"])
        return (y, r, c, s, kept) if keep else (y, r)

    y, r, c, s, kept = forward(P, True)
    n = pkg.residual_norm_backward(b.dy, b.dr, r, s, P["weight"], P["post"], b.gate, "sigmoid", P["scale"])
    m = pkg.selective_scan_backward(c, b.dt, P["A"], b.B, b.Cm, n["d_block"], cu, kept, D=P["D"], z=b.z, dt_bias=P["bias"])
    k = pkg.short_convolution_backward(b.x, P["w"], m["dx"], cu, P["b"])
    grads = {"w": k["dweight"], "b": k["dbias"], "A": m["dA"], "D": m["dD"], "bias": m["ddt_bias"], "weight": n["dweight"],
             "post": n["dpost_weight"], "scale": n["dscale"]}

    def loss(P):
        y, r = forward(P)
        return float((y.double() * b.dy).sum() + (r.double() * b.dr).sum())

    for name, g in grads.items():
        step = _rand(P[name].shape, 50).to(dev) * 2.0 ** -9
        up, down = ({**P, name: P[name] + sign * step} for sign in (1, -1))
        slope, want = (loss(up) - loss(down)) / 2, float((g.double() * step).sum())
        assert abs(slope - want) < 5e-3 * (float((g.double() * step).abs().sum()) + 1e-3), (name, slope, want)

    # serving: caches, a prompt of all but the last three tokens of the non-empty sequences, then one token at a time
    new, live = 3, [0, 2]
    starts = [sum(lengths[:i]) for i in range(N)]
    prompt = torch.cat([torch.arange(starts[i], starts[i] + lengths[i] - new) for i in live]).to(dev)
    pcu, slots = _cu([lengths[i] - new for i in live], dev), torch.tensor([2, 0], dtype=torch.int32, device=dev)
    conv, state = torch.zeros(4, 3, C, device=dev), torch.zeros(4, C, S, device=dev)

    def rows(at, step):
        where = {"state": conv, "state_indices": slots}
        c = pkg.short_convolution_decode(b.x[at], P["w"], P["b"], **where) if step else pkg.short_convolution(b.x[at], P["w"], pcu, P["b"], **where)
        ins, how = (c, b.dt[at], P["A"], b.B[at], b.Cm[at]), {"D": P["D"], "z": b.z[at], "dt_bias": P["bias"], "state": state, "state_indices": slots}
        s = pkg.selective_scan_decode(*ins, **how) if step else pkg.selective_scan(*ins, pcu, **how)
        return pkg.residual_norm(b.res[at], s, P["weight"], P["post"], b.gate[at], "sigmoid", P["scale"])[0]

    got = [rows(prompt, False)]
    assert float((got[0] - y[prompt]).abs().max()) < 1e-3
    for t in range(new):
        at = torch.tensor([starts[i] + lengths[i] - new + t for i in live], device=dev)
        assert float((rows(at, True) - y[at]).abs().max()) < 1e-3


@pytest.mark.parametrize("S", [3, 16, 20, 64])
@pytest.mark.parametrize("lengths", [[40, 9], [300, 400]])
def test_an_infinite_step(cuda_device, lengths, S):
    """A step of +inf forgets what was and takes in what the formula gives, +inf for positive x, B and C, whatever number of
    states the lanes are padded to; the channel's other sequences and the other channels are as without it."""
    dev, T, C, at, ch = cuda_device, sum(lengths), 24, 5, 3
    x, B, Cm = (1 + _rand(shape, i, F32, 1.0).abs().to(dev) for i, shape in enumerate(((T, C), (T, S), (T, S))))
    dt, A = _rand((T, C), 3, F32, 0.5).to(dev), -torch.exp(_rand((C, S), 4, F32, 0.5)).to(dev)
    cu = _cu(lengths, dev)
    clean, fin = pkg.selective_scan(x, dt, A, B, Cm, cu, output_final_state=True)
    dt[at, ch] = math.inf
    y, state = pkg.selective_scan(x, dt, A, B, Cm, cu, output_final_state=True)
    assert bool((y[at:lengths[0], ch] == math.inf).all()) and bool((state[0, ch] == math.inf).all())
    y[at:lengths[0], ch], state[0, ch] = clean[at:lengths[0], ch], fin[0, ch]
    assert torch.equal(y, clean) and torch.equal(state, fin)
    step, after = pkg.selective_scan_decode(x[at:at + 1], dt[at:at + 1], A, B[at:at + 1], Cm[at:at + 1], output_final_state=True)
    assert bool((step[0, ch] == math.inf).all()) and bool((after[0, ch] == math.inf).all())
    assert bool(torch.isfinite(step[0, :ch]).all()) and bool(torch.isfinite(after[0, ch + 1:]).all())


def test_bounds_of_no_rows(cuda_device):
    """Bounds are checked where there are no rows too, and the states pass through."""
    dev = cuda_device
    b = Block(0, 24, 16, 2, dev)
    for bounds, bad in (([0, 0, 0], False), ([0, 3, 3], True)):
        cu = torch.tensor(bounds, dtype=torch.int32, device=dev)
        for call, state in ((b.conv, b.c0), (b.scan, b.h0)):
            for how in ({}, {"initial_state": state, "output_final_state": True},
                        {"state": state.clone(), "state_indices": torch.tensor([1, 0], dtype=torch.int32, device=dev)}):
                status = torch.zeros(1, dtype=torch.int32, device=dev)
                got = call(cu, device_status=status, **how)
                assert bool(int(status) & pkg.GDP_DEV_ERR_CU_SEQLENS) == bad
                assert "initial_state" not in how or torch.equal(got[1], state)
                assert "state" not in how or torch.equal(how["state"], state)


@pytest.mark.parametrize("dtype,stream", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("gated", [False, True])
def test_residual_norm_of_many_rows_at_every_width(cuda_device, dtype, stream, gated):
    """Every width of CTA and number of rows that it has places for, with rows enough for the widest grids: the first and last
    rows against the reference."""
    dev, T, most = cuda_device, 10000, 8192
    wide = [_rand((T * 2048,), i, F32, 1.0).to(dev).to(t) for i, t in enumerate((dtype, stream, dtype, dtype, stream))]
    for C in [8, 200, 256] + list(range(264, most, 248)) + [512, 1024, 2048, 4096, 5120, most]:
        rows = min(T, T * 2048 // C)
        x, r, g, dy, dr = (v[:rows * C].view(rows, C) for v in wide)
        w, post, scale = (_rand((C,), 7 + i, F32, 0.2).add(1.0).to(dev) for i in range(3))
        g = g if gated else None
        y, out = pkg.residual_norm(r, x, w, post, g, "silu", scale)
        d = pkg.residual_norm_backward(dy, dr, out, x, w, post, g, "silu", scale)
        at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device=dev)
        few = lambda t: None if t is None else t[at].cpu()  # noqa: E731
        cols = [t.cpu() for t in (w, post)], scale.cpu()
        want = R.residual_norm(few(r), few(x), *cols[0], few(g), "silu", cols[1])
        check(few(y), *want["y"], f"y {C}")
        check(few(out), *want["r"], f"r {C}")
        want = R.residual_norm_backward(few(dy), few(dr), few(out), few(x), *cols[0], few(g), "silu", cols[1])
        for name in ("d_residual", "d_block") + (("d_gate",) if gated else ()):
            check(few(d[name]), *want[name], f"{name} {C}")
        assert all(bool(torch.isfinite(d[k]).all()) for k in ("dweight", "dpost_weight", "dscale"))


@pytest.mark.parametrize("widths", [(2200, 70), (33, 4200)])
def test_two_streams_at_once(cuda_device, widths):
    """Calls that run beside one another on two streams give the bits that they give alone."""
    dev, lengths = cuda_device, [100, 0, 290, 400]
    cu = _cu(lengths, dev)
    blocks = [Block(sum(lengths), c, 16, 4, dev, seed=c) for c in widths]
    alone = [b.everything(cu) for b in blocks]
    streams = [torch.cuda.Stream(dev) for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                got.append(b.everything(cu))
        torch.cuda.synchronize()
        for mine, want in zip(got, alone):
            for name, v in want.items():
                assert (v is None and mine[name] is None) or torch.equal(mine[name], v), name


def test_wide_rows_captured_and_replayed(cuda_device):
    """Rows of two CTAs, and pieces, in a graph that is replayed with other inputs."""
    dev, lengths = cuda_device, [30, 0, 200]
    cu, b, other = _cu(lengths, dev), Block(230, 4200, 16, 3, dev), Block(230, 4200, 16, 3, dev, seed=50)
    b.everything(cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.everything(cu)
    for source in (other, Block(230, 4200, 16, 3, dev, seed=90)):
        for name, v in vars(b).items():
            v.copy_(getattr(source, name))
        graph.replay()
        torch.cuda.synchronize()
        for name, v in source.everything(cu).items():
            assert (v is None and got[name] is None) or torch.equal(got[name], v), name
