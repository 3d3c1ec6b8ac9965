"""The layer operators at the edges of their types and of what a call may be."""
import ctypes
import math

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from tests import _layer_ref as R
from tests.test_gpu_layer import _as_laid_out, _cu, _gates, _rand

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# ---- the norm's gate far below zero.  Where sigmoid(z) is below fp32's smallest normal number it counts as zero:
# 2^-126 off, times what it is multiplied with.
FLUSH = 2.0 ** -126


@pytest.fixture
def exact_slopes(monkeypatch):
    """The reference with 1 - sigmoid(t) as sigmoid(-t): the difference cancels to 0 in 64 bits for t above 36."""
    def act(kind, t):
        q, rest = torch.sigmoid(t), torch.sigmoid(-t)
        return (t * q, q * (1 + t * rest)) if kind == "silu" else (q, q * rest)
    monkeypatch.setattr(R, "_act", act)


def _masked_gate(dt, T, H, D):
    lowest = torch.finfo(dt).min
    z = _rand((T, H, D), 2, F32, 2.0)
    values = [lowest, 0.5 * lowest, -1e36, -1e33, -1e30, -1e4, -100.0, -89.0, -88.0, -87.0, -80.0, -40.0, 40.0, 100.0]
    for i, v in enumerate(values):
        z[:, :, 3 * i] = max(v, lowest)
    z[1], z[2, :, ::2] = lowest, lowest  # a whole row masked, and half of one
    return z.to(dt)


@pytest.mark.parametrize("dt,D,act,layout", [(BF16, 128, "silu", "dense"), (BF16, 100, "sigmoid", "odd"), (F32, 128, "silu", "slice"),
                                             (F32, 1024, "sigmoid", "dense"), (F32, 61, "silu", "odd"), (F16, 64, "silu", "dense"),
                                             (BF16, 1000, "silu", "dense")])
def test_group_norm_gate_at_the_lowest_value(cuda_device, exact_slopes, dt, D, act, layout):
    dev, T, H = cuda_device, 9, 3
    o, z, dy = _rand((T, H, D), 1, dt, 2.0), _masked_gate(dt, T, H, D), _rand((T, H, D), 5, dt)
    w, b = 1 + _rand((D,), 3, sigma=0.3), _rand((D,), 4, sigma=0.3)
    on = lambda t: _as_laid_out(t, layout, dev)  # noqa: E731
    y, kept = pkg.gated_group_norm(on(o), w.to(dev), on(z), b.to(dev), activation=act, save_checkpoint=True)
    ref, err = R.group_norm(o, w, z, b, act=act)
    u = R._normed(o.double(), 1e-5, False)[0] * w + b
    R.check(y, ref, err + FLUSH * u.abs() * (z.double().abs().clamp(max=128) if act == "silu" else 1.0), "y")
    for saved in ("tensors", "checkpoint"):
        if saved == "checkpoint":  # what the codes stand for: finite, however large the block's largest value
            assert bool(torch.isfinite(kept.z.dequantize()).all())
            o, z = (c.dequantize().cpu().double() for c in kept)
        got = pkg.gated_group_norm_backward(on(dy), kept if saved == "checkpoint" else (on(o), on(z)), w.to(dev), b.to(dev),
                                            activation=act)
        ref = R.group_norm_backward(dy, o, w, z, b, act=act)
        n, r = R._normed(o.double(), 1e-5, False)
        u, size = n * w + b, FLUSH * (1 + z.double().abs().clamp(max=128)) * dy.double().abs()
        d = size * w.abs()  # of dn
        extra = {"dz": size * u.abs(), "do": r * (d + n.abs() * (d * n.abs()).mean(-1, keepdim=True)),
                 "dweight": (size * n.abs()).sum((0, 1)), "dbias": size.sum((0, 1))}
        for name in ("do", "dz", "dweight", "dbias"):
            R.check(got[name], ref[name][0], ref[name][1] + extra[name], f"{name} from {saved}")


def test_group_norm_of_itself_far_below_zero(cuda_device):
    """Without z the affine norm gates itself: weights that take it far below zero."""
    dev, D = cuda_device, 128
    o, dy, w = _rand((4, 2, D), 1, F32), _rand((4, 2, D), 2, F32), _rand((D,), 3)
    w[::4] = 1e35
    y = pkg.gated_group_norm(o.to(dev), w.to(dev))
    R.check(y, *R.group_norm(o, w), "y")
    # far below zero the slope is zero, far above it is one; in between (|u| < 128) the reference's bound
    got = pkg.gated_group_norm_backward(dy.to(dev), (o.to(dev), None), w.to(dev))
    n = R._normed(o.double(), 1e-5, False)[0]
    u = n * w
    slope = R._act("silu", u)[1]
    far = (u.abs() > 1e3).all(0).all(0)
    assert bool(far.any())
    dw = (dy.double() * slope * n).sum((0, 1))
    assert bool(torch.isfinite(got["do"]).all())
    # a sum of eight products, each off by a few 2^-22
    assert bool(((got["dweight"].cpu() - dw).abs() <= 2.0 ** -18 * (dy.double() * n).abs().sum((0, 1)))[far].all())


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("saved", ["tensors", "checkpoint"])
@pytest.mark.parametrize("bias", [False, True])
def test_empty_gated_batch(cuda_device, act, saved, bias):
    dev = cuda_device
    o = torch.empty((0, 3, 8), dtype=BF16, device=dev)
    w = torch.ones(8, device=dev)
    b = torch.zeros(8, device=dev) if bias else None
    y, kept = pkg.gated_group_norm(o, w, o.clone(), b, activation=act, save_checkpoint=True)
    d = pkg.gated_group_norm_backward(y, kept if saved == "checkpoint" else (o, o.clone()), w, b, activation=act)
    assert y.shape == o.shape and d["do"].shape == o.shape and d["dz"].shape == o.shape
    assert not bool(d["dweight"].any()) and (b is None or not bool(d["dbias"].any()))


def test_stream_argument_allocates_on_that_stream(cuda_device):
    """What a call on a given stream allocates is not memory that the current stream has yet to write."""
    dev, T, C = cuda_device, 2000, 128
    x, g, cu = _rand((T, C), 1, BF16).to(dev), _gates("log", (T, C), 2, BF16).to(dev), _cu([T], dev)
    w, z, zero = torch.ones(64, device=dev), _rand((T, 2, 64), 3, BF16).to(dev), torch.zeros((1, C), device=dev)
    side = torch.cuda.Stream()

    def calls(**how):
        h, fin = pkg.gated_linear_recurrence(x, g, cu, output_final_state=True, **how)
        y, kept = pkg.gated_group_norm(x.view(T, 2, 64), w, z, save_checkpoint=True, **how)
        d = pkg.gated_group_norm_backward(z, kept, w, **how)
        r = pkg.gated_linear_recurrence_backward(g, x, x, cu, initial_state=zero, **how)
        step = pkg.gated_linear_recurrence_decode(x, g, **how)
        return [h, fin, y, *kept.o, *kept.z, d["do"], d["dz"], d["dweight"], r["dx"], r["dg"], r["d_initial_state"], step]

    want = calls()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms: the fills below come after the calls on the other stream
    late = [torch.full_like(t, 77) for t in want for _ in range(3)] + [torch.full((1 << 22,), 77, dtype=torch.uint8, device=dev)]
    del late
    got = calls(stream=side.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cu", [[0, -2 ** 63], [0, 2 ** 63 - 1], [2 ** 63 - 1, 10], [-2 ** 63, 2 ** 63 - 1], [0, 5, -2 ** 63 + 3],
                                [2 ** 63 - 5, 2 ** 63 - 1], [0, 300]])
@pytest.mark.parametrize("C", [64, 61])
def test_wild_sequence_bounds_write_nothing_outside(cuda_device, cu, C):
    """Offsets at the ends of 64 bits are reported, and nothing but the outputs' rows is written."""
    dev, T = cuda_device, 200
    x = _rand((T, C), 1, BF16).to(dev)
    cu = torch.tensor(cu, dtype=torch.int64, device=dev)
    n = cu.numel() - 1
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    pad = 1024 * C
    fence = {k: torch.full((2 * pad + T * C,), 7.0, dtype=BF16, device=dev) for k in ("h", "dx", "dg")}
    inner = {k: v[pad:pad + T * C] for k, v in fence.items()}
    pkg.gated_linear_recurrence(x, x, cu, output=inner["h"].view(T, C), device_status=st)
    assert int(st) == pkg.GDP_DEV_ERR_CU_SEQLENS
    st.zero_()
    a = pkg.GdpRecurrenceBackwardArgs(
        g=x.data_ptr(), g_stride_t=C, h=x.data_ptr(), h_stride_t=C, d_output=x.data_ptr(), d_output_stride_t=C,
        cu_seqlens=cu.data_ptr(), T=T, N=n, C=C, dx=inner["dx"].data_ptr(), dg=inner["dg"].data_ptr(), device_status=st.data_ptr(),
        cu_seqlens_int64=1, x_dtype=pkg.GDP_DTYPE_BF16, g_dtype=pkg.GDP_DTYPE_BF16, gate=0)
    lib = pkg.layer._library()
    assert lib.gdp_linear_recurrence_backward(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == pkg.GDP_OK
    assert int(st) == pkg.GDP_DEV_ERR_CU_SEQLENS
    for k, v in fence.items():
        assert bool((v[:pad] == 7.0).all()) and bool((v[pad + T * C:] == 7.0).all()), k


# ---- rows at or past the last sequence's end (a captured batch's padding)
def _poison(*shapes):
    """Fills memory that the allocator will hand out again with NaN."""
    held = [torch.full(s, math.nan, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("lengths,T", [([130, 77], 400), ([0, 0], 130), ([64], 65), ([], 50), ([200, 0], 200)])
@pytest.mark.parametrize("C,xt,gt,kind", [(80, BF16, BF16, "log"), (61, F16, F32, "sigmoid"), (128, F32, F32, "log")])
def test_padding_rows_are_zeros(cuda_device, lengths, T, C, xt, gt, kind):
    """Of what the wrappers allocate: outputs and gradients of padding rows are zeros, so that sums over all rows
    stay right; a caller's output buffer keeps its rows."""
    dev, n = cuda_device, sum(lengths)
    x, g, dh = _rand((T, C), 1, xt).to(dev), _gates(kind, (T, C), 2, gt).to(dev), _rand((T, C), 3, xt).to(dev)
    x[n:], g[n:], dh[n:] = math.nan, math.nan, math.nan
    cu = _cu(lengths, dev)
    _poison(((T, C), xt), ((T, C), gt))
    h = pkg.gated_linear_recurrence(x, g, cu, gate=kind)
    assert not bool(h[n:].any())
    d = pkg.gated_linear_recurrence_backward(g, h, dh, cu, gate=kind, x=x if kind == "sigmoid" else None)
    assert not bool(d["dx"][n:].any()) and not bool(d["dg"][n:].any())
    if n:
        rh, _, eh, _ = R.recurrence(x.cpu()[:n], g.cpu()[:n], lengths, kind)
        R.check(h[:n], rh, eh, "h")
        dx, dg, _, ex, eg, _ = R.recurrence_backward(g.cpu()[:n], h.cpu()[:n], dh.cpu()[:n], lengths, kind, x.cpu()[:n])
        R.check(d["dx"][:n], dx, ex, "dx")
        R.check(d["dg"][:n], dg, eg + 2.0 ** -23 * dg.abs(), "dg")
    out = torch.full((T, C), 9.0, dtype=xt, device=dev)
    assert pkg.gated_linear_recurrence(x, g, cu, gate=kind, output=out) is out
    assert bool((out[n:] == 9.0).all()) and torch.equal(out[:n], h[:n])
    # behind it the norm, whose weight gradient sums over all rows
    y, kept = pkg.gated_group_norm(h.view(T, 1, C), torch.ones(C, device=dev), save_checkpoint=True)
    dy = torch.zeros((T, 1, C), dtype=xt, device=dev)
    assert bool(torch.isfinite(pkg.gated_group_norm_backward(dy, kept, torch.ones(C, device=dev))["dweight"]).all())


def test_one_row_of_any_stride(cuda_device):
    """A single row's stride means nothing, whatever the view says."""
    dev, C = cuda_device, 128
    x, g = _rand((1, C), 1, BF16), _gates("log", (1, C), 2, BF16)
    rh, rfin, eh, efin = R.recurrence(x, g, [1], "log")
    for stride in (0, 1, 8, 64, 1 << 40):
        lay = lambda t: t.to(dev).as_strided((1, C), (stride, 1))  # noqa: E731
        R.check(pkg.gated_linear_recurrence(lay(x), lay(g), _cu([1], dev)), rh, eh, f"h, stride {stride}")
        R.check(pkg.gated_linear_recurrence_decode(lay(x), lay(g)), rh, eh, f"step, stride {stride}")
        d = pkg.gated_linear_recurrence_backward(lay(g), lay(x), lay(x), _cu([1], dev))
        assert torch.equal(d["dx"].cpu(), x) and not bool(d["dg"].any())


# a value below fp32's smallest normal number may be held as zero, at any token
SMALL = 2.0 ** -125


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("C", [64, 37])
def test_gate_logits_at_the_lowest_value(cuda_device, dt, C):
    """A sigmoid gate closed by a mask: the state is dropped, the input taken whole, no gradient to the logit."""
    dev, T = cuda_device, 300
    x, dh, s0 = _rand((T, C), 1, dt), _rand((T, C), 4, dt), _rand((1, C), 3)
    g = _gates("sigmoid", (T, C), 2, dt)
    for t, v in ((5, torch.finfo(dt).min), (17, -1e4), (18, -90.0), (140, torch.finfo(dt).min), (299, -1e30)):
        g[t] = v
        x[t] = 0.0
    h, fin = pkg.gated_linear_recurrence(x.to(dev), g.to(dev), _cu([T], dev), gate="sigmoid", initial_state=s0.to(dev), output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, g, [T], "sigmoid", s0)
    # sigmoid(g) below 2^-125 may come out as that
    R.check(h, rh, eh + SMALL * (1 + rh.abs().max()), "h")
    R.check(fin, rfin, efin + SMALL * (1 + rh.abs().max()), "final")
    d = pkg.gated_linear_recurrence_backward(g.to(dev), h, dh.to(dev), _cu([T], dev), gate="sigmoid", x=x.to(dev), initial_state=s0.to(dev))
    dx, dg, dinit, ex, eg, einit = R.recurrence_backward(g, h.cpu(), dh, [T], "sigmoid", x, s0)
    R.check(d["dx"], dx, ex + 1e3 * SMALL, "dx")
    R.check(d["dg"], dg, eg + 2.0 ** -23 * dg.abs() + 1e3 * SMALL * (1 + rh.abs().max()), "dg")


# ---- products of decays beyond fp32's range: the definition never forms them
def _case(name, T, C, xt, gt):
    """(x, decays, state, upstream gradient); the strong decays are powers of two."""
    x, a, s0, dh = _rand((T, C), 1, xt), torch.full((T, C), 0.9), _rand((1, C), 3), _rand((T, C), 4, xt)
    if name != "infinite state":
        x[:], dh[:] = 0.0, 0.0
    if name == "growth of nothing":  # a masked stretch under gates above one
        a[:] = 64.0
        s0[:] = 0.0
        x[T - 20], dh[20] = 1.0, 1.0
    elif name == "growth from far below":
        a[:] = 1.0
        a[130:165] = 64.0  # by 2^210
        s0[:] = 2.0 ** -120
        dh[300] = 2.0 ** -120
    elif name == "growth of nothing, then a reset":
        a[:250], a[250], s0[:] = 64.0, 0.0, 0.0
        x[251:] = _rand((T - 251, C), 1, xt)
        dh[20] = 1.0
    elif name == "growth and its undoing":  # by 2^132 and back, or by 2^-132 and back
        a[:] = 1.0
        for lane, (at, up) in enumerate(((130, True), (130, False), (165, True), (165, False))):
            a[at:at + 22, lane::4], a[at + 22:at + 44, lane::4] = (64.0, 1 / 64) if up else (1 / 64, 64.0)
            s0[0, lane::4] = 2.0 ** (-40 if up else 60)
            dh[400, lane::4] = 2.0 ** (60 if up else -40)
    elif name == "infinite state":
        a[:] = 0.1
        s0[0, ::3], s0[0, 1::3] = math.inf, -math.inf
    elif name == "large state, strong decays":
        a[:], s0[:] = 1.0, 2.0 ** 120
        a[150:166] = 2.0 ** -10
        dh[T - 5] = 2.0 ** 119
    elif name == "large state, decays about a half":
        a[:], s0[:] = 0.5, 2.0 ** 120
        dh[T - 5] = 2.0 ** 100
    elif name == "negative decays":
        a[10:43, ::2], a[200:250, 1::2] = -64.0, -1 / 64
        s0[0, ::2], s0[0, 1::2] = 2.0 ** -100, 2.0 ** 98
        dh[150, ::2], dh[390, 1::2] = 2.0 ** -100, 2.0 ** 40
    return x, a.to(gt), s0, dh


CASES = ["growth of nothing", "growth from far below", "growth of nothing, then a reset", "growth and its undoing", "infinite state",
         "large state, strong decays", "large state, decays about a half", "negative decays"]
@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("T,C,dt,gt", [(450, 128, BF16, BF16), (450, 61, F32, F32), (3000, 64, F32, F32), (1300, 1024, BF16, F32),
                                       (1300, 515, BF16, F32), (2000, 512, BF16, BF16)])
def test_products_of_decays_beyond_fp32(cuda_device, name, T, C, dt, gt):
    dev = cuda_device
    x, a, s0, dh = _case(name, T, C, dt, gt)
    cu, lengths = _cu([T], dev), [T]
    h, fin = pkg.gated_linear_recurrence(x.to(dev), a.to(dev), cu, gate="alpha", initial_state=s0.to(dev), output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, a, lengths, "alpha", s0)
    # values that fp32 does not hold (beyond 2^127 to either side) are left out from there on, as every form's are
    held = (rh.abs() < 2.0 ** 127).cummin(0)[0].bool() if name != "infinite state" else torch.ones_like(rh, dtype=torch.bool)
    keep = lambda v, m: torch.where(m, v, torch.zeros_like(v))  # noqa: E731
    R.check(keep(h.cpu(), held), keep(rh, held), keep(eh, held) + SMALL, "h")
    R.check(keep(fin.cpu(), held[-1:]), keep(rfin, held[-1:]), keep(efin, held[-1:]) + SMALL, "final")
    # the one-token step goes the same way
    state = s0.to(dev).clone()
    for t in range(min(T, 460)):
        hs = pkg.gated_linear_recurrence_decode(x[t:t + 1].to(dev), a[t:t + 1].to(dev), gate="alpha", initial_state=state,
                                                output_state=state)
        if t % 50 == 49:
            m = held[t:t + 1]
            R.check(keep(hs.cpu(), m), keep(rh[t:t + 1], m), keep(eh[t:t + 1], m) + SMALL, f"step {t}")
    kept = _rand((T, C), 6, dt)
    got = pkg.gated_linear_recurrence_backward(a.to(dev), kept.to(dev), dh.to(dev), cu, gate="alpha", initial_state=torch.zeros_like(s0).to(dev),
                                               d_final_state=(s0 if "state" in name else torch.zeros_like(s0)).to(dev))
    dx, dg, dinit, ex, eg, einit = R.recurrence_backward(a, kept, dh, lengths, "alpha", None, torch.zeros_like(s0),
                                                         s0 if "state" in name else None)
    held = (dx.abs() < 2.0 ** 126).flip(0).cummin(0)[0].flip(0) if name != "infinite state" else torch.ones_like(held)
    small = SMALL * (1 + kept.double().abs())
    R.check(keep(got["dx"].cpu(), held), keep(dx, held), keep(ex, held) + SMALL, "dx")
    if name != "infinite state":
        R.check(keep(got["dg"].cpu(), held), keep(dg, held), keep(eg + 2.0 ** -23 * dg.abs(), held) + small, "dg")
    R.check(keep(got["d_initial_state"].cpu(), held[:1]), keep(dinit, held[:1]), keep(einit, held[:1]) + SMALL, "d_initial_state")


@pytest.mark.parametrize("gate,value", [("log", 3.0), ("log", -9.0), ("sigmoid", -9.0), ("sigmoid", -0.4)])
@pytest.mark.parametrize("C", [64, 33])
def test_long_runs_of_one_gate(cuda_device, gate, value, C):
    """Growth of nothing and strong decays of a large state, by the other gates."""
    dev, T = cuda_device, 700
    g = torch.full((T, C), value)
    x, s0 = torch.zeros((T, C)), torch.zeros((1, C))
    if value > 0:
        x[T - 25] = 1.0
    else:
        s0[:] = 2.0 ** 120
        s0[0, 1::2] = math.inf
    h, fin = pkg.gated_linear_recurrence(x.to(dev), g.to(dev), _cu([T], dev), gate=gate, initial_state=s0.to(dev), output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, g, [T], gate, s0)
    R.check(h, rh, eh + SMALL, "h")
    R.check(fin, rfin, efin + SMALL, "final")


@pytest.mark.parametrize("C", [64, 61])
@pytest.mark.parametrize("how", ["growth", "large state", "infinite state"])
def test_neighbours_keep_their_bits(cuda_device, how, C):
    """A sequence, or a pair of channels, whose products of decays leave fp32's range changes no bit of the others: not
    where its neighbours' products are tiny (below 2^-126 over a tile) either."""
    dev, lengths = cuda_device, [700, 900, 500]
    T, cu = sum(lengths), _cu(lengths, dev)
    x, dh, s0 = _rand((T, C), 1, F32).to(dev), _rand((T, C), 2, F32).to(dev), _rand((3, C), 3).to(dev)
    a = (0.3 + 0.2 * torch.rand((T, C), generator=torch.Generator().manual_seed(4))).to(dev)
    x[100:400], dh[100:400] = 0.0, 0.0  # a stretch where only the products tell

    def run(x, a, s0, dh):
        h, fin = pkg.gated_linear_recurrence(x, a, cu, gate="alpha", initial_state=s0, output_final_state=True)
        d = pkg.gated_linear_recurrence_backward(a, x, dh, cu, gate="alpha", initial_state=s0, d_final_state=s0)
        return h, fin, d["dx"], d["dg"], d["d_initial_state"]

    want = run(x, a, s0, dh)
    for rows, channels in ((slice(700, 1600), slice(0, C)), (slice(0, T), slice(6, 8))):
        x2, a2, s2, dh2 = x.clone(), a.clone(), s0.clone(), dh.clone()
        if how == "growth":
            x2[rows, channels], dh2[rows, channels] = 0.0, 0.0
            a2[rows, channels], s2[:, channels] = 8.0, 0.0
        else:
            s2[:, channels] = 2.0 ** 100 if how == "large state" else math.inf
        others = [i for i in range(3) if not (rows.start == 700 and i == 1)]
        if rows.start == 700:
            s2[others] = s0[others]
        free = torch.ones((T, C), dtype=torch.bool, device=dev)
        free[rows, channels] = False
        kept = torch.ones((3, C), dtype=torch.bool, device=dev)
        kept[1 if rows.start == 700 else slice(0, 3), channels] = False
        for was, now in zip(want, run(x2, a2, s2, dh2)):
            m = free if was.shape[0] == T else kept
            assert torch.equal(was[m], now[m])


@pytest.mark.parametrize("lengths,slots", [([4, 0, 6], [0, 7, 1]), ([4, 6, 0], [0, 1, -3]), ([0, 0], [2, 1 << 30])])
def test_slots_of_empty_sequences_are_checked(cuda_device, lengths, slots):
    """A slot outside the cache is reported for a sequence without tokens too; nothing of the cache is written for it."""
    dev, C = cuda_device, 96
    x = _rand((sum(lengths), C), 1, BF16).to(dev)
    cache, st = _rand((3, C), 2).to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    before = cache.clone()
    pkg.gated_linear_recurrence(x, x, _cu(lengths, dev), state=cache, state_indices=torch.tensor(slots, dtype=torch.int32, device=dev),
                                device_status=st)
    assert int(st) == pkg.GDP_DEV_ERR_SLOT
    written = [s for s, n in zip(slots, lengths) if n and 0 <= s < 3]
    rest = [s for s in range(3) if s not in written]
    assert torch.equal(cache[rest], before[rest])
    st.zero_()
    ok = torch.tensor([s if 0 <= s < 3 else -1 for s in slots], dtype=torch.int32, device=dev)
    pkg.gated_linear_recurrence(x, x, _cu(lengths, dev), state=cache, state_indices=ok, device_status=st)
    assert int(st) == 0
