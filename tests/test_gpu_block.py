"""The block operators on the GPU against the float64 references, each element within the derived bounds of
``tests/_block_ref.py``."""
import math

import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from tests import _block_ref as R
from tests._layer_ref import check

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(shape, seed, dtype=F32, sigma=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(dtype)


def _cu(lengths, dev, dtype=torch.int32):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=dtype, device=dev)


def _as_laid_out(t, how, dev):
    """The tensor on the GPU as a contiguous one, as a slice of wider rows, or as a slice whose rows start off every
    vector boundary."""
    if t is None:
        return None
    t = t.to(dev)
    if how == "dense":
        return t
    flat = t.reshape(t.shape[0], -1)
    pad = 16 if how == "slice" else 3
    wide = torch.full((t.shape[0], flat.shape[1] + 2 * pad), math.nan, dtype=t.dtype, device=dev)
    part = wide[:, pad:pad + flat.shape[1]]
    part.copy_(flat)
    return part if t.dim() == 2 else part.unflatten(1, t.shape[1:])


def _on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def _close(got, want, names=None):
    """Every gradient of `got` against the reference's (value, error)."""
    for name, g in got.items():
        if g is not None and (names is None or name in names):
            check(g, *want[name], name)


RAGGED = [100, 257, 0, 64, 1, 500, 2, 0, 3]

# ---- the short convolution ---------------------------------------------------------------------------
# lengths, channels, width, type, activation, bias, layout
CONV = [
    (RAGGED, 128, 4, BF16, "silu", True, "dense"), (RAGGED, 96, 3, F16, None, False, "slice"),
    (RAGGED, 61, 2, BF16, "silu", True, "odd"), (RAGGED, 66, 4, F32, "silu", False, "odd"),
    (RAGGED, 40, 4, F32, None, True, "slice"), ([1], 1, 4, BF16, "silu", True, "dense"), ([2], 8, 4, F16, "silu", False, "dense"),
    ([3], 4, 4, F32, None, True, "dense"), ([0, 0], 16, 3, BF16, "silu", True, "dense"), ([1] * 200, 24, 4, BF16, "silu", True, "dense"),
    ([15, 1, 16, 17, 31, 33, 64, 65], 264, 4, BF16, "silu", True, "dense"), ([4, 5, 6, 7, 8], 10, 3, F16, "silu", True, "odd"),
    ([3000], 64, 4, BF16, "silu", True, "dense"), ([1500, 1499], 33, 4, F32, "silu", True, "dense"),
]


def _conv_case(case, init):
    lengths, C, W, xt, act, bias, layout = case
    T, N = sum(lengths), len(lengths)
    return {"x": _rand((T, C), 1, xt), "w": _rand((C, W), 2, sigma=0.5), "b": _rand((C,), 3) if bias else None,
            "init": _rand((N, W - 1, C), 4, xt) if init else None, "dy": _rand((T, C), 5, xt),
            "dfin": _rand((N, W - 1, C), 6, xt) if init else None}


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("case", CONV)
def test_convolution(cuda_device, case, init):
    lengths, C, W, xt, act, bias, layout = case
    v, dev = _conv_case(case, init), cuda_device
    w, b, s0 = _on(dev, v["w"], v["b"], v["init"])
    y, fin = pkg.short_convolution(_as_laid_out(v["x"], layout, dev), w, _cu(lengths, dev, torch.int64 if init else torch.int32), b, act,
                                   initial_state=s0, output_final_state=True)
    want, err, wfin = R.convolution(v["x"], v["w"], lengths, v["b"], act, v["init"])
    check(y, want, err, "y")
    assert torch.equal(fin.cpu().double(), wfin), "final state"


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("case", CONV)
def test_convolution_backward(cuda_device, case, init):
    lengths, C, W, xt, act, bias, layout = case
    v, dev = _conv_case(case, init), cuda_device
    w, b, s0, dfin = _on(dev, v["w"], v["b"], v["init"], v["dfin"])
    got = pkg.short_convolution_backward(_as_laid_out(v["x"], layout, dev), w, _as_laid_out(v["dy"], layout, dev), _cu(lengths, dev), b, act,
                                         initial_state=s0, d_final_state=dfin)
    assert (got["dbias"] is None) == (b is None) and (got["d_initial_state"] is None) == (s0 is None)
    _close(got, R.convolution_backward(v["x"], v["w"], v["dy"], lengths, v["b"], act, v["init"], v["dfin"]))


@pytest.mark.parametrize("xt,C,W", [(BF16, 64, 4), (F16, 33, 3), (F32, 20, 2)])
def test_convolution_cache(cuda_device, xt, C, W):
    """The cache in place: slots in any order, padding entries, slots that nobody has; prompt, then token by token."""
    lengths, dev = [7, 0, 1, 130, 2], cuda_device
    T, N, new = sum(lengths), len(lengths), 3
    x, w, b = _rand((T, C), 1, xt), _rand((C, W), 2), _rand((C,), 3)
    steps, cache = _rand((new, N, C), 4, xt), _rand((9, W - 1, C), 5, xt)
    slots = torch.tensor([4, 8, -1, 0, 2], dtype=torch.int32)
    gx, gw, gb, gcache, gslots, gsteps = _on(dev, x, w, b, cache, slots, steps)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ys = [pkg.short_convolution(gx, gw, _cu(lengths, dev), gb, state=gcache, state_indices=gslots, device_status=status)]
    for s in gsteps:
        ys.append(pkg.short_convolution_decode(s, gw, gb, state=gcache, state_indices=gslots, device_status=status))
    assert int(status) == 0
    init = torch.stack([cache[s] if s >= 0 else torch.zeros_like(cache[0]) for s in slots.tolist()])
    at, whole = 0, []
    for i, n in enumerate(lengths):
        whole += [x[at:at + n], steps[:, i]] if int(slots[i]) >= 0 else [x[at:at + n]]
        at += n
    longer = [n + (new if int(slots[i]) >= 0 else 0) for i, n in enumerate(lengths)]
    want, err, fin = R.convolution(torch.cat(whole), w, longer, b, "silu", init)
    at = 0
    for i, n in enumerate(lengths):
        first = sum(lengths[:i])
        check(ys[0][first:first + n], want[at:at + n], err[at:at + n], "prompt")
        if int(slots[i]) >= 0:
            for k in range(new):
                check(ys[1 + k][i:i + 1], want[at + n + k][None], err[at + n + k][None], "step")
            assert torch.equal(gcache[int(slots[i])].cpu().double(), fin[i])
        else:
            for k in range(new):  # from zeros at every step
                one, e1, _ = R.convolution(steps[k, i:i + 1], w, [1], b, "silu")
                check(ys[1 + k][i:i + 1], one, e1, "padding entry")
        at += longer[i]
    rest = [i for i in range(9) if i not in slots.tolist()]
    assert torch.equal(gcache[rest].cpu(), cache[rest])


def test_convolution_states_in_place(cuda_device):
    lengths, C, dev = [5, 2, 0, 40], 24, cuda_device
    x, w, s0 = _rand((sum(lengths), C), 1, BF16), _rand((C, 4), 2), _rand((4, 3, C), 3, BF16)
    gx, gw, state = _on(dev, x, w, s0)
    y = pkg.short_convolution(gx, gw, _cu(lengths, dev), initial_state=state, output_state=state)
    want, err, fin = R.convolution(x, w, lengths, None, "silu", s0)
    check(y, want, err, "y")
    assert torch.equal(state.cpu().double(), fin)
    y = pkg.short_convolution_decode(gx[:4], gw, initial_state=state, output_state=state)
    want, err, fin = R.convolution(x[:4], w, [1] * 4, None, "silu", fin)
    check(y, want, err, "step")
    assert torch.equal(state.cpu().double(), fin)


# ---- the selective scan ------------------------------------------------------------------------------
# lengths, channels, states, groups, x's type, dt's type, softplus, gated, D, layout
SCAN = [
    (RAGGED, 64, 16, 1, BF16, BF16, True, True, True, "dense"), (RAGGED, 40, 16, 1, BF16, F32, True, False, True, "slice"),
    (RAGGED, 33, 16, 1, F16, F16, True, True, False, "odd"), (RAGGED, 24, 8, 2, F32, F32, False, True, True, "odd"),
    (RAGGED, 20, 5, 4, F32, F32, True, True, True, "dense"), (RAGGED, 48, 32, 1, BF16, BF16, True, True, True, "dense"),
    (RAGGED, 18, 64, 2, BF16, F32, True, False, True, "dense"), (RAGGED, 9, 63, 1, F16, F32, False, True, True, "odd"),
    ([1], 1, 1, 1, BF16, BF16, True, False, False, "dense"), ([1], 32, 16, 1, F32, F32, True, True, True, "dense"),
    ([2, 3], 7, 3, 7, F16, F32, True, True, True, "odd"), ([0, 0], 8, 16, 1, BF16, BF16, True, True, True, "dense"),
    ([15, 1, 16, 17, 31, 32, 33], 70, 16, 1, BF16, BF16, True, True, True, "slice"),
    ([1] * 100, 36, 16, 1, F32, F32, True, False, True, "dense"), ([1200], 32, 16, 1, BF16, BF16, True, True, True, "dense"),
    ([700, 701], 16, 17, 1, F32, F32, True, True, True, "dense"),
]
# few sequences of few channels: the plan runs them in pieces
PIECES = [
    ([1200], 32, 16, 1, BF16, BF16, True, True, True, "dense"), ([600], 20, 5, 2, F32, F32, True, True, True, "odd"),
    ([100, 0, 300, 64, 1, 1500, 0], 40, 16, 1, BF16, F32, True, False, True, "slice"), ([0, 900, 0], 48, 32, 1, F16, F16, True, True, False, "dense"),
    ([129, 127, 128, 640], 9, 64, 1, F32, F32, False, True, True, "dense"),
]


def _scan_case(case, init=True):
    lengths, C, S, G, xt, dt, softplus, gated, D, layout = case
    T, N = sum(lengths), len(lengths)
    start = torch.exp(_rand((C,), 20) - 3.0)
    return {"x": _rand((T, C), 1, xt), "dt": _rand((T, C), 2, dt, 0.5) if softplus else (start * torch.exp(_rand((T, C), 2))).to(dt),
            "A": -torch.exp(_rand((C, S), 3)) * 2.0, "B": _rand((T, G, S), 4, xt), "Cm": _rand((T, G, S), 5, xt),
            "D": _rand((C,), 6) if D else None, "z": _rand((T, C), 7, xt) if gated else None,
            "bias": torch.log(torch.expm1(start)) if softplus else None, "init": _rand((N, C, S), 8) if init else None,
            "dy": _rand((T, C), 9, xt), "dfin": _rand((N, C, S), 10) if init else None}


def _scan_inputs(v, layout, dev):
    lay = lambda t: _as_laid_out(t, layout, dev)  # noqa: E731
    ins = (lay(v["x"]), lay(v["dt"]), v["A"].to(dev), lay(v["B"]), lay(v["Cm"]))
    return ins, {"D": _on(dev, v["D"])[0], "z": lay(v["z"]), "dt_bias": _on(dev, v["bias"])[0]}


def _scan_reference(v, lengths, softplus):
    return (v["x"], v["dt"], v["A"], v["B"], v["Cm"]), dict(D=v["D"], z=v["z"], dt_bias=v["bias"], softplus=softplus, init=v["init"])


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("case", SCAN + PIECES)
def test_scan(cuda_device, case, init):
    lengths, softplus, layout, dev = case[0], case[6], case[-1], cuda_device
    v = _scan_case(case, init)
    ins, how = _scan_inputs(v, layout, dev)
    y, fin = pkg.selective_scan(*ins, _cu(lengths, dev, torch.int64 if init else torch.int32), dt_softplus=softplus,
                                initial_state=_on(dev, v["init"])[0], output_final_state=True, **how)
    args, kw = _scan_reference(v, lengths, softplus)
    want = R.scan(*args, lengths, **kw)
    check(y, *want["y"], "y")
    check(fin, *want["final"], "final state")


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("case", SCAN + PIECES)
def test_scan_backward(cuda_device, case, init):
    lengths, softplus, layout, dev = case[0], case[6], case[-1], cuda_device
    v = _scan_case(case, init)
    ins, how = _scan_inputs(v, layout, dev)
    cu = _cu(lengths, dev)
    y, kept = pkg.selective_scan(*ins, cu, dt_softplus=softplus, initial_state=_on(dev, v["init"])[0], save_states=True, **how)
    got = pkg.selective_scan_backward(*ins, _as_laid_out(v["dy"], layout, dev), cu, kept, dt_softplus=softplus,
                                      d_final_state=_on(dev, v["dfin"])[0], output_d_initial_state=init, **how)
    args, kw = _scan_reference(v, lengths, softplus)
    for name, given in (("dD", v["D"]), ("dz", v["z"]), ("ddt_bias", v["bias"]), ("d_initial_state", v["init"])):
        assert (got[name] is None) == (given is None), name
    assert got["dB"].shape == v["B"].shape and got["ddt"].dtype == v["dt"].dtype
    _close(got, R.scan_backward(*args, v["dy"], lengths, dfin=v["dfin"], **kw))


@pytest.mark.parametrize("case", PIECES)
def test_pieces_are_used(cuda_device, case):
    lengths, C, S, G = case[:4]
    assert pkg.gdp_scan_forward_workspace_bytes(sum(lengths), len(lengths), C, S, G) > 0


def test_scan_without_groups(cuda_device):
    """B and C [T, S] are one group."""
    case = ([30, 50], 12, 16, 1, BF16, BF16, True, True, True, "dense")
    v, dev = _scan_case(case), cuda_device
    ins, how = _scan_inputs(v, "dense", dev)
    cu = _cu(case[0], dev)
    a, ka = pkg.selective_scan(*ins, cu, save_states=True, **how)
    flat = (*ins[:3], ins[3][:, 0], ins[4][:, 0])
    b, kb = pkg.selective_scan(*flat, cu, save_states=True, **how)
    assert torch.equal(a, b)
    dy = v["dy"].to(dev)
    ga, gb = (pkg.selective_scan_backward(*i, dy, cu, k, **how) for i, k in ((ins, ka), (flat, kb)))
    assert gb["dB"].shape == (80, 16) and torch.equal(ga["dB"][:, 0], gb["dB"]) and torch.equal(ga["dC"][:, 0], gb["dC"])


def test_scan_gradient_against_differences(cuda_device):
    """The GPU's own forward, moved by a step in fp32, against its gradients."""
    lengths, dev = [20, 0, 37], cuda_device
    case = (lengths, 8, 6, 2, F32, F32, True, True, True, "dense")
    v = _scan_case(case)
    cu = _cu(lengths, dev)
    names = ["x", "dt", "A", "B", "Cm", "D", "z", "bias", "init"]
    vals = dict(zip(names, _on(dev, *(v[n] for n in names))))
    dy, dfin = _on(dev, v["dy"], v["dfin"])

    def call(p, **kw):
        return pkg.selective_scan(p["x"], p["dt"], p["A"], p["B"], p["Cm"], cu, D=p["D"], z=p["z"], dt_bias=p["bias"],
                                  initial_state=p["init"], **kw)

    kept = call(vals, save_states=True)[1]
    got = pkg.selective_scan_backward(*(vals[n] for n in names[:5]), dy, cu, kept, D=vals["D"], z=vals["z"], dt_bias=vals["bias"],
                                      d_final_state=dfin, output_d_initial_state=True)
    grads = dict(zip(names, (got[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state"))))

    def loss(p):
        y, fin = call(p, output_final_state=True)
        return float((y.double() * dy).sum() + (fin.double() * dfin).sum())

    for name in names:
        step = _rand(vals[name].shape, 99).to(dev) * 2.0 ** -9
        up, down = ({**vals, name: vals[name] + s * step} for s in (1, -1))
        slope = (loss(up) - loss(down)) / 2
        want = float((grads[name].double() * step).sum())
        size = float((grads[name].double() * step).abs().sum()) + 1e-3
        assert abs(slope - want) < 2e-3 * size, (name, slope, want)  # third-order terms: 2^-18 of the first


@pytest.mark.parametrize("case", [([9, 0, 1, 40, 33], 40, 16, 1, BF16, BF16, True, True, True), ([9, 0, 1, 40, 33], 6, 30, 2, F32, F32, True, False, True),
                                  ([9, 0, 1, 40, 33], 8, 64, 1, F16, F32, False, True, False)])
def test_scan_cache(cuda_device, case):
    """The cache in place: prompt, then token by token, padding entries, slots that nobody has."""
    lengths, dev, new = case[0], cuda_device, 3
    N = len(lengths)
    C, S, softplus = case[1], case[2], case[6]
    slots = [4, 8, -1, 0, 2]
    longer = [n + new for n in lengths]
    v = _scan_case((longer, *case[1:], "dense"), False)
    cache = _rand((9, C, S), 11)
    starts = [sum(longer[:i]) for i in range(N)]
    prompt = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lengths)])
    gcache, gslots = cache.to(dev), torch.tensor(slots, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def rows(at):
        return {k: (t[at] if t is not None and k in ("x", "dt", "B", "Cm", "z") else t) for k, t in v.items()}

    ins, how = _scan_inputs(rows(prompt), "dense", dev)
    ys = [pkg.selective_scan(*ins, _cu(lengths, dev), dt_softplus=softplus, state=gcache, state_indices=gslots, device_status=status, **how)]
    for k in range(new):
        ins, how = _scan_inputs(rows(torch.tensor([s + n + k for s, n in zip(starts, lengths)])), "odd" if k else "dense", dev)
        ys.append(pkg.selective_scan_decode(*ins, dt_softplus=softplus, state=gcache, state_indices=gslots, device_status=status, **how))
    assert int(status) == 0
    v["init"] = torch.stack([cache[s] if s >= 0 else torch.zeros(C, S) for s in slots])
    args, kw = _scan_reference(v, longer, softplus)
    want = R.scan(*args, longer, **kw)
    y, e = want["y"]
    for i, n in enumerate(lengths):
        first = sum(lengths[:i])
        check(ys[0][first:first + n], y[starts[i]:starts[i] + n], e[starts[i]:starts[i] + n], "prompt")
        if slots[i] >= 0:
            for k in range(new):
                check(ys[1 + k][i], y[starts[i] + n + k], e[starts[i] + n + k], "step")
            check(gcache[slots[i]], want["final"][0][i], want["final"][1][i], "cache")
    rest = [i for i in range(9) if i not in slots]
    assert torch.equal(gcache[rest].cpu(), cache[rest])


# ---- the residual norm -------------------------------------------------------------------------------
# rows, channels, block's type, residual's type, post, gate's activation ("" for none), scale, layout
NORM = [
    (37, 256, BF16, BF16, True, "sigmoid", True, "dense"), (5, 64, BF16, F32, True, "silu", False, "slice"), (7, 61, F16, F32, True, None, True, "odd"),
    (9, 255, F32, F32, False, "sigmoid", False, "odd"), (1, 1, BF16, BF16, True, "sigmoid", True, "dense"), (3, 8, F32, F32, True, "", True, "dense"),
    (33, 257, BF16, F32, True, "sigmoid", True, "dense"), (50, 1024, F16, F16, True, "silu", True, "dense"), (20, 1601, BF16, F32, True, "sigmoid", True, "odd"),
    (11, 4096, BF16, F32, True, "sigmoid", True, "slice"), (6, 4100, F32, F32, True, "sigmoid", True, "dense"), (5, 8192, BF16, BF16, True, "sigmoid", True, "dense"),
    (4, 8191, F16, F32, False, "", False, "odd"), (1000, 72, BF16, BF16, True, "sigmoid", True, "dense"), (2000, 512, BF16, F32, True, "silu", True, "dense"),
]


def _norm_case(case):
    T, C, xt, rt, post, gate, scale, layout = case
    return {"residual": _rand((T, C), 1, rt), "block": _rand((T, C), 2, xt, 2.0), "w": 1 + _rand((C,), 3, sigma=0.2),
            "post": 1 + _rand((C,), 4, sigma=0.2) if post else None, "gate": _rand((T, C), 5, xt, 2.0) if gate != "" else None,
            "scale": _rand((C,), 6) if scale else None, "dy": _rand((T, C), 7, xt), "dr": _rand((T, C), 8, rt)}


@pytest.mark.parametrize("case", NORM)
def test_residual_norm(cuda_device, case):
    layout, act, dev = case[-1], case[5] or None, cuda_device
    v = _norm_case(case)
    w, post, scale = _on(dev, v["w"], v["post"], v["scale"])
    y, r = pkg.residual_norm(*(_as_laid_out(v[k], layout, dev) for k in ("residual", "block")), w, post, _as_laid_out(v["gate"], layout, dev), act, scale)
    want = R.residual_norm(v["residual"], v["block"], v["w"], v["post"], v["gate"], act, v["scale"])
    check(y, *want["y"], "y")
    check(r, *want["r"], "r")


@pytest.mark.parametrize("onward", [False, True])
@pytest.mark.parametrize("case", NORM)
def test_residual_norm_backward(cuda_device, case, onward):
    layout, act, dev = case[-1], case[5] or None, cuda_device
    v = _norm_case(case)
    w, post, scale = _on(dev, v["w"], v["post"], v["scale"])
    lay = lambda k: _as_laid_out(v[k], layout, dev)  # noqa: E731
    got = pkg.residual_norm_backward(lay("dy"), lay("dr") if onward else None, lay("residual"), lay("block"), w, post, lay("gate"), act, scale)
    want = R.residual_norm_backward(v["dy"], v["dr"] if onward else None, v["residual"], v["block"], v["w"], v["post"], v["gate"], act, v["scale"])
    for name, given in (("d_gate", v["gate"]), ("dpost_weight", v["post"]), ("dscale", v["scale"])):
        assert (got[name] is None) == (given is None), name
    _close(got, want)


def test_residual_in_place(cuda_device):
    case = (40, 320, BF16, F32, True, "sigmoid", True, "dense")
    v, dev = _norm_case(case), cuda_device
    w, post, scale, residual, block, gate = _on(dev, *(v[k] for k in ("w", "post", "scale", "residual", "block", "gate")))
    y, r = pkg.residual_norm(residual, block, w, post, gate, "sigmoid", scale)
    y2, r2 = pkg.residual_norm(residual, block, w, post, gate, "sigmoid", scale, output_residual=residual)
    assert r2 is residual and torch.equal(r, r2) and torch.equal(y, y2)
