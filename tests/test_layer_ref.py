"""The layer operators' float64 references on their own ground (CPU): the gradients against reverse-mode
autograd of the forward definition and against central differences, the checkpoint's codes against their
definition, and the error bounds against planted mistakes."""
import math

import pytest
import torch

from tests import _layer_ref as R

F64 = torch.float64


def _rand(*shape, seed=0, sigma=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * sigma


def _forward(x, g, lengths, kind, init):
    """The definition in differentiable torch."""
    a = {"log": torch.exp, "alpha": lambda v: v, "sigmoid": torch.sigmoid}[kind](g)
    b = (1 - a) * x if kind == "sigmoid" else x
    rows, fins, t = [], [], 0
    for i, n in enumerate(lengths):
        s = init[i]
        for _ in range(n):
            s = a[t] * s + b[t]
            rows.append(s)
            t += 1
        fins.append(s)
    return torch.stack(rows), torch.stack(fins)


@pytest.mark.parametrize("kind", ["log", "alpha", "sigmoid"])
def test_recurrence_gradients(kind):
    lengths, C = [5, 0, 1, 9], 3
    T = sum(lengths)
    x, init = _rand(T, C, seed=1), _rand(4, C, seed=2)
    g = -_rand(T, C, seed=3).abs() * 0.3 if kind == "log" else _rand(T, C, seed=3)
    if kind == "alpha":
        g = torch.sigmoid(g)
    dh, dfin = _rand(T, C, seed=4), _rand(4, C, seed=5)
    for t in (x, g, init):
        t.requires_grad_()
    h, fin = _forward(x, g, lengths, kind, init)
    ref_h, ref_fin, _, _ = R.recurrence(x.detach(), g.detach(), lengths, kind, init.detach())
    assert torch.allclose(h, ref_h, rtol=1e-12, atol=1e-14) and torch.allclose(fin, ref_fin, rtol=1e-12, atol=1e-14)
    want = torch.autograd.grad((h * dh).sum() + (fin * dfin).sum(), (x, g, init))
    dx, dg, dinit, _, _, _ = R.recurrence_backward(g.detach(), ref_h, dh, lengths, kind, x.detach(), init.detach(), dfin)
    for name, a, b in (("dx", dx, want[0]), ("dg", dg, want[1]), ("dinit", dinit, want[2])):
        assert torch.allclose(a, b, rtol=1e-11, atol=1e-13), name
    # central differences of the loss in one entry of each
    step = 1e-5
    for name, v, grad, at in (("x", x, dx, (2, 1)), ("g", g, dg, (7, 0)), ("init", init, dinit, (3, 2))):
        vals = []
        for s in (step, -step):
            moved = {"x": x.detach().clone(), "g": g.detach().clone(), "init": init.detach().clone()}
            moved[name][at] += s
            hh, ff, _, _ = R.recurrence(moved["x"], moved["g"], lengths, kind, moved["init"])
            vals.append(float((hh * dh).sum() + (ff * dfin).sum()))
        assert math.isclose((vals[0] - vals[1]) / (2 * step), float(grad[at]), rel_tol=1e-7, abs_tol=1e-9), name


@pytest.mark.parametrize("gated,act,center,bias,per_head", [
    (True, "silu", False, False, False), (True, "sigmoid", True, True, True), (False, "silu", True, True, False),
    (False, None, False, True, True)])
def test_group_norm_gradients(gated, act, center, bias, per_head):
    T, H, D = 3, 2, 7
    o, z = _rand(T, H, D, seed=1).requires_grad_(), _rand(T, H, D, seed=2).requires_grad_() if gated else None
    shape = (H, D) if per_head else (D,)
    w, b = (1 + _rand(*shape, seed=3)).requires_grad_(), _rand(*shape, seed=4).requires_grad_() if bias else None
    dy = _rand(T, H, D, seed=5)
    c = o - o.mean(-1, keepdim=True) if center else o
    u = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w + (b if bias else 0)
    t = u if z is None else z
    y = u if act is None else u * torch.sigmoid(t) * (z if gated and act == "silu" else 1)
    det = lambda v: None if v is None else v.detach()  # noqa: E731
    ref, _ = R.group_norm(det(o), det(w), det(z), det(b), 1e-5, center, act)
    assert torch.allclose(y, ref, rtol=1e-12, atol=1e-13)
    names = [n for n, v in (("do", o), ("dz", z), ("dweight", w), ("dbias", b)) if v is not None]
    want = torch.autograd.grad((y * dy).sum(), [v for v in (o, z, w, b) if v is not None])
    got = R.group_norm_backward(dy, det(o), det(w), det(z), det(b), 1e-5, center, act)
    for name, v in zip(names, want):
        assert torch.allclose(got[name][0], v, rtol=1e-10, atol=1e-12), name
    step, at = 1e-5, (1, 1, 3)
    vals = []
    for s in (step, -step):
        moved = det(o).clone()
        moved[at] += s
        vals.append(float((R.group_norm(moved, det(w), det(z), det(b), 1e-5, center, act)[0] * dy).sum()))
    assert math.isclose((vals[0] - vals[1]) / (2 * step), float(got["do"][0][at]), rel_tol=1e-6, abs_tol=1e-8)


def test_checkpoint_codes():
    """The codes use at least 8/9 of the range, stand within half a step of the value, and are the same
    formed in fp32 or in float64 for 16-bit values (halves included)."""
    for dt in (torch.bfloat16, torch.float16):
        v = _rand(64, 3, 200, seed=9).to(dt)
        v[0, 0, :128] = (torch.arange(128) * 0.5).to(dt)  # many exact ties
        codes, scales, values = R.quantize(v)
        top = codes.to(F64).abs()[..., :128].amax(-1)
        assert int(top.min()) >= 112 and int(top.max()) <= 127
        step = scales.repeat_interleave(128, -1)[..., :200]
        assert bool(((values - v.to(F64)).abs() <= 0.5000001 * step).all())
        amax = v.float()[..., :128].abs().amax(-1, keepdim=True)
        inv = ((127.0 / amax).view(torch.int32) & -0x100000).view(torch.float32)
        assert torch.equal(torch.round(v.float()[..., :128] * inv).to(torch.int8), codes[..., :128])


def test_checkpoint_blocks_apart():
    v = torch.zeros(1, 1, 260)
    v[..., 5] = math.inf
    v[..., 130] = 3.0
    v[..., 257] = 1e-37
    codes, scales, values = R.quantize(v)
    assert bool(torch.isnan(values[..., :128]).all())
    assert bool(torch.isfinite(values[..., 128:]).all()) and float(scales[..., 2]) == 0.0
    assert int(codes[..., 130]) == 120  # 127 / 3 = 42.3, cut to 40


@pytest.mark.parametrize("mistake", ["decay after input", "carry across sequences", "final before last", "gate in base 2"])
def test_bounds_catch_planted_mistakes(mistake):
    lengths, C = [40, 30], 4
    x, g = _rand(70, C, seed=11), -_rand(70, C, seed=12).abs() * 0.05
    init = _rand(2, C, seed=13)
    h, fin, err, ferr = R.recurrence(x, g, lengths, "log", init)
    if mistake == "decay after input":
        bad, bfin, _, _ = R.recurrence(x * torch.exp(g), g, lengths, "log", init)
    elif mistake == "carry across sequences":
        bad, bfin, _, _ = R.recurrence(x, g, lengths, "log", torch.stack([init[0], fin[0]]))
    elif mistake == "final before last":
        bad, bfin = h, torch.stack([h[38], h[68]])
    else:
        bad, bfin, _, _ = R.recurrence(x, g * math.log(2), lengths, "log", init)
    with pytest.raises(AssertionError):
        R.check(bad.to(torch.bfloat16), h, err, "h")
        R.check(bfin.float(), fin, ferr, "final")
