"""The float64 references of the block operators against autograd through independent formulations, and planted
mistakes that the bounds have to catch."""
import pytest
import torch

from tests import _block_ref as R

F64 = torch.float64
LENGTHS = [5, 0, 1, 2, 9]


def _r(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", None])
def test_convolution_gradients(W, act):
    T, C, N = sum(LENGTHS), 3, len(LENGTHS)
    x, w, b, init = _r((T, C), 1), _r((C, W), 2), _r((C,), 3), _r((N, W - 1, C), 4)
    dy, dfin = _r((T, C), 5), _r((N, W - 1, C), 6)
    leaves = [v.clone().requires_grad_() for v in (x, w, b, init)]
    xs, ws, bs, ins = leaves
    loss, at, ys, fins = 0.0, 0, [], []
    for i, n in enumerate(LENGTHS):
        signal = torch.cat([ins[i], xs[at:at + n]])
        if n:
            p = torch.nn.functional.conv1d(signal.t()[None], ws[:, None], bs, groups=C)[0].t()
            y = torch.nn.functional.silu(p) if act else p
            ys.append(y)
            loss = loss + (y * dy[at:at + n]).sum()
        fins.append(signal[n:])
        loss = loss + (signal[n:] * dfin[i]).sum()
        at += n
    got = torch.autograd.grad(loss, leaves)
    y, _, fin = R.convolution(x, w, LENGTHS, b, act, init)
    assert torch.allclose(y, torch.cat(ys).detach(), atol=1e-12) and torch.equal(fin, torch.stack(fins).detach())
    back = R.convolution_backward(x, w, dy, LENGTHS, b, act, init, dfin)
    for name, g in zip(("dx", "dweight", "dbias", "d_initial_state"), got):
        assert torch.allclose(back[name][0], g, atol=1e-12), name


@pytest.mark.parametrize("G,gated,softplus", [(1, True, True), (2, False, False), (2, True, True)])
def test_scan_gradients(G, gated, softplus):
    T, C, S, N = sum(LENGTHS), 4, 3, len(LENGTHS)
    x, dt, A, B, Cm = _r((T, C), 1), _r((T, C), 2).abs(), -_r((C, S), 3).abs(), _r((T, G, S), 4), _r((T, G, S), 5)
    D, z, bias, init = _r((C,), 6), _r((T, C), 7) if gated else None, _r((C,), 8), _r((N, C, S), 9)
    dy, dfin = _r((T, C), 10), _r((N, C, S), 11)
    names = ["dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state"]
    leaves = [None if v is None else v.clone().requires_grad_() for v in (x, dt, A, B, Cm, D, z, bias, init)]
    X, DT, AA, BB, CC, DD, Z, BI, IN = leaves
    e = torch.nn.functional.softplus(DT + BI) if softplus else DT + BI
    group = torch.arange(C) // (C // G)
    loss, t, ys, fins = 0.0, 0, [], []
    for i, n in enumerate(LENGTHS):
        h = IN[i]
        for _ in range(n):
            h = torch.exp(e[t][:, None] * AA) * h + (e[t] * X[t])[:, None] * BB[t][group]
            y = torch.einsum("cs,cs->c", h, CC[t][group]) + DD * X[t]
            y = y if Z is None else y * torch.nn.functional.silu(Z[t])
            ys.append(y)
            loss = loss + (y * dy[t]).sum()
            t += 1
        fins.append(h)
        loss = loss + (h * dfin[i]).sum()
    f = R.scan(x, dt, A, B, Cm, LENGTHS, D, z, bias, softplus, init)
    assert torch.allclose(f["y"][0], torch.stack(ys).detach(), atol=1e-12)
    assert torch.allclose(f["final"][0], torch.stack(fins).detach(), atol=1e-12)
    back = R.scan_backward(x, dt, A, B, Cm, dy, LENGTHS, D, z, bias, softplus, init, dfin)
    live = [(k, v) for k, v in zip(names, leaves) if v is not None]
    for (name, _), g in zip(live, torch.autograd.grad(loss, [v for _, v in live])):
        assert torch.allclose(back[name][0], g, atol=1e-11), name


@pytest.mark.parametrize("post,gate,act,scale", [(True, True, "sigmoid", True), (False, True, "silu", False), (True, True, None, False),
                                                 (True, False, None, True), (False, False, None, False)])
def test_residual_norm_gradients(post, gate, act, scale):
    T, C = 6, 5
    residual, block, w = _r((T, C), 1), _r((T, C), 2), _r((C,), 3)
    pw, g, sc = _r((C,), 4) if post else None, _r((T, C), 5) if gate else None, _r((C,), 6) if scale else None
    dy, dr = _r((T, C), 7), _r((T, C), 8)
    leaves = [None if v is None else v.clone().requires_grad_() for v in (residual, block, w, pw, g, sc)]
    RE, BL, WW, PW, GG, SC = leaves
    m = BL if PW is None else torch.nn.functional.rms_norm(BL, (C,), PW, 1e-5)
    if GG is not None:
        m = m * (GG if act is None else getattr(torch.nn.functional, act)(GG))
    m = m if SC is None else m * SC
    r = RE + m
    y = torch.nn.functional.rms_norm(r, (C,), WW, 1e-5)
    f = R.residual_norm(residual, block, w, pw, g, act, sc)
    assert torch.allclose(f["y"][0], y.detach(), atol=1e-12) and torch.allclose(f["r"][0], r.detach(), atol=1e-12)
    names = ["d_residual", "d_block", "dweight", "dpost_weight", "d_gate", "dscale"]
    live = [(k, v) for k, v in zip(names, leaves) if v is not None]
    back = R.residual_norm_backward(dy, dr, f["r"][0], block, w, pw, g, act, sc)
    for (name, _), grad in zip(live, torch.autograd.grad((y * dy).sum() + (r * dr).sum(), [v for _, v in live])):
        assert torch.allclose(back[name][0], grad, atol=1e-11), name


@pytest.mark.parametrize("mistake", ["state order", "tap order", "no bias"])
def test_bounds_catch_convolution_mistakes(mistake):
    x, w, b, init = (v.float() for v in (_r((20, 4), 1), _r((4, 4), 2), _r((4,), 3), _r((1, 3, 4), 4)))
    y, err, _ = R.convolution(x, w, [20], b, "silu", init)
    wrong = R.convolution(x, w.flip(1) if mistake == "tap order" else w, [20], None if mistake == "no bias" else b, "silu",
                          init.flip(1) if mistake == "state order" else init)[0]
    assert bool(((wrong - y).abs() > 2.0 ** -8 * y.abs() + err).any())


@pytest.mark.parametrize("mistake", ["decay after input", "no softplus", "group", "gate before D"])
def test_bounds_catch_scan_mistakes(mistake):
    T, C, S = 12, 4, 3
    x, dt, A, B, Cm = _r((T, C), 1), _r((T, C), 2), -_r((C, S), 3).abs(), _r((T, 2, S), 4), _r((T, 2, S), 5)
    D, z = _r((C,), 6), _r((T, C), 7)
    y, err = R.scan(x, dt, A, B, Cm, [T], D, z)["y"]
    if mistake == "decay after input":
        e = torch.nn.functional.softplus(dt)
        h, out = torch.zeros(C, S, dtype=F64), []
        group = torch.arange(C) // 2
        for t in range(T):
            h = torch.exp(e[t][:, None] * A) * (h + (e[t] * x[t])[:, None] * B[t][group])
            out.append(((h * Cm[t][group]).sum(-1) + D * x[t]) * torch.nn.functional.silu(z[t]))
        wrong = torch.stack(out)
    elif mistake == "no softplus":
        wrong = R.scan(x, dt, A, B, Cm, [T], D, z, softplus=False)["y"][0]
    elif mistake == "group":
        wrong = R.scan(x, dt, A, B.flip(1), Cm, [T], D, z)["y"][0]
    else:
        wrong = R.scan(x, dt, A, B, Cm, [T], None, z)["y"][0] + D * x
    assert bool(((wrong - y).abs() > 2.0 ** -8 * y.abs() + err).any())
