"""Float64 references of the layer operators (CPU, plain torch loops), with the bound on the GPU's
rounding that each output is held to.

Bounds.  u is the unit roundoff of the output type (2^-8 bf16, 2^-11 f16, 2^-24 fp32: 8, 11 and 24
significant bits, round to nearest); every fp32 operation is off by at most 2^-24 relative.  A decay or sigmoid
computed from the hardware's base-2 exponential (2^-22) with a rounded argument (|g| 2^-23) and an
approximate division (2^-22) is off by at most delta = 2^-20 + |g| 2^-23.  Along a recurrence an error
e_t obeys e_t = a_t e_{t-1} + delta (|a_t h_{t-1}| + |b_t|), whatever the grouping of the steps: each
regrouped product of decays carries one delta per factor.  Sums of n terms run in chains of at most
n / 32 + 32 additions.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25, torch.float32: 1e-37}


def gate(kind, g):
    """(a, f, delta): decay, input factor and the relative error of either on the GPU."""
    g = g.to(F64)
    delta = 2.0 ** -20 + g.abs().clamp(max=1e3) * 2.0 ** -23
    if kind == "log":
        return torch.exp(g), torch.ones_like(g), delta
    if kind == "alpha":
        return g, torch.ones_like(g), torch.full_like(g, 2.0 ** -23)
    return torch.sigmoid(g), torch.sigmoid(-g), delta


def recurrence(x, g, lengths, kind, init=None):
    """h, final [N, C] and the error bounds of both (before the output's rounding)."""
    a, f, delta = gate(kind, g)
    b = f * x.to(F64)
    C = x.shape[1]
    h, err = torch.zeros_like(b), torch.zeros_like(b)
    fin = torch.zeros(len(lengths), C, dtype=F64) if init is None else init.to(F64).clone()
    ferr = torch.zeros_like(fin)
    t = 0
    for i, n in enumerate(lengths):
        s, e = fin[i].clone(), torch.zeros(C, dtype=F64)
        for _ in range(n):
            e = a[t].abs() * e + delta[t] * ((a[t] * s).abs() + b[t].abs())
            s = a[t] * s + b[t]
            h[t], err[t] = s, e
            t += 1
        fin[i], ferr[i] = s, e
    return h, fin, err, ferr


def recurrence_backward(g, h, dout, lengths, kind, x=None, init=None, dfin=None):
    """dx, dg, dinit and their error bounds, from the states h as they are given."""
    a, f, delta = gate(kind, g)
    h, dout = h.to(F64), dout.to(F64)
    C = g.shape[1]
    dx, dg, ex, eg = (torch.zeros_like(dout) for _ in range(4))
    N = len(lengths)
    dinit = torch.zeros(N, C, dtype=F64) if dfin is None else dfin.to(F64).clone()
    einit = torch.zeros_like(dinit)
    starts = [sum(lengths[:i]) for i in range(N)]
    for i, n in enumerate(lengths):
        E, eE = dinit[i].clone(), torch.zeros(C, dtype=F64)
        for t in range(starts[i] + n - 1, starts[i] - 1, -1):
            if t > starts[i]:
                prev = h[t - 1]
            else:
                prev = init[i].to(F64) if init is not None else torch.zeros(C, dtype=F64)
            D = dout[t] + E
            eD = eE + 2.0 ** -23 * (dout[t].abs() + E.abs())
            E = a[t] * D
            eE = a[t].abs() * eD + delta[t] * E.abs()
            dx[t], ex[t] = f[t] * D, f[t] * eD + delta[t] * (f[t] * D).abs()
            if kind == "log":
                dg[t], eg[t] = E * prev, eE * prev.abs()
            elif kind == "alpha":
                dg[t], eg[t] = D * prev, eD * prev.abs()
            else:
                q = prev - x[t].to(F64)
                dg[t], eg[t] = f[t] * E * q, f[t] * (eE * q.abs() + E.abs() * (prev.abs() + x[t].to(F64).abs()) * 2.0 ** -23)
                eg[t] += delta[t] * dg[t].abs()
            eg[t] += 2.0 ** -22 * dg[t].abs()
        dinit[i], einit[i] = E, eE
    return dx, dg, dinit, ex, eg, einit


def quantize(v):
    """(codes, scales, values) of an 8-bit checkpoint of v [T, H, D]."""
    v = v.to(F64)
    D = v.shape[-1]
    nb = -(-D // 128)
    codes, scales = torch.zeros_like(v), torch.zeros(*v.shape[:-1], nb, dtype=F64)
    values = torch.zeros_like(v)
    for i in range(nb):
        part = v[..., 128 * i:128 * i + 128]
        amax = part.abs().amax(-1)
        mant, expo = torch.frexp(127.0 / amax)
        inv = torch.ldexp(torch.floor(mant * 16.0), expo - 4)
        inv = torch.where(amax < 2.0 ** -100, torch.zeros_like(inv), inv)
        bad = ~torch.isfinite(amax)
        inv = torch.where(bad, torch.zeros_like(inv), inv)
        scale = torch.where(inv > 0, 1.0 / inv, torch.zeros_like(inv))
        scale = torch.where(bad, torch.full_like(scale, math.nan), scale)
        c = torch.where(inv[..., None] > 0, torch.round(part * inv[..., None]), torch.zeros_like(part))
        codes[..., 128 * i:128 * i + 128], scales[..., i] = c, scale
        values[..., 128 * i:128 * i + 128] = c * scale[..., None]
    return codes.to(torch.int8), scales, values


def _act(act, t):
    q = torch.sigmoid(t)
    return (t * q, q * (1 + t * (1 - q))) if act == "silu" else (q, q * (1 - q))


def _normed(o, eps, center):
    m = o.mean(-1, keepdim=True) if center else torch.zeros_like(o[..., :1])
    r = 1.0 / torch.sqrt(((o - m) ** 2).mean(-1, keepdim=True) + eps)
    return (o - m) * r, r


def _norm_errors(o, n, r):
    """Bound on n's error: the mean's (a sum), the variance's (a sum) and the reciprocal root's."""
    kappa = 2.0 ** -24 * (o.shape[-1] / 32 + 32)
    return r * kappa * o.abs().mean(-1, keepdim=True) * (1 + n.abs()) + n.abs() * (kappa + 2.0 ** -21)


def group_norm(o, w, z=None, b=None, eps=1e-5, center=False, act="silu"):
    """y and its error bound."""
    o, w = o.to(F64), w.to(F64)
    n, r = _normed(o, eps, center)
    u = n * w + (b.to(F64) if b is not None else 0.0)
    eu = _norm_errors(o, n, r) * w.abs() + 2.0 ** -22 * (u.abs() + (n * w).abs())
    if z is None:
        if act is None:
            return u, eu
        q = torch.sigmoid(u)
        return u * q, 1.2 * eu + (u * q).abs() * (2.0 ** -20 + u.abs() * 2.0 ** -22)
    z = z.to(F64)
    v, _ = _act(act, z)
    return u * v, eu * v.abs() + (u * v).abs() * (2.0 ** -20 + z.abs() * 2.0 ** -22)


def group_norm_backward(dy, o, w, z=None, b=None, eps=1e-5, center=False, act="silu"):
    """dict of (gradient, error bound), from o and z as they are given."""
    dy, o, w = dy.to(F64), o.to(F64), w.to(F64)
    D = o.shape[-1]
    kappa = 2.0 ** -24 * (D / 32 + 32)
    n, r = _normed(o, eps, center)
    en = _norm_errors(o, n, r)
    u = n * w + (b.to(F64) if b is not None else 0.0)
    eu = en * w.abs() + 2.0 ** -22 * (u.abs() + (n * w).abs())
    t = u if z is None else z.to(F64)
    da = 2.0 ** -19 + t.abs() * 2.0 ** -21  # relative error of the activation's factors
    out = {}
    if act is None:
        du, edu = dy, torch.zeros_like(dy)
    elif z is None:
        _, slope = _act(act, t)
        du = dy * slope
        edu = dy.abs() * (eu + (1 + t.abs()) * da)  # |silu''| <= 1/2, |q (1 + t (1 - q))| <= 1 + |t|
    else:
        v, slope = _act(act, t)
        du, edu = dy * v, (dy * v).abs() * da
        size = (torch.sigmoid(t) * (1 + t.abs())) if act == "silu" else slope.abs()
        out["dz"] = (dy * u * slope, dy.abs() * (eu * slope.abs() + u.abs() * size * da))
    dn, edn = du * w, edu * w.abs() + 2.0 ** -23 * (du * w).abs()
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    s1 = mean(dn) if center else torch.zeros_like(r)
    s2 = mean(dn * n)
    es1 = mean(edn) + kappa * mean(dn.abs())
    es2 = mean(edn * n.abs() + dn.abs() * en) + kappa * mean((dn * n).abs())
    do = r * (dn - s1 - n * s2)
    edo = r * (edn + es1 + n.abs() * es2 + en * s2.abs() + 2.0 ** -22 * (dn.abs() + s1.abs() + (n * s2).abs()))
    er = kappa + 2.0 ** -21 + r * kappa * o.abs().mean(-1, keepdim=True)
    out["do"] = (do, edo + do.abs() * er)
    axes = (0,) if w.dim() == 2 else (0, 1)
    rows = o.shape[0] * (1 if w.dim() == 2 else o.shape[1])
    chain = 2.0 ** -24 * (rows / 32 + 1024)
    for name, v, e in (("dweight", du * n, edu * n.abs() + du.abs() * en), ("dbias", du, edu)):
        out[name] = (v.sum(axes), e.sum(axes) + chain * v.abs().sum(axes))
    return out


def check(got, ref, err, label):
    """got within its own rounding and the operation's error of ref, elementwise; NaN where ref has NaN."""
    dt = got.dtype
    got = got.detach().cpu().to(F64).reshape(ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{label}: NaN in other places"
    rest = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[rest], ref[rest]), f"{label}: infinities differ"
    bound = UNIT[dt] * (ref.abs() + err) * 1.01 + err + TINY[dt]
    off = torch.where(fine, (got - ref).abs() - bound, torch.zeros_like(ref))
    if off.numel() and float(off.max()) > 0:
        i = int(off.argmax())
        raise AssertionError(f"{label}: element {i} of {tuple(ref.shape)}: got {float(got.flatten()[i])!r}, "
                             f"reference {float(ref.flatten()[i])!r}, bound {float(bound.flatten()[i]):.3g}; "
                             f"{int((off > 0).sum())} of {off.numel()} outside")
