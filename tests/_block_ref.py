"""Float64 references of the block operators (CPU, plain torch loops), with the bound on the GPU's rounding that
each output is held to (``check`` of ``tests/_layer_ref.py`` adds the output type's own rounding).

Bounds.  Every fp32 operation is off by at most 2^-24 relative; a sum of n terms in any order by n 2^-24 times the sum of
their sizes.  A sigmoid from the hardware's exponential (2^-22, its rounded argument |v| 2^-23) and reciprocal
(2^-22) is off by at most ACT(v) = 2^-20 + |v| 2^-22 relative, and so are e^v and softplus(v) (its series adds
2^-22).  A decay exp(e A) whose exponent is off by a relative r is off by |e A| (r + 2^-22) + 2^-21, and an error
of a state decays along the recurrence with it.  Grouping the steps of a recurrence changes none of this but the number
of roundings, which the factor of two in STEP covers.
"""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24
STEP = 2.0 ** -22


def act_error(v):
    return 2.0 ** -20 + v.abs() * 2.0 ** -22


def activation(act, v):
    """(value, slope) of "silu", "sigmoid" or None (the value itself)."""
    if act is None:
        return v, torch.ones_like(v)
    q = torch.sigmoid(v)
    return (v * q, q * (1 + v * (1 - q))) if act == "silu" else (q, q * (1 - q))


def _slope_error(act, v, ev):
    """Of the slope, for a v that is off by ev (the second derivatives are below 1/2)."""
    return torch.zeros_like(v) if act is None else 0.5 * ev + (1 + v.abs()) * 2 * act_error(v)


# ---- the short convolution ---------------------------------------------------------------------------

def _signals(x, lengths, init, K):
    at = 0
    for i, n in enumerate(lengths):
        old = torch.zeros(K, x.shape[1], dtype=F64) if init is None else init[i].to(F64)
        yield i, at, n, torch.cat([old, x[at:at + n].to(F64)])
        at += n


def _taps(signal, w, b, n):
    W = w.shape[1]
    terms = [w[:, j] * signal[j:j + n] for j in range(W)]
    p, size = sum(terms), sum(t.abs() for t in terms)
    if b is not None:
        p, size = p + b, size + b.abs()
    return p, size * U * (W + 1)


def convolution(x, w, lengths, b=None, act="silu", init=None):
    """y, its error, and the final states (exact)."""
    w, b = w.to(F64), None if b is None else b.to(F64)
    K = w.shape[1] - 1
    y, err = (torch.zeros(x.shape, dtype=F64) for _ in range(2))
    fin = torch.zeros(len(lengths), K, x.shape[1], dtype=F64)
    for i, at, n, signal in _signals(x, lengths, init, K):
        p, ep = _taps(signal, w, b, n)
        v = activation(act, p)[0]
        y[at:at + n] = v
        err[at:at + n] = 1.1 * ep + (v.abs() * act_error(p) if act else 0.0)
        fin[i] = signal[n:]
    return y, err, fin


def convolution_backward(x, w, dy, lengths, b=None, act="silu", init=None, dfin=None):
    """dict of (gradient, error bound)."""
    w, b, dy = w.to(F64), None if b is None else b.to(F64), dy.to(F64)
    C, W = w.shape
    K, T = W - 1, x.shape[0]
    out = {k: torch.zeros(s, dtype=F64) for k, s in (("dx", (T, C)), ("dweight", (C, W)), ("dbias", (C,)),
                                                     ("d_initial_state", (len(lengths), K, C)))}
    err = {k: torch.zeros_like(v) for k, v in out.items()}
    chain = U * (T + 64)
    for i, at, n, signal in _signals(x, lengths, init, K):
        p, ep = _taps(signal, w, b, n)
        dp = dy[at:at + n] * activation(act, p)[1]
        edp = dy[at:at + n].abs() * _slope_error(act, p, ep) + 2 * U * dp.abs()
        ds, es = torch.zeros_like(signal), torch.zeros_like(signal)
        for j in range(W):
            ds[j:j + n] += w[:, j] * dp
            es[j:j + n] += w[:, j].abs() * (edp + 8 * U * dp.abs())
            out["dweight"][:, j] += (dp * signal[j:j + n]).sum(0)
            err["dweight"][:, j] += ((edp + chain * dp.abs()) * signal[j:j + n].abs()).sum(0)
        if dfin is not None:
            ds[n:] += dfin[i].to(F64)
            es[n:] += 2 * U * dfin[i].to(F64).abs()
        out["dbias"] += dp.sum(0)
        err["dbias"] += (edp + chain * dp.abs()).sum(0)
        out["d_initial_state"][i], err["d_initial_state"][i] = ds[:K], es[:K]
        out["dx"][at:at + n], err["dx"][at:at + n] = ds[K:], es[K:]
    return {k: (v, err[k]) for k, v in out.items()}


# ---- the selective scan ------------------------------------------------------------------------------

def _steps(dt, dt_bias, softplus):
    """(e, its relative error, de/dv, that one's relative error)."""
    v = dt.to(F64) if dt_bias is None else dt.to(F64) + dt_bias.to(F64)
    if not softplus:
        return v, torch.full_like(v, U), torch.ones_like(v), torch.zeros_like(v)
    e = torch.logaddexp(v, torch.zeros_like(v))
    return e, 2.0 ** -19 + v.abs() * 2.0 ** -22, torch.sigmoid(v), act_error(v)


def _grouped(v, C):
    """[T, G, S] or [T, S] -> [T, C, S] in fp64."""
    v = v.to(F64)
    v = v[:, None] if v.dim() == 2 else v
    return v.repeat_interleave(C // v.shape[1], 1)


def scan(x, dt, A, B, C, lengths, D=None, z=None, dt_bias=None, softplus=True, init=None, history=False):
    """dict of (value, error): y, final; with history the states before every token and after it, and the
    ungated readout, for the backward pass."""
    e, re, _, _ = _steps(dt, dt_bias, softplus)
    x, A = x.to(F64), A.to(F64)
    T, ch = x.shape
    B, C = _grouped(B, ch), _grouped(C, ch)
    S, N = A.shape[1], len(lengths)
    fin, efin = torch.zeros(N, ch, S, dtype=F64), torch.zeros(N, ch, S, dtype=F64)
    if init is not None:
        fin = init.to(F64).clone()
    y, ey = torch.zeros(T, ch, dtype=F64), torch.zeros(T, ch, dtype=F64)
    before, after = (torch.zeros(T, ch, S, dtype=F64) if history else None for _ in range(2))
    errors = torch.zeros(T, ch, S, dtype=F64) if history else None
    t = 0
    for i, n in enumerate(lengths):
        h, eh = fin[i].clone(), efin[i].clone()
        for _ in range(n):
            ex = e[t][:, None] * A
            a, b = torch.exp(ex), (e[t] * x[t])[:, None] * B[t]
            ra = ex.abs() * (re[t][:, None] + STEP) + 2.0 ** -21
            if history:
                before[t], errors[t] = h, eh
            eh = a * eh * (1 + 2.0 ** -20) + (a * h).abs() * (ra + STEP) + b.abs() * (re[t][:, None] + STEP)
            h = a * h + b
            if history:
                after[t] = h
            y[t] = (C[t] * h).sum(-1)
            ey[t] = (C[t].abs() * (eh + h.abs() * U * (S + 4))).sum(-1)
            t += 1
        fin[i], efin[i] = h, eh
    if D is not None:
        y, ey = y + D.to(F64) * x, ey + 4 * U * (D.to(F64) * x).abs()
    plain, eplain = y, ey + 2 * U * y.abs()
    if z is not None:
        v = activation("silu", z.to(F64))[0]
        y, ey = y * v, ey * v.abs() + (y * v).abs() * act_error(z.to(F64)) + 2 * U * (y * v).abs()
    out = {"y": (y, ey), "final": (fin, efin)}
    if history:
        out.update(before=before, after=after, errors=errors, plain=(plain, eplain))
    return out


def scan_backward(x, dt, A, B, C, dy, lengths, D=None, z=None, dt_bias=None, softplus=True, init=None, dfin=None):
    """dict of (gradient, error bound)."""
    f = scan(x, dt, A, B, C, lengths, D, z, dt_bias, softplus, init, history=True)
    e, re, slope, rs = _steps(dt, dt_bias, softplus)
    shape, G = B.shape, 1 if B.dim() == 2 else B.shape[1]
    x, A, dy = x.to(F64), A.to(F64), dy.to(F64)
    T, ch = x.shape
    S, N = A.shape[1], len(lengths)
    B, C = _grouped(B, ch), _grouped(C, ch)
    g, eg, out = dy, torch.zeros_like(dy), {}
    if z is not None:
        zz = z.to(F64)
        v, sl = activation("silu", zz)
        plain, eplain = f["plain"]
        out["dz"] = (dy * plain * sl, dy.abs() * (eplain * sl.abs() + plain.abs() * (1 + zz.abs()) * 2 * act_error(zz)))
        g, eg = dy * v, (dy * v).abs() * (act_error(zz) + 2 * U)
    dinit = torch.zeros(N, ch, S, dtype=F64) if dfin is None else dfin.to(F64).clone()
    einit = torch.zeros_like(dinit)
    names = {"u": (T, ch), "v": (T, ch), "dA": (ch, S), "dB": (T, ch, S), "dC": (T, ch, S)}
    val, err = ({k: torch.zeros(s, dtype=F64) for k, s in names.items()} for _ in range(2))
    at = 0
    chain = U * (T + 64)
    for i, n in enumerate(lengths):
        back, eb = dinit[i].clone(), einit[i].clone()
        for t in range(at + n - 1, at - 1, -1):
            ex = e[t][:, None] * A
            a = torch.exp(ex)
            ra = ex.abs() * (re[t][:, None] + STEP) + 2.0 ** -21
            gr, er = g[t][:, None], re[t][:, None] + STEP
            H = gr * C[t] + back
            eH = eb + eg[t][:, None] * C[t].abs() + STEP * ((gr * C[t]).abs() + back.abs())
            d = (e[t] * x[t])[:, None]
            h, hb, eh = f["after"][t], f["before"][t], f["errors"][t]
            eha = a * eh * (1 + 2.0 ** -20) + (a * hb).abs() * (ra + STEP) + (d * B[t]).abs() * er
            val["dB"][t], err["dB"][t] = H * d, (eH + H.abs() * er) * d.abs()
            val["dC"][t], err["dC"][t] = gr * h, eg[t][:, None] * h.abs() + gr.abs() * (eha + U * h.abs())
            val["u"][t], err["u"][t] = (H * B[t]).sum(-1), ((eH + H.abs() * U * (S + 4)) * B[t].abs()).sum(-1)
            back, eb = a * H, a * eH * (1 + 2.0 ** -20) + (a * H).abs() * (ra + STEP)
            w, ew = back * hb, eb * hb.abs() + back.abs() * (eh + STEP * hb.abs())
            val["v"][t], err["v"][t] = (w * A).sum(-1), ((ew + w.abs() * U * (S + 4)) * A.abs()).sum(-1)
            val["dA"] += w * e[t][:, None]
            err["dA"] += (ew + w.abs() * (re[t][:, None] + chain)) * e[t][:, None].abs()
        dinit[i], einit[i] = back, eb
        at += n
    u, v, eu, ev = val["u"], val["v"], err["u"], err["v"]
    Dv = torch.zeros(ch, dtype=F64) if D is None else D.to(F64)
    out["dx"] = (u * e + g * Dv, (eu + u.abs() * (re + STEP)) * e.abs() + (eg + STEP * g.abs()) * Dv.abs())
    de, ede = v + u * x, ev + eu * x.abs() + STEP * (v.abs() + (u * x).abs())
    ddt, eddt = de * slope, slope * (ede + de.abs() * (rs + STEP))
    out["ddt"] = (ddt, eddt)
    out["ddt_bias"] = (ddt.sum(0), (eddt + chain * ddt.abs()).sum(0))
    out["dD"] = ((g * x).sum(0), ((eg + chain * g.abs()) * x.abs()).sum(0))
    out["dA"] = (val["dA"], err["dA"])
    for k in ("dB", "dC"):
        per = val[k].view(T, G, ch // G, S)
        e2 = err[k].view(T, G, ch // G, S) + U * (ch // G + 8) * per.abs()
        out[k] = (per.sum(2).reshape(shape), e2.sum(2).reshape(shape))
    out["d_initial_state"] = (dinit, einit)
    return out


# ---- the residual norm -------------------------------------------------------------------------------

def _unit(v, eps):
    r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _sum_error(C):
    return U * (C / 32 + 32)


def residual_norm(residual, block, w, post=None, gate=None, act="sigmoid", scale=None, eps=1e-5):
    """dict of (value, error): y and r."""
    residual, m, w = residual.to(F64), block.to(F64), w.to(F64)
    kappa = _sum_error(m.shape[1]) + 2.0 ** -21
    rel = torch.full_like(m, 4 * U)
    if post is not None:
        m, rel = _unit(m, eps)[0] * post.to(F64), rel + kappa
    if gate is not None:
        m = m * activation(act, gate.to(F64))[0]
        rel = rel + act_error(gate.to(F64))
    if scale is not None:
        m = m * scale.to(F64)
    r = residual + m
    er = m.abs() * rel + 2 * U * (residual.abs() + m.abs())
    n, inv = _unit(r, eps)
    en = inv * er + n.abs() * ((n.abs() * er).mean(-1, keepdim=True) * inv + kappa)
    return {"r": (r, er), "y": (n * w, en * w.abs() + 2 * U * (n * w).abs())}


def _unit_back(dn, edn, n, inv, C):
    """Gradient through n = v inv(v), and its error."""
    kappa = _sum_error(C)
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    en = n.abs() * (kappa + 2.0 ** -21)
    s, es = mean(dn * n), mean(edn * n.abs() + dn.abs() * en) + kappa * mean((dn * n).abs())
    d = inv * (dn - n * s)
    return d, inv * (edn + n.abs() * es + en * s.abs() + 2.0 ** -22 * (dn.abs() + (n * s).abs())) + d.abs() * (kappa + 2.0 ** -21)


def residual_norm_backward(dy, dr, r, block, w, post=None, gate=None, act="sigmoid", scale=None, eps=1e-5):
    """dict of (gradient, error bound), from r as it is given."""
    dy, r, block, w = dy.to(F64), r.to(F64), block.to(F64), w.to(F64)
    T, C = block.shape
    kappa = _sum_error(C) + 2.0 ** -21
    chain = U * (T + 64)
    out = {}
    n, inv = _unit(r, eps)
    out["dweight"] = ((dy * n).sum(0), ((dy * n).abs() * (kappa + chain)).sum(0))
    d, ed = _unit_back(dy * w, 2 * U * (dy * w).abs(), n, inv, C)
    if dr is not None:
        d, ed = d + dr.to(F64), ed + 2 * U * (d.abs() + dr.to(F64).abs())
    out["d_residual"] = (d, ed)
    m, q = _unit(block, eps) if post is not None else (block, None)
    em = m.abs() * kappa if post is not None else torch.zeros_like(m)
    pw = post.to(F64) if post is not None else torch.ones(C, dtype=F64)
    sc = scale.to(F64) if scale is not None else torch.ones(C, dtype=F64)
    a, sl, ra = torch.ones_like(m), None, torch.zeros_like(m)
    if gate is not None:
        v = gate.to(F64)
        a, sl = activation(act, v)
        ra = act_error(v) if act else ra
        size = dg_scale = (d * sc * m * pw)
        esl = _slope_error(act, v, torch.zeros_like(v))
        out["d_gate"] = (size * sl, (ed * (sc * m * pw).abs() + (d * sc * pw).abs() * em + 8 * U * dg_scale.abs()) * sl.abs() + size.abs() * esl)
    if scale is not None:
        t = d * a * m * pw
        out["dscale"] = (t.sum(0), (ed * (a * m * pw).abs() + (d * a * pw).abs() * em + t.abs() * (ra + 8 * U + chain)).sum(0))
    dm, edm = d * a * sc, (ed * a.abs() + (d * a).abs() * (ra + 4 * U)) * sc.abs()
    if post is not None:
        out["dpost_weight"] = ((dm * m).sum(0), (edm * m.abs() + dm.abs() * em + (dm * m).abs() * chain).sum(0))
        dm, edm = _unit_back(dm * pw, edm * pw.abs() + 2 * U * (dm * pw).abs(), m, q, C)
    out["d_block"] = (dm, edm)
    return out
