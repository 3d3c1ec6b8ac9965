"""Measured cases of the recurrent layer's operators: the gated linear recurrence (packed sequences, its
backward pass, its one-token step) and the grouped norm with an activated gate, whose 8-bit activation
checkpoints the backward passes read.

``own`` selects what ``run`` calls: the plain form below (elementary torch operations in fp32, rounded once
at the end) or the framework's operators.  ``exact`` computes the same outputs in 64 bits.

Recurrence, per packed sequence and channel:  h_t = a_t h_{t-1} + b_t, with (a, b) from the gate value g and
the input x:  "log": (exp g, x);  "alpha": (g, x);  "sigmoid": (s(g), (1 - s(g)) x).
Norm over the D channels of each (token, head):  y = (n w + bias) act(z),  n = (o - m) / sqrt(var + eps)
(m = 0 unless centred; without z the activation takes the norm itself).
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MOST = 65536 * 4096  # elements of the largest case


def _batching():
    """64 lengths, log-uniform in [16, 8192], one of them replaced by an empty request."""
    import random
    r = random.Random(1005)
    n = [int(math.exp(r.uniform(math.log(16), math.log(8192)))) for _ in range(64)]
    n[17] = 0
    return ",".join(map(str, n))


def listed():
    return [
        # a small packed batch with ragged lengths, entering states given: the latency of a short prefill
        {"name": "rec_fwd_varlen", "kind": "rec_fwd", "lengths": "100,257,64,1000", "C": 1024, "gate": "log",
         "xt": "bf16", "gt": "f32", "init": True, "fused": False},
        # the long-context prefill: one sequence, the full width of 32 heads of 128
        {"name": "rec_fwd_long", "kind": "rec_fwd", "lengths": "65536", "C": 4096, "gate": "log", "xt": "bf16",
         "gt": "bf16", "init": True, "fused": False},
        # dynamic batching: 64 requests of very different lengths, x and g two slices of one projection
        {"name": "rec_fwd_batching", "kind": "rec_fwd", "lengths": _batching(), "C": 2048, "gate": "sigmoid",
         "xt": "bf16", "gt": "bf16", "init": False, "fused": True},
        # a training batch, gradients of x, the gate's logits and the initial state
        {"name": "rec_bwd_batch", "kind": "rec_bwd", "lengths": ",".join(["4096"] * 8), "C": 2048,
         "gate": "sigmoid", "xt": "bf16", "gt": "bf16", "init": True, "q8": False},
        # training on one long sequence, the states kept in 8 bits
        {"name": "rec_bwd_long_q8", "kind": "rec_bwd", "lengths": "65536", "C": 4096, "gate": "log", "xt": "bf16",
         "gt": "bf16", "init": False, "q8": True},
        # a serving step over the state cache, some requests of the captured batch size padding
        {"name": "step_serving", "kind": "step", "N": 64, "C": 2048, "gate": "sigmoid", "xt": "bf16", "gt": "bf16",
         "slots": 128, "padding": 8},
        # one user's next token
        {"name": "step_one", "kind": "step", "N": 1, "C": 4096, "gate": "log", "xt": "f16", "gt": "f32",
         "slots": 8, "padding": 0},
        # the output stage of one serving step: 64 tokens, 16 heads
        {"name": "norm_serving", "kind": "norm", "T": 64, "H": 16, "D": 128, "act": "silu", "gated": True,
         "center": False, "bias": False, "per_head": False, "type": "bf16", "fused": True},
        # a prefill's output stage in the centred form with affine channels and its own activation, small heads
        {"name": "norm_ragged", "kind": "norm", "T": 1421, "H": 25, "D": 64, "act": "silu", "gated": False,
         "center": True, "bias": True, "per_head": True, "type": "f16", "fused": False},
        # a training step of the output stage (forward with 8-bit checkpoints, backward from them)
        {"name": "norm_train_batch", "kind": "norm_train", "T": 32768, "H": 16, "D": 128, "act": "silu",
         "gated": True, "center": False, "bias": False, "per_head": False, "type": "bf16", "fused": False},
        # the same over the long sequence, 32 heads
        {"name": "norm_train_long", "kind": "norm_train", "T": 65536, "H": 32, "D": 128, "act": "silu",
         "gated": True, "center": False, "bias": False, "per_head": False, "type": "bf16", "fused": False},
        # one group as wide as the model, centred, on a small packed batch
        {"name": "norm_train_wide", "kind": "norm_train", "T": 1421, "H": 1, "D": 4096, "act": "sigmoid",
         "gated": True, "center": True, "bias": True, "per_head": True, "type": "bf16", "fused": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A channel count over [lo, hi]: half of them multiples of 64, the others as they fall (odd ones too)."""
    c = _log_int(rng, lo, hi)
    return max(lo, c // 64 * 64) if rng.random() < 0.5 and c >= 64 else c


def draw(rng):
    kind = rng.choice(["rec_fwd", "rec_bwd", "step", "norm", "norm_train"])
    xt = rng.choice(["bf16", "bf16", "f16", "f32"])
    gate = rng.choice(["log", "alpha", "sigmoid"])
    gt = rng.choice([xt, "f32"])
    if gate == "alpha" and gt != "f32":
        gate = "log"  # decays near one are not held in 16 bits
    if kind in ("rec_fwd", "rec_bwd"):
        c = _width(rng, 16, 4096)
        total = _log_int(rng, 1, 65536 if xt != "f32" else 32768)
        n = _log_int(rng, 1, 64)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        if n > 2 and rng.random() < 0.3:
            lengths[lengths.index(min(lengths))] = 0
        case = {"kind": kind, "lengths": ",".join(map(str, lengths)), "C": c, "gate": gate, "xt": xt, "gt": gt,
                "init": rng.random() < 0.5}
        if kind == "rec_fwd":
            case["fused"] = rng.random() < 0.5 and gt == xt
        else:
            case["q8"] = rng.random() < 0.5
        return case
    if kind == "step":
        n = _log_int(rng, 1, 512)
        return {"kind": kind, "N": n, "C": _width(rng, 16, 4096), "gate": gate, "xt": xt, "gt": gt,
                "slots": n + rng.randint(0, 64), "padding": rng.randint(0, n // 4)}
    d = rng.choice([_log_int(rng, 16, 4096), 64, 96, 128, 192, 256])
    h = 1 if d > 512 else _log_int(rng, 1, 32)
    t = _log_int(rng, 1, min(65536, MOST // (h * d)) // (2 if xt == "f32" else 1))
    gated = rng.random() < 0.7
    return {"kind": kind, "T": t, "H": h, "D": d, "act": rng.choice(["silu", "sigmoid"]) if gated else "silu",
            "gated": gated, "center": rng.random() < 0.4, "bias": rng.random() < 0.4, "per_head": rng.random() < 0.4,
            "type": xt, "fused": rng.random() < 0.5}


# ---- inputs ------------------------------------------------------------------------------------------

def _gate(case, rows, gen):
    """Gate values as such layers produce them: decays exp(-U(0, 0.05)), logits around 2."""
    shape = (rows, case["C"])
    if case["gate"] == "sigmoid":
        g = torch.randn(shape, generator=gen, device="cuda") + 2.0
    else:
        g = torch.rand(shape, generator=gen, device="cuda") * -0.05
        if case["gate"] == "alpha":
            g = g.exp()
    return g.to(TYPES[case["gt"]])


def _packed(case):
    """cu_seqlens and the host's view of it: first and last rows of the non-empty sequences, their numbers."""
    lengths = [int(n) for n in case["lengths"].split(",")]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    full = [i for i, n in enumerate(lengths) if n > 0]
    dev = {"cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}
    for name, v in (("first", [cu[i] for i in full]), ("last", [cu[i + 1] - 1 for i in full]), ("seq", full)):
        dev[name] = torch.tensor(v, dtype=torch.int64, device="cuda")
    return lengths, cu[-1], dev


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]

    def normal(shape, dtype=torch.float32, sigma=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)

    s = {"case": case}
    if kind in ("rec_fwd", "rec_bwd"):
        lengths, rows, dev = _packed(case)
        s.update(dev)
        c, n, xt = case["C"], len(lengths), TYPES[case["xt"]]
        x, g = normal((rows, c), xt), _gate(case, rows, gen)
        if case.get("fused"):  # two slices of one projection's output
            both = torch.cat([x, g], 1)
            x, g = both[:, :c], both[:, c:]
        s.update(x=x, g=g, init=normal((n, c), sigma=0.5) if case["init"] else None)
        if kind == "rec_bwd":
            h = _rec_fwd(s)[0]
            s["dout"] = normal((rows, c), xt)
            s["dfin"] = normal((n, c), sigma=0.5) if case["init"] else None
            if case["q8"]:
                s["codes"], s["scales"] = _quantize(h.float().view(rows, 1, c))
            else:
                s["h"] = h
            if case["gate"] != "sigmoid":
                del s["x"]
    elif kind == "step":
        n, c = case["N"], case["C"]
        slot = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
        pad = torch.randperm(n, generator=gen, device="cuda")[:case["padding"]]
        slot[pad] = -1
        live = (slot >= 0).nonzero()[:, 0]
        s.update(x=normal((n, c), TYPES[case["xt"]]), g=_gate(case, n, gen), slot=slot, live=live,
                 live_slot=slot[live].long(), cache=normal((case["slots"], c), sigma=0.5))
    else:
        t, h, d, xt = case["T"], case["H"], case["D"], TYPES[case["type"]]
        parts = 2 if case["gated"] else 1
        if case["fused"]:  # o and z are slices of one wider buffer
            rows = normal((t, parts * h * d + 8), xt)
            o = rows[:, :h * d].view(t, h, d)
            z = rows[:, h * d:2 * h * d].view(t, h, d) if case["gated"] else None
        else:
            o, z = normal((t, h, d), xt), normal((t, h, d), xt) if case["gated"] else None
        shape = (h, d) if case["per_head"] else (d,)
        s.update(o=o, z=z, w=1.0 + normal(shape, sigma=0.1), b=normal(shape, sigma=0.1) if case["bias"] else None)
        if kind == "norm_train":
            s["dy"] = normal((t, h, d), xt)
    return s


# ---- plain forms -------------------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis from h = 0: pairs of steps are composed, the half-length
    recurrence gives every second state, and one step the others."""
    rows = a.shape[0]
    if rows <= 1:
        return b
    even = rows // 2 * 2
    a0, a1 = a[0:even:2], a[1::2]
    odd = _scan(a1 * a0, a1 * b[0:even:2] + b[1::2])
    h = torch.empty_like(b)
    h[0], h[1::2] = b[0], odd
    h[2::2] = a[2::2] * odd[:(rows - 1) // 2] + b[2::2]
    return h


def _gates(case, g):
    """(decay, factor of the input) in fp32; the factor is None where it is one."""
    g = g.float()
    if case["gate"] == "log":
        return torch.exp(g), None
    if case["gate"] == "alpha":
        return g, None
    return 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))


def _rec_fwd(s):
    case, x = s["case"], s["x"]
    a, f = _gates(case, s["g"])
    b = x.float() if f is None else f * x.float()
    a, b = a.clone(), b.clone()
    if s["init"] is not None:
        b[s["first"]] += a[s["first"]] * s["init"][s["seq"]]
    a[s["first"]] = 0.0
    h = _scan(a, b)
    n = s["cu"].numel() - 1
    fin = s["init"].clone() if s["init"] is not None else torch.zeros((n, x.shape[1]), device=x.device)
    fin[s["seq"]] = h[s["last"]]
    return h.to(x.dtype), fin


def _rec_bwd(s):
    case, dout = s["case"], s["dout"].float()
    h = s["codes"].float() * _spread(s["scales"], s["codes"].shape) if case["q8"] else s["h"]
    h = h.float().view(dout.shape)
    a, f = _gates(case, s["g"])
    carry, b = a.clone(), a * dout
    if s["dfin"] is not None:
        b[s["last"]] += a[s["last"]] * s["dfin"][s["seq"]]
    carry[s["last"]] = 0.0
    e = _scan(carry.flip(0), b.flip(0)).flip(0)  # a_t times the gradient of h_t
    nxt = torch.cat([e[1:], torch.zeros_like(e[:1])])
    nxt[s["last"]] = s["dfin"][s["seq"]] if s["dfin"] is not None else 0.0
    d = dout + nxt
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[s["first"]] = s["init"][s["seq"]] if s["init"] is not None else 0.0
    if case["gate"] == "log":
        dx, dg = d, e * prev
    elif case["gate"] == "alpha":
        dx, dg = d, d * prev
    else:
        dx, dg = f * d, f * e * (prev - s["x"].float())
    dinit = None
    if s["init"] is not None:
        dinit = s["dfin"].clone()
        dinit[s["seq"]] = e[s["first"]]
    return dx.to(TYPES[case["xt"]]), dg.to(TYPES[case["gt"]]), dinit


def _step(s):
    a, f = _gates(s["case"], s["g"])
    b = s["x"].float() if f is None else f * s["x"].float()
    keep = (s["slot"] >= 0).float()[:, None]
    h = a * (keep * s["cache"][s["slot"].clamp(min=0).long()]) + b
    s["cache"][s["live_slot"]] = h[s["live"]]
    return h.to(s["x"].dtype), s["cache"]


def _blocks(x):
    """[T, H, D] -> [T, H, blocks, 128], the last block filled up with zeros."""
    d = x.shape[-1]
    pad = -d % 128
    return torch.nn.functional.pad(x, (0, pad)).view(*x.shape[:-1], (d + pad) // 128, 128)


def _spread(scales, shape):
    return scales[..., None].expand(*scales.shape, 128).reshape(*scales.shape[:-1], -1)[..., :shape[-1]]


def _quantize(x):
    """8-bit codes of fp32 values in blocks of 128 channels, and each block's scale.  The inverse scale is
    127 / amax cut to four significant bits, so that its product with a 16-bit value is exact."""
    amax = _blocks(x).abs().amax(-1)
    inv = ((127.0 / amax.clamp(min=2.0 ** -100)).view(torch.int32) & -0x100000).view(torch.float32)
    inv = torch.where(amax < 2.0 ** -100, torch.zeros_like(inv), inv)
    scales = torch.where(inv > 0, 1.0 / inv, torch.zeros_like(inv))
    return torch.round(x * _spread(inv, x.shape)).to(torch.int8), scales


def _normed(case, o):
    m = o.mean(-1, keepdim=True) if case["center"] else 0.0
    r = torch.rsqrt((o - m).square().mean(-1, keepdim=True) + EPS)
    return (o - m) * r, r


def _norm(s, o, z):
    case = s["case"]
    u = _normed(case, o)[0] * s["w"]
    if s["b"] is not None:
        u = u + s["b"]
    t = u if z is None else z
    q = 1.0 / (1.0 + torch.exp(-t))
    return u * (q if case["act"] == "sigmoid" or z is None else t * q)


def _norm_bwd(s, o, z, dy):
    case = s["case"]
    n, r = _normed(case, o)
    u = n * s["w"]
    if s["b"] is not None:
        u = u + s["b"]
    t = u if z is None else z
    q = 1.0 / (1.0 + torch.exp(-t))
    silu = case["act"] == "silu"
    slope = q * (1.0 + t * (1.0 - q)) if silu else q * (1.0 - q)
    if z is None:
        du, dz = dy * slope, None
    else:
        du, dz = dy * (t * q if silu else q), dy * u * slope
    over = (0,) if case["per_head"] else (0, 1)
    dw = (du * n).sum(over)
    db = du.sum(over) if s["b"] is not None else None
    dn = du * s["w"]
    do = dn - n * (dn * n).mean(-1, keepdim=True)
    if case["center"]:
        do = do - dn.mean(-1, keepdim=True)
    return do * r, dz, dw, db


def _norm_train(s):
    o, z = s["o"].float(), s["z"].float() if s["z"] is not None else None
    y = _norm(s, o, z)
    codes, scales = _quantize(o)
    o = codes.float() * _spread(scales, codes.shape)
    if z is not None:
        codes, scales = _quantize(z)
        z = codes.float() * _spread(scales, codes.shape)
    do, dz, dw, db = _norm_bwd(s, o, z, s["dy"].float())
    t = s["o"].dtype
    return {"y": y.to(t), "do": do.to(t), "dz": dz.to(t) if dz is not None else None, "dw": dw, "db": db}


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        return _run_own(s, case, kind)
    if kind == "rec_fwd":
        h, fin = _rec_fwd(s)
        return {"h": h, "final": fin}
    if kind == "rec_bwd":
        dx, dg, dinit = _rec_bwd(s)
        return {"dx": dx, "dg": dg, "dinit": dinit}
    if kind == "step":
        h, cache = _step(s)
        return {"h": h, "cache": cache}
    if kind == "norm":
        y = _norm(s, s["o"].float(), s["z"].float() if s["z"] is not None else None)
        return {"y": y.to(s["o"].dtype)}
    return _norm_train(s)


def _run_own(s, case, kind):
    import chunked_gated_deltaproduct_gb300 as gdp
    if kind == "rec_fwd":
        h, fin = gdp.gated_linear_recurrence(s["x"], s["g"], s["cu"], gate=case["gate"], initial_state=s["init"],
                                             output_final_state=True)
        return {"h": h, "final": fin}
    if kind == "rec_bwd":
        h = gdp.ActivationCheckpoint(s["codes"], s["scales"]) if case["q8"] else s["h"]
        d = gdp.gated_linear_recurrence_backward(s["g"], h, s["dout"], s["cu"], gate=case["gate"], x=s.get("x"),
                                                 initial_state=s["init"], d_final_state=s["dfin"])
        return {"dx": d["dx"], "dg": d["dg"], "dinit": d["d_initial_state"]}
    if kind == "step":
        h = gdp.gated_linear_recurrence_decode(s["x"], s["g"], gate=case["gate"], state=s["cache"],
                                               state_indices=s["slot"])
        return {"h": h, "cache": s["cache"]}
    how = {"eps": EPS, "center": case["center"], "activation": case["act"]}
    if kind == "norm":
        return {"y": gdp.gated_group_norm(s["o"], s["w"], s["z"], s["b"], **how)}
    y, saved = gdp.gated_group_norm(s["o"], s["w"], s["z"], s["b"], save_checkpoint=True, **how)
    d = gdp.gated_group_norm_backward(s["dy"], saved, s["w"], s["b"], **how)
    return {"y": y, "do": d["do"], "dz": d["dz"], "dw": d["dweight"], "db": d["dbias"]}


# ---- work and the 64-bit values ----------------------------------------------------------------------

def work(case):
    """Bytes: each call's inputs read once and its outputs written once (a training step of the norm is two
    calls: the checkpoint is an output of the first and an input of the second).  flops: the formulas' own."""
    kind = case["kind"]
    if kind in ("rec_fwd", "rec_bwd"):
        n = [int(v) for v in case["lengths"].split(",")]
        e, st = sum(n) * case["C"], len(n) * case["C"] * 4
        x, g = SIZE[case["xt"]], SIZE[case["gt"]]
        if kind == "rec_fwd":
            return {"bytes": e * (2 * x + g) + st * (2 if case["init"] else 1), "flops": 4 * e}
        h = 1 + 4 / 128 if case["q8"] else x
        more = x if case["gate"] == "sigmoid" else 0
        return {"bytes": e * (2 * x + 2 * g + h + more) + st * (3 if case["init"] else 0), "flops": 8 * e}
    if kind == "step":
        e, live = case["N"] * case["C"], (case["N"] - case["padding"]) * case["C"]
        return {"bytes": e * (2 * SIZE[case["xt"]] + SIZE[case["gt"]]) + 8 * live, "flops": 4 * e}
    e, x, ins = case["T"] * case["H"] * case["D"], SIZE[case["type"]], 2 if case["gated"] else 1
    par = (case["H"] if case["per_head"] else 1) * case["D"] * 4 * (2 if case["bias"] else 1)
    if kind == "norm":
        return {"bytes": e * x * (ins + 1) + par, "flops": 12 * e}
    kept = ins * (e + 4 * case["T"] * case["H"] * math.ceil(case["D"] / 128))
    return {"bytes": e * x * (ins + 1) + kept + kept + e * x * (1 + ins) + 3 * par, "flops": 40 * e}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("rec_fwd", "rec_bwd"):
        return _exact_rec(case, s)
    if kind == "step":
        a, b = _exact_gate(case, s["g"], s["x"])
        cache = s["cache"].double()
        h = torch.zeros_like(b)
        for i, slot in enumerate(s["slot"].tolist()):
            h[i] = b[i] if slot < 0 else a[i] * cache[slot] + b[i]
            if slot >= 0:
                cache[slot] = h[i]
        return {"h": h, "cache": cache}
    o = s["o"].double()
    z = s["z"].double() if s["z"] is not None else None
    w, bias = s["w"].double().requires_grad_(), s["b"].double().requires_grad_() if s["b"] is not None else None
    with torch.no_grad():
        y = _exact_norm(case, o, w, bias, z)
    if kind == "norm":
        return {"y": y}
    o, z = (None if v is None else _exact_kept(v).requires_grad_() for v in (o, z))
    leaves = [v for v in (o, z, w, bias) if v is not None]
    got = iter(torch.autograd.grad(_exact_norm(case, o, w, bias, z), leaves, s["dy"].double()))
    do, dz, dw, db = (None if v is None else next(got) for v in (o, z, w, bias))
    return {"y": y, "do": do, "dz": dz, "dw": dw, "db": db}


def _exact_gate(case, g, x):
    g = g.double()
    a = {"log": torch.exp, "alpha": lambda v: v, "sigmoid": torch.sigmoid}[case["gate"]](g)
    x = x.double() if x is not None else None
    return a, x if case["gate"] != "sigmoid" or x is None else (1.0 - a) * x


def _exact_rec(case, s):
    """Token by token, all sequences side by side (longest first, so that the running ones are a prefix)."""
    lengths = [int(v) for v in case["lengths"].split(",")]
    order = sorted(range(len(lengths)), key=lambda i: -lengths[i])
    start = s["cu"].long()[torch.tensor(order, device="cuda")]
    order_dev = torch.tensor(order, device="cuda")
    running = [sum(n > t for n in lengths) for t in range(max(lengths))]
    a, b = _exact_gate(case, s["g"], s.get("x"))
    n, c = len(lengths), case["C"]
    init = s["init"].double() if s["init"] is not None else torch.zeros((n, c), dtype=torch.float64, device="cuda")
    if case["kind"] == "rec_fwd":
        state, h = init[order_dev], torch.empty_like(b)
        for t, k in enumerate(running):
            rows = start[:k] + t
            state[:k] = a[rows] * state[:k] + b[rows]
            h[rows] = state[:k]
        final = torch.empty_like(state)
        final[order_dev] = state
        return {"h": h, "final": final}
    dout = s["dout"].double()
    if case["q8"]:
        d = s["codes"].shape[-1]
        which = torch.arange(d, device="cuda") // 128
        h = (s["codes"].double() * s["scales"].double()[..., which]).view(dout.shape)
    else:
        h = s["h"].double()
    back = s["dfin"].double()[order_dev] if s["dfin"] is not None else torch.zeros_like(init)
    dx, dg = torch.empty_like(dout), torch.empty_like(dout)
    for t in reversed(range(len(running))):
        k = running[t]
        rows = start[:k] + t
        prev = h[rows - 1] if t > 0 else init[order_dev[:k]]
        d, at = dout[rows] + back[:k], a[rows]
        if case["gate"] == "log":
            dx[rows], dg[rows] = d, d * prev * at
        elif case["gate"] == "alpha":
            dx[rows], dg[rows] = d, d * prev
        else:
            dx[rows], dg[rows] = d * (1.0 - at), d * (prev - s["x"][rows].double()) * at * (1.0 - at)
        back[:k] = d * at
    dinit = None
    if s["init"] is not None:
        dinit = torch.empty_like(back)
        dinit[order_dev] = back
    return {"dx": dx, "dg": dg, "dinit": dinit}


def _exact_norm(case, o, w, bias, z):
    if case["center"]:
        o = o - o.mean(-1, keepdim=True)
    u = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * w
    if bias is not None:
        u = u + bias
    if z is None:
        return u * torch.sigmoid(u)
    return u * torch.sigmoid(z) * (z if case["act"] == "silu" else 1.0)


def _exact_kept(v):
    """The values that the 8-bit codes of v stand for."""
    out = torch.zeros_like(v)
    for lo in range(0, v.shape[-1], 128):
        part = v[..., lo:lo + 128]
        mant, expo = torch.frexp(127.0 / part.abs().amax(-1, keepdim=True))
        inv = torch.ldexp(torch.floor(mant * 16.0), expo - 4)
        out[..., lo:lo + 128] = torch.round(part * inv) / inv
    return out.detach()
