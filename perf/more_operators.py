"""Measured cases of a recurrent block's other operators: the short causal convolution (packed sequences, a
training step, one token), the selective state space scan (the same three) and the residual norm (the norms behind
one block and before the next in one pass; a training step of it).

``own`` selects what ``run`` calls: the plain form below (elementary torch operations in fp32, sums over many rows in
fp64, rounded once at the end) or the framework's operators.  ``exact`` computes the same outputs in 64 bits.

Convolution, per channel along a packed sequence:  p_t = b + sum_j w_j x_{t-W+1+j},  y_t = p_t or silu(p_t).
Scan, per channel c and state s:  e_t = softplus(dt_t + bias) (or dt_t + bias),  h_t = exp(e_t A) h_{t-1} + e_t x_t B_t,
y_t = (sum_s C_t h_t + D x_t) silu(z_t);  B and C are shared by the channels of a group.
Residual norm over the channels of a token:  r = residual + scale act(gate) (block / rms(block) post),
y = r / rms(r) weight.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MOST = 65536 * 4096  # elements of the largest case
MOST_STATES = MOST * 16  # tokens x channels x states of the largest scan
MOST_TRAINED = 32768 * 2048 * 16  # of the largest training step of the scan


def _batching():
    """64 lengths, log-uniform in [16, 8192], one of them replaced by an empty request."""
    import random
    r = random.Random(1005)
    n = [int(math.exp(r.uniform(math.log(16), math.log(8192)))) for _ in range(64)]
    n[17] = 0
    return ",".join(map(str, n))


def listed():
    return [
        # a small packed batch with ragged lengths behind earlier tokens: the latency of a short prefill
        {"name": "conv_ragged", "kind": "conv", "lengths": "100,257,64,1000", "C": 1024, "W": 4, "act": "silu",
         "bias": True, "init": True, "cache": False, "xt": "bf16", "fused": True},
        # training on one long sequence, the full width: forward and gradients
        {"name": "conv_train_long", "kind": "conv_train", "lengths": "65536", "C": 4096, "W": 4, "act": "silu",
         "bias": True, "init": False, "xt": "bf16", "fused": False},
        # a serving step over the convolution's cache, some requests of the captured batch size padding
        {"name": "conv_step", "kind": "conv_step", "N": 64, "C": 4096, "W": 4, "act": "silu", "bias": True,
         "slots": 128, "padding": 8, "xt": "bf16"},
        # the ragged batch through the scan, entering states given, not gated
        {"name": "scan_ragged", "kind": "scan", "lengths": "100,257,64,1000", "C": 1024, "S": 16, "G": 1,
         "softplus": True, "gated": False, "init": True, "cache": False, "xt": "bf16", "dtt": "f32", "fused": False},
        # the long-context prefill at full width, gated; B and C are slices of one projection
        {"name": "scan_long", "kind": "scan", "lengths": "65536", "C": 4096, "S": 16, "G": 1, "softplus": True,
         "gated": True, "init": False, "cache": False, "xt": "bf16", "dtt": "bf16", "fused": True},
        # dynamic batching: 64 requests of very different lengths over the state cache
        {"name": "scan_batching", "kind": "scan", "lengths": _batching(), "C": 2048, "S": 16, "G": 1,
         "softplus": True, "gated": True, "init": True, "cache": True, "xt": "bf16", "dtt": "bf16", "fused": True},
        # a training batch: forward, and the gradients of every input
        {"name": "scan_train_batch", "kind": "scan_train", "lengths": ",".join(["4096"] * 8), "C": 2048, "S": 16,
         "G": 1, "softplus": True, "gated": True, "init": False, "xt": "bf16", "dtt": "bf16", "fused": True},
        # fine-tuning on a few short sequences: two groups of B and C, twice the states, learned entering states
        {"name": "scan_train_ragged", "kind": "scan_train", "lengths": "100,257,64,1000", "C": 512, "S": 32, "G": 2,
         "softplus": True, "gated": False, "init": True, "xt": "f32", "dtt": "f32", "fused": False},
        # a serving step over the state cache
        {"name": "scan_step", "kind": "scan_step", "N": 64, "C": 4096, "S": 16, "G": 1, "softplus": True,
         "gated": True, "slots": 128, "padding": 8, "xt": "bf16", "dtt": "bf16"},
        # between two blocks of a serving step
        {"name": "norm_serving", "kind": "norm", "T": 64, "C": 2048, "post": True, "gate": "sigmoid", "scale": True,
         "type": "bf16", "rt": "bf16", "fused": True},
        # a prefill's rows, an odd width, no gate
        {"name": "norm_ragged", "kind": "norm", "T": 1421, "C": 1601, "post": True, "gate": "", "scale": False,
         "type": "f16", "rt": "f32", "fused": False},
        # a training step between two blocks over the long sequence, the residual stream in fp32
        {"name": "norm_train_long", "kind": "norm_train", "T": 65536, "C": 4096, "post": True, "gate": "sigmoid",
         "scale": True, "type": "bf16", "rt": "f32", "fused": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A channel count over [lo, hi]: half of them multiples of 64, the others as they fall (odd ones too)."""
    c = _log_int(rng, lo, hi)
    return max(lo, c // 64 * 64) if rng.random() < 0.5 and c >= 64 else c


def _lengths(rng, most):
    total = _log_int(rng, 1, max(1, most))
    n = _log_int(rng, 1, 64)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if n > 2 and rng.random() < 0.3:
        lengths[lengths.index(min(lengths))] = 0
    return ",".join(map(str, lengths))


def draw(rng):
    kind = rng.choice(["conv", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_train", "scan_step", "norm",
                       "norm_train"])
    xt = rng.choice(["bf16", "bf16", "f16", "f32"])
    half = 2 if xt == "f32" else 1
    if kind.startswith("conv"):
        c = _width(rng, 16, 4096)
        case = {"kind": kind, "C": c, "W": rng.choice([2, 3, 4, 4]), "act": rng.choice(["silu", "silu", ""]),
                "bias": rng.random() < 0.6, "xt": xt}
        if kind == "conv_step":
            n = _log_int(rng, 1, 512)
            return {**case, "N": n, "slots": n + rng.randint(0, 64), "padding": rng.randint(0, n // 4)}
        case.update(lengths=_lengths(rng, 65536 // half), init=rng.random() < 0.5, fused=rng.random() < 0.5)
        if kind == "conv":
            case["cache"] = rng.random() < 0.4
        return case
    if kind.startswith("scan"):
        s = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
        g = rng.choice([1, 1, 1, 2, 4])
        c = max(1, _width(rng, 16, 4096) // g) * g
        case = {"kind": kind, "C": c, "S": s, "G": g, "softplus": rng.random() < 0.8, "gated": rng.random() < 0.6, "xt": xt,
                "dtt": rng.choice([xt, "f32"])}
        if kind == "scan_step":
            n = _log_int(rng, 1, 512)
            return {**case, "N": n, "slots": n + rng.randint(0, 64), "padding": rng.randint(0, n // 4)}
        most = (MOST_STATES if kind == "scan" else MOST_TRAINED) // (c * s) // half
        case.update(lengths=_lengths(rng, min(65536 if kind == "scan" else 32768, most)), init=rng.random() < 0.5,
                    fused=rng.random() < 0.5)
        if kind == "scan":
            case["cache"] = rng.random() < 0.4
        return case
    c = _width(rng, 16, 8192)
    return {"kind": kind, "T": _log_int(rng, 1, min(65536, MOST // c) // half), "C": c, "post": rng.random() < 0.7,
            "gate": rng.choice(["sigmoid", "silu", "plain", ""]), "scale": rng.random() < 0.6, "type": xt,
            "rt": rng.choice([xt, "f32"]), "fused": rng.random() < 0.5}


# ---- inputs ------------------------------------------------------------------------------------------

def _packed(case):
    """cu_seqlens and the host's view of it: every row's sequence and position, first and last rows of the
    non-empty sequences, their numbers."""
    lengths = torch.tensor([int(n) for n in case["lengths"].split(",")], dtype=torch.int64)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(len(lengths)), lengths)
    full = (lengths > 0).nonzero()[:, 0]
    host = {"cu": cu.to(torch.int32), "row_seq": seq, "row_pos": torch.arange(int(cu[-1])) - cu[seq], "lengths": lengths,
            "first": cu[full], "last": cu[full + 1] - 1, "seq": full}
    return len(lengths), int(cu[-1]), {k: v.to("cuda") for k, v in host.items()}


def _slots(case, gen):
    n = case["N"]
    slot = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
    slot[torch.randperm(n, generator=gen, device="cuda")[:case["padding"]]] = -1
    live = (slot >= 0).nonzero()[:, 0]
    return {"slot": slot, "live": live, "live_slot": slot[live].long()}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]

    def normal(shape, dtype=torch.float32, sigma=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)

    def slices(rows, widths, dtype, fused):
        """Tensors [rows, width]: each its own, or all of them slices of one projection's rows."""
        if not fused:
            return [normal((rows, w), dtype) for w in widths]
        parts = normal((rows, sum(widths)), dtype).split(widths, 1)
        return list(parts)

    s = {"case": case}
    if kind in ("norm", "norm_train"):
        t, c, xt, rt = case["T"], case["C"], TYPES[case["type"]], TYPES[case["rt"]]
        block, gate = slices(t, [c, c], xt, case["fused"])
        s.update(residual=normal((t, c), rt), block=block, gate=gate if case["gate"] else None,
                 weight=1.0 + normal((c,), sigma=0.1), post=1.0 + normal((c,), sigma=0.1) if case["post"] else None,
                 scale=0.5 + normal((c,), sigma=0.1) if case["scale"] else None)
        if kind == "norm_train":
            s.update(dy=normal((t, c), xt), dr=normal((t, c), rt))
        return s
    c, xt = case["C"], TYPES[case["xt"]]
    step = kind.endswith("step")
    if step:
        n, rows = case["N"], case["N"]
        s.update(_slots(case, gen))
        slots = case["slots"]
    else:
        n, rows, dev = _packed(case)
        s.update(dev)
        slots = n + 3
        if case.get("cache"):
            s["slot"] = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
            s["live"], s["live_slot"] = torch.arange(n, device="cuda"), s["slot"].long()
    in_cache = step or case.get("cache")
    if kind.startswith("conv"):
        k = case["W"] - 1
        s["x"] = slices(rows, [c, c], xt, case.get("fused"))[0]
        s["w"] = normal((c, case["W"]), sigma=0.5)
        s["b"] = normal((c,), sigma=0.1) if case["bias"] else None
        state, state_type = (k, c), xt
        if kind == "conv_train":
            s.update(dy=normal((rows, c), xt), dfin=normal((n, k, c), xt) if case["init"] else None)
    else:
        S, g = case["S"], case["G"]
        bc = slices(rows, [g * S, g * S], xt, case.get("fused"))
        xz = slices(rows, [c, c], xt, case.get("fused"))
        # steps as such layers have them: softplus(bias) log-uniform in [0.001, 0.1], decays from the slowest state
        # (about exp(-step)) to the fastest (exp(-S step))
        start = torch.exp(torch.rand((c,), generator=gen, device="cuda") * math.log(100.0) + math.log(0.001))
        dt = normal((rows, c), sigma=0.5)
        if not case["softplus"]:
            dt = start * torch.exp(dt)
        s.update(x=xz[0], z=xz[1] if case["gated"] else None, dt=dt.to(TYPES[case["dtt"]]),
                 B=bc[0].view(rows, g, S), C=bc[1].view(rows, g, S),
                 A=-(torch.arange(1, S + 1, device="cuda") * torch.exp(normal((c, S), sigma=0.1))),
                 D=1.0 + normal((c,), sigma=0.1),
                 bias=start + torch.log(-torch.expm1(-start)) if case["softplus"] else None)
        state, state_type = (c, S), torch.float32
        if kind == "scan_train":
            s.update(dy=normal((rows, c), xt), dfin=normal((n, *state), sigma=0.5) if case["init"] else None)
    s["cache"] = normal((slots, *state), state_type, 0.5) if in_cache else None
    s["init"] = normal((n, *state), state_type, 0.5) if not in_cache and case["init"] else None
    return s


# ---- plain forms -------------------------------------------------------------------------------------

def _entering(s, n):
    """Entering states of the sequences in fp32, zero where there are none."""
    if s["cache"] is None:
        return None if s["init"] is None else s["init"].float()
    keep = (s["slot"] >= 0).float().view(-1, *[1] * (s["cache"].dim() - 1))
    return keep * s["cache"][s["slot"].clamp(min=0).long()].float()


def _leave(s, final):
    """Final states into the cache, or as they are."""
    if s["cache"] is None:
        return final
    s["cache"][s["live_slot"]] = final[s["live"]].to(s["cache"].dtype)
    return s["cache"]


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _lagged(s, x, enter, lag, k):
    """x_{t-lag} of every row, from the entering state [N, k, C] before a sequence's first token."""
    out = torch.zeros_like(x)
    out[lag:] = x[:x.shape[0] - lag]
    before = (s["row_pos"] < lag).nonzero()[:, 0]
    out[before] = enter[s["row_seq"][before], k + s["row_pos"][before] - lag] if enter is not None else 0.0
    return out


def _conv(s):
    case, w = s["case"], s["w"]
    x, k = s["x"].float(), case["W"] - 1
    n = s["cu"].numel() - 1
    enter = _entering(s, n)
    p = w[:, k] * x
    for lag in range(1, k + 1):
        p = p + w[:, k - lag] * _lagged(s, x, enter, lag, k)
    if s["b"] is not None:
        p = p + s["b"]
    # the last k inputs of every sequence, entering ones among them where it is shorter
    at = s["lengths"][:, None] - k + torch.arange(k, device=x.device)
    rows = (s["cu"][:-1].long()[:, None] + at).clamp(min=0, max=max(0, x.shape[0] - 1))
    final = x[rows] if x.shape[0] > 0 else torch.zeros((n, k, x.shape[1]), device=x.device)
    old = torch.zeros_like(final)
    if enter is not None:
        old = torch.gather(enter, 1, (at + k).clamp(max=k - 1)[:, :, None].expand_as(final))
    return p, torch.where((at >= 0)[:, :, None], final, old), enter


def _act(p, act):
    return p * _sigmoid(p) if act == "silu" else p


def _conv_train(s):
    case, w = s["case"], s["w"]
    k, x = case["W"] - 1, s["x"].float()
    p, final, enter = _conv(s)
    y = _act(p, case["act"]).to(s["x"].dtype)
    dp = s["dy"].float()
    if case["act"] == "silu":
        q = _sigmoid(p)
        dp = dp * (q * (1.0 + p * (1.0 - q)))
    del p
    dx, dw = w[:, k] * dp, [(dp * x).sum(0, dtype=torch.float64)]
    n = s["cu"].numel() - 1
    dinit = torch.zeros((n, k, x.shape[1]), device=x.device) if s["init"] is not None else None
    pos, seq = s["row_pos"], s["row_seq"]
    for lag in range(1, k + 1):
        dw.insert(0, (dp * _lagged(s, x, enter, lag, k)).sum(0, dtype=torch.float64))
        g = w[:, k - lag] * dp
        within = (pos >= lag).nonzero()[:, 0]
        dx[within - lag] += g[within]
        if dinit is not None:
            before = (pos < lag).nonzero()[:, 0]
            dinit.index_put_((seq[before], k + pos[before] - lag), g[before], accumulate=True)
    if s["dfin"] is not None:
        at = s["lengths"][:, None] - k + torch.arange(k, device=x.device)
        i, j = (at >= 0).nonzero(as_tuple=True)
        dx.index_put_((s["cu"][i].long() + at[i, j],), s["dfin"][i, j].float(), accumulate=True)
        i, j = (at < 0).nonzero(as_tuple=True)
        dinit.index_put_((i, at[i, j] + k), s["dfin"][i, j].float(), accumulate=True)
    t = s["x"].dtype
    return {"y": y, "final": final.to(t) if s["init"] is not None else None, "dx": dx.to(t), "dw": torch.stack(dw, 1).float(),
            "db": dp.sum(0, dtype=torch.float64).float() if s["b"] is not None else None,
            "dinit": dinit.to(t) if dinit is not None else None}


def _conv_step(s):
    case, w, x = s["case"], s["w"], s["x"].float()
    k = case["W"] - 1
    window = torch.cat([_entering(s, x.shape[0]), x[:, None]], 1)
    p = (window * w.t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"]
    return {"y": _act(p, case["act"]).to(s["x"].dtype), "state": _leave(s, window[:, 1:])}


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


def _deltas(s):
    v = s["dt"].float()
    if s["bias"] is not None:
        v = v + s["bias"]
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs())) if s["case"]["softplus"] else v


def _blocks(case, rows):
    """Channel blocks within a group whose [rows, channels, S] tensors take about a GiB."""
    per, c = case["C"] // case["G"], case["C"]
    width = max(1, min(per, 2 ** 28 // max(1, rows * case["S"])))
    return [(g, g * per + i, min(g * per + i + width, (g + 1) * per)) for g in range(case["G"]) for i in range(0, per, width)]


def _scan_fwd(s):
    case, x, e = s["case"], s["x"].float(), _deltas(s)
    rows, n = x.shape[0], s["cu"].numel() - 1
    enter = _entering(s, n)
    final = enter.clone() if enter is not None else torch.zeros((n, case["C"], case["S"]), device=x.device)
    y = torch.empty_like(x)
    for g, lo, hi in _blocks(case, rows):
        a, h = _states(s, e, x, enter, g, lo, hi)
        final[s["seq"], lo:hi] = h[s["last"]]
        y[:, lo:hi] = (h * s["C"][:, g, None].float()).sum(-1)
    y += s["D"] * x
    return y, final, e


def _states(s, e, x, enter, g, lo, hi):
    """Decays and states [rows, channels, S] of one channel block."""
    a = torch.exp(e[:, lo:hi, None] * s["A"][lo:hi])
    b = (e[:, lo:hi] * x[:, lo:hi])[..., None] * s["B"][:, g, None].float()
    kept = a.clone()
    if enter is not None:
        b[s["first"]] += a[s["first"]] * enter[s["seq"], lo:hi]
    a[s["first"]] = 0.0
    return kept, _scan(a, b)


def _scan_train(s):
    case, x = s["case"], s["x"].float()
    y, final, e = _scan_fwd(s)
    enter, n = _entering(s, s["cu"].numel() - 1), s["cu"].numel() - 1
    dy, t = s["dy"].float(), s["x"].dtype
    out, dz = y, None
    if s["z"] is not None:
        z = s["z"].float()
        q = _sigmoid(z)
        out, dz = y * (z * q), (dy * y * (q * (1.0 + z * (1.0 - q)))).to(t)
        dy = dy * (z * q)
    out = out.to(t)
    du, de = torch.empty_like(x), torch.empty_like(x)
    dA = torch.empty_like(s["A"])
    dB, dC = (torch.zeros(s["B"].shape, dtype=torch.float64, device=x.device) for _ in range(2))
    dinit = s["dfin"].clone() if s["dfin"] is not None else None
    for g, lo, hi in _blocks(case, x.shape[0]):
        a, h = _states(s, e, x, enter, g, lo, hi)
        dC[:, g] += (h * dy[:, lo:hi, None]).sum(1, dtype=torch.float64)
        prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
        prev[s["first"]] = enter[s["seq"], lo:hi] if enter is not None else 0.0
        del h
        grow = dy[:, lo:hi, None] * s["C"][:, g, None].float()
        b, carry = a * grow, a.clone()
        if s["dfin"] is not None:
            b[s["last"]] += a[s["last"]] * s["dfin"][s["seq"], lo:hi]
        carry[s["last"]] = 0.0
        back = _scan(carry.flip(0), b.flip(0)).flip(0)  # a_t times the gradient of h_t
        if dinit is not None:
            dinit[s["seq"], lo:hi] = back[s["first"]]
        prev = prev * back  # gradient of the exponent
        after = torch.cat([back[1:], torch.zeros_like(back[:1])])
        after[s["last"]] = s["dfin"][s["seq"], lo:hi] if s["dfin"] is not None else 0.0
        d = grow + after
        du[:, lo:hi] = (d * s["B"][:, g, None].float()).sum(-1)
        dB[:, g] += (d * (e * x)[:, lo:hi, None]).sum(1, dtype=torch.float64)
        de[:, lo:hi] = (prev * s["A"][lo:hi]).sum(-1)
        dA[lo:hi] = (prev * e[:, lo:hi, None]).sum(0, dtype=torch.float64).float()
    dx, de = du * e + dy * s["D"], de + du * x
    if case["softplus"]:
        de = de * _sigmoid(s["dt"].float() + (s["bias"] if s["bias"] is not None else 0.0))
    return {"y": out, "final": final if s["init"] is not None else None, "dx": dx.to(t), "ddt": de.to(s["dt"].dtype), "dA": dA,
            "dB": dB.to(t), "dC": dC.to(t), "dD": (dy * x).sum(0, dtype=torch.float64).float(), "dz": dz,
            "dbias": de.sum(0, dtype=torch.float64).float() if s["bias"] is not None else None, "dinit": dinit}


def _scan_step(s):
    x, e = s["x"].float(), _deltas(s)
    per = s["case"]["C"] // s["case"]["G"]
    B, C = (v.float().repeat_interleave(per, 1) for v in (s["B"], s["C"]))
    h = torch.exp(e[..., None] * s["A"]) * _entering(s, x.shape[0]) + (e * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _act(s["z"].float(), "silu")
    return {"y": y.to(s["x"].dtype), "state": _leave(s, h)}


def _gate(case, gate):
    """act(gate) and its slope."""
    if gate is None:
        return 1.0, None
    v = gate.float()
    if case["gate"] == "plain":
        return v, 1.0
    q = _sigmoid(v)
    return (q, q * (1.0 - q)) if case["gate"] == "sigmoid" else (v * q, q * (1.0 + v * (1.0 - q)))


def _unit(v):
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r, r


def _norm(s):
    m = s["block"].float()
    if s["post"] is not None:
        m = _unit(m)[0] * s["post"]
    m = m * _gate(s["case"], s["gate"])[0]
    if s["scale"] is not None:
        m = m * s["scale"]
    r = s["residual"].float() + m
    return _unit(r)[0] * s["weight"], r


def _unit_grad(dn, n, r):
    return (dn - n * (dn * n).mean(-1, keepdim=True)) * r


def _norm_train(s):
    t, rt, case = s["block"].dtype, s["residual"].dtype, s["case"]
    y, r = _norm(s)
    y, kept = y.to(t), r.to(rt)
    r = kept.float()
    dy = s["dy"].float()
    n, inv = _unit(r)
    dweight = (dy * n).sum(0, dtype=torch.float64).float()
    dr = s["dr"].float() + _unit_grad(dy * s["weight"], n, inv)
    del n, r
    block = s["block"].float()
    b, inv = _unit(block) if s["post"] is not None else (block, None)
    m = b if s["post"] is None else b * s["post"]
    act, slope = _gate(case, s["gate"])
    scale = 1.0 if s["scale"] is None else s["scale"]
    dscale = (dr * m * act).sum(0, dtype=torch.float64).float() if s["scale"] is not None else None
    dgate = (dr * scale * m * slope).to(t) if s["gate"] is not None else None
    dm = dr * scale * act
    dpost, dblock = None, dm
    if s["post"] is not None:
        dpost = (dm * b).sum(0, dtype=torch.float64).float()
        dblock = _unit_grad(dm * s["post"], b, inv)
    return {"y": y, "residual": kept, "dresidual": dr.to(rt), "dblock": dblock.to(t), "dgate": dgate, "dweight": dweight,
            "dpost": dpost, "dscale": dscale}


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, s["case"], kind)
    if kind == "conv":
        p, final, _ = _conv(s)
        return {"y": _act(p, s["case"]["act"]).to(s["x"].dtype), "state": _leave(s, final.to(s["x"].dtype))}
    if kind == "scan":
        y, final, _ = _scan_fwd(s)
        if s["z"] is not None:
            y = y * _act(s["z"].float(), "silu")
        return {"y": y.to(s["x"].dtype), "state": _leave(s, final)}
    if kind == "norm":
        y, r = _norm(s)
        return {"y": y.to(s["block"].dtype), "residual": r.to(s["residual"].dtype)}
    return {"conv_train": _conv_train, "conv_step": _conv_step, "scan_train": _scan_train, "scan_step": _scan_step,
            "norm_train": _norm_train}[kind](s)


def _run_own(s, case, kind):
    import chunked_gated_deltaproduct_gb300 as gdp
    if kind in ("norm", "norm_train"):
        how = {"activation": None if case["gate"] in ("plain", "") else case["gate"], "scale": s["scale"], "eps": EPS}
        y, r = gdp.residual_norm(s["residual"], s["block"], s["weight"], s["post"], s["gate"], **how)
        if kind == "norm":
            return {"y": y, "residual": r}
        d = gdp.residual_norm_backward(s["dy"], s["dr"], r, s["block"], s["weight"], s["post"], s["gate"], **how)
        return {"y": y, "residual": r, "dresidual": d["d_residual"], "dblock": d["d_block"], "dgate": d["d_gate"],
                "dweight": d["dweight"], "dpost": d["dpost_weight"], "dscale": d["dscale"]}
    step, train = kind.endswith("step"), kind.endswith("train")
    cached = step or case.get("cache")
    where = {"state": s["cache"], "state_indices": s["slot"]} if cached else {"initial_state": s["init"]}
    if not cached and (not train or s["init"] is not None):
        where["output_final_state"] = True
    if kind.startswith("conv"):
        how = {"bias": s["b"], "activation": case["act"] or None}
        if step:
            return {"y": gdp.short_convolution_decode(s["x"], s["w"], **how, **where), "state": s["cache"]}
        got = gdp.short_convolution(s["x"], s["w"], s["cu"], **how, **where)
        y, final = got if "output_final_state" in where else (got, None)
        if not train:
            return {"y": y, "state": s["cache"] if cached else final}
        d = gdp.short_convolution_backward(s["x"], s["w"], s["dy"], s["cu"], initial_state=s["init"], d_final_state=s["dfin"],
                                           **how)
        return {"y": y, "final": final, "dx": d["dx"], "dw": d["dweight"], "db": d["dbias"], "dinit": d["d_initial_state"]}
    ins = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    how = {"D": s["D"], "z": s["z"], "dt_bias": s["bias"], "dt_softplus": case["softplus"]}
    if step:
        return {"y": gdp.selective_scan_decode(*ins, **how, **where), "state": s["cache"]}
    if not train:
        got = gdp.selective_scan(*ins, s["cu"], **how, **where)
        return {"y": got, "state": s["cache"]} if cached else {"y": got[0], "state": got[1]}
    y, *final, kept = gdp.selective_scan(*ins, s["cu"], save_states=True, **how, **where)
    d = gdp.selective_scan_backward(*ins, s["dy"], s["cu"], kept, d_final_state=s["dfin"],
                                    output_d_initial_state=s["init"] is not None, **how)
    return {"y": y, "final": final[0] if final else None, "dx": d["dx"], "ddt": d["ddt"], "dA": d["dA"], "dB": d["dB"],
            "dC": d["dC"], "dD": d["dD"], "dz": d["dz"], "dbias": d["ddt_bias"], "dinit": d["d_initial_state"]}


# ---- work and the 64-bit values ----------------------------------------------------------------------

def work(case):
    """Bytes: each call's inputs read once and its outputs written once (a training step is two calls; what the
    first one keeps for the second is not counted).  flops: the formulas' own operations, an exponential as one."""
    kind = case["kind"]
    if kind in ("norm", "norm_train"):
        e, x, r = case["T"] * case["C"], SIZE[case["type"]], SIZE[case["rt"]]
        gate = 1 if case["gate"] else 0
        par = case["C"] * 4 * (1 + bool(case["post"]) + bool(case["scale"]))
        fwd = e * (2 * r + x * (2 + gate)) + par
        if kind == "norm":
            return {"bytes": fwd, "flops": 14 * e}
        return {"bytes": fwd + e * (3 * r + x * (3 + 2 * gate)) + 2 * par, "flops": 45 * e}
    step, train = kind.endswith("step"), kind.endswith("train")
    n = [1] * case["N"] if step else [int(v) for v in case["lengths"].split(",")]
    live = len(n) - case["padding"] if step else len(n)
    enters, leaves = step or case["init"] or case.get("cache"), not train or case["init"]
    x, e, c = SIZE[case["xt"]], sum(n) * case["C"], case["C"]
    if kind.startswith("conv"):
        state = live * (case["W"] - 1) * c * x * (bool(enters) + bool(leaves))
        par = c * 4 * (case["W"] + bool(case["bias"]))
        f = (2 * case["W"] + 5) * e
        if train:
            return {"bytes": 5 * e * x + (2 if case["init"] else 1) * state + 3 * par, "flops": f + (4 * case["W"] + 12) * e}
        return {"bytes": 2 * e * x + state + par, "flops": f}
    S, dt = case["S"], SIZE[case["dtt"]]
    z = x if case["gated"] else 0
    state = live * c * S * 4 * (bool(enters) + bool(leaves))
    par = c * 4 * (S + 1 + bool(case["softplus"]))
    bc = 2 * sum(n) * case["G"] * S * x
    if train:
        return {"bytes": e * (2 * x + dt + z) + bc + state + par + e * (3 * x + 2 * dt + 2 * z) + 2 * bc + state + 2 * par,
                "flops": e * (26 * S + 30)}
    return {"bytes": e * (2 * x + dt + z) + bc + state + par, "flops": e * (7 * S + 15)}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm_train"):
        return _exact_norm(case, s)
    if kind == "conv_step":
        return _exact_conv_step(case, s)
    if kind == "scan_step":
        return _exact_scan_step(case, s)
    return _exact_conv(case, s) if kind.startswith("conv") else _exact_scan(case, s)


def _f64(v):
    return None if v is None else v.double()


def _old_states(s, n, shape):
    """Entering states in 64 bits, one request at a time."""
    out = torch.zeros((n, *shape), dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        out = s["init"].double()
    elif s["cache"] is not None:
        for i, slot in enumerate(s["slot"].tolist()):
            if slot >= 0:
                out[i] = s["cache"][slot].double()
    return out


def _new_states(s, final):
    if s["cache"] is None:
        return final
    cache = s["cache"].double()
    for i, slot in enumerate(s["slot"].tolist()):
        if slot >= 0:
            cache[slot] = final[i]
    return cache


def _silu64(v):
    return v * torch.sigmoid(v)


def _exact_conv_step(case, s):
    n, k = case["N"], case["W"] - 1
    old, x, w = _old_states(s, n, (k, case["C"])), s["x"].double(), s["w"].double()
    p = x * w[:, k] + (0.0 if s["b"] is None else s["b"].double())
    for j in range(k):
        p = p + old[:, j] * w[:, j]
    return {"y": _silu64(p) if case["act"] else p, "state": _new_states(s, torch.cat([old[:, 1:], x[:, None]], 1))}


def _exact_conv(case, s):
    """Sequence by sequence, over the entering inputs and the sequence's own as one signal; gradients by autograd."""
    train, k = case["kind"] == "conv_train", case["W"] - 1
    lengths = [int(v) for v in case["lengths"].split(",")]
    old = _old_states(s, len(lengths), (k, case["C"]))
    w, b = s["w"].double().requires_grad_(train), _f64(s["b"])
    if b is not None:
        b.requires_grad_(train)
    ys, finals, dxs, dinits = [], [], [], []
    dw, db, at = torch.zeros_like(w), None if b is None else torch.zeros_like(b), 0
    for i, n in enumerate(lengths):
        signal = torch.cat([old[i], s["x"][at:at + n].double()]).requires_grad_(train)
        p = sum(w[:, j] * signal[j:j + n] for j in range(k + 1))
        p = p if b is None else p + b
        y = _silu64(p) if case["act"] else p
        ys.append(y.detach())
        finals.append(signal[n:].detach())
        if train:
            leaves = [signal, w] + ([b] if b is not None else [])
            loss = (y * s["dy"][at:at + n].double()).sum()
            if s["dfin"] is not None:
                loss = loss + (signal[n:] * s["dfin"][i].double()).sum()
            elif n == 0:
                loss = loss + 0.0 * (signal.sum() + w.sum())
            got = torch.autograd.grad(loss, leaves, allow_unused=True)
            dinits.append(got[0][:k])
            dxs.append(got[0][k:])
            dw = dw + (got[1] if got[1] is not None else 0.0)
            if b is not None:
                db = db + (got[2] if got[2] is not None else 0.0)
        at += n
    y, final = torch.cat(ys), torch.stack(finals)
    if not train:
        return {"y": y, "state": _new_states(s, final)}
    return {"y": y, "final": final if s["init"] is not None else None, "dx": torch.cat(dxs), "dw": dw.detach(), "db": _plain(db),
            "dinit": torch.stack(dinits) if s["init"] is not None else None}


def _plain(v):
    return None if v is None else v.detach()


def _exact_delta(case, s):
    v = s["dt"].double()
    if s["bias"] is not None:
        v = v + s["bias"].double()
    return (torch.logaddexp(v, torch.zeros_like(v)), torch.sigmoid(v)) if case["softplus"] else (v, torch.ones_like(v))


def _exact_scan_step(case, s):
    n, per = case["N"], case["C"] // case["G"]
    e, x = _exact_delta(case, s)[0], s["x"].double()
    group = torch.arange(case["C"], device="cuda") // per
    h = _old_states(s, n, (case["C"], case["S"])) * torch.exp(e[:, :, None] * s["A"].double())
    h = h + s["B"].double()[:, group] * x[:, :, None] * e[:, :, None]
    y = torch.einsum("ncs,ncs->nc", h, s["C"].double()[:, group]) + x * s["D"].double()
    if s["z"] is not None:
        y = y * _silu64(s["z"].double())
    return {"y": y, "state": _new_states(s, h)}


def _exact_scan(case, s):
    """Token by token, all sequences side by side (longest first, so that the running ones are a prefix)."""
    train, C, S, G = case["kind"] == "scan_train", case["C"], case["S"], case["G"]
    lengths = [int(v) for v in case["lengths"].split(",")]
    n, per = len(lengths), C // G
    order = sorted(range(n), key=lambda i: -lengths[i])
    order_dev = torch.tensor(order, device="cuda")
    start = s["cu"].long()[order_dev]
    running = [sum(m > t for m in lengths) for t in range(max(lengths))]
    e, slope = _exact_delta(case, s)
    x, A, D = s["x"].double(), s["A"].double().view(G, per, S), s["D"].double()
    B, Cm = s["B"].double(), s["C"].double()
    enter = _old_states(s, n, (C, S))[order_dev].view(n, G, per, S)
    state, y = enter.clone(), torch.empty_like(x)
    hist = torch.empty((x.shape[0], G, per, S), dtype=torch.float64, device="cuda") if train else None
    for t, k in enumerate(running):
        rows = start[:k] + t
        ev = e[rows].view(k, G, per, 1)
        state[:k] = state[:k] * torch.exp(ev * A) + ev * x[rows].view(k, G, per, 1) * B[rows][:, :, None]
        if train:
            hist[rows] = state[:k]
        y[rows] = torch.matmul(state[:k], Cm[rows][..., None]).reshape(k, C)
    y = y + x * D
    final = torch.empty_like(state)
    final[order_dev] = state
    final = final.view(n, C, S)
    z = _f64(s["z"])
    out = y if z is None else y * _silu64(z)
    if not train:
        return {"y": out, "state": _new_states(s, final)}
    dout, dz, dy = s["dy"].double(), None, s["dy"].double()
    if z is not None:
        q = torch.sigmoid(z)
        dz, dy = dout * y * (q + z * q * (1.0 - q)), dout * z * q
    back = s["dfin"].double()[order_dev].view(n, G, per, S) if s["dfin"] is not None else torch.zeros_like(enter)
    dx, de, dA = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(A)
    dB, dC = torch.empty_like(B), torch.empty_like(Cm)
    for t in reversed(range(len(running))):
        k = running[t]
        rows = start[:k] + t
        g, ev, xv = dy[rows].view(k, G, per, 1), e[rows].view(k, G, per, 1), x[rows].view(k, G, per, 1)
        d = back[:k] + g * Cm[rows][:, :, None]
        dC[rows] = (hist[rows] * g).sum(2)
        dB[rows] = (d * ev * xv).sum(2)
        into = (d * B[rows][:, :, None]).sum(-1, keepdim=True)
        a = torch.exp(ev * A)
        prev = hist[rows - 1] if t > 0 else enter[:k]
        back[:k] = d * a
        expo = back[:k] * prev
        dA += (expo * ev).sum(0)
        dx[rows] = (into * ev).view(k, C) + dy[rows] * D
        de[rows] = ((expo * A).sum(-1, keepdim=True) + into * xv).view(k, C)
    dinit = None
    if s["init"] is not None:
        dinit = torch.empty_like(back)
        dinit[order_dev] = back
        dinit = dinit.view(n, C, S)
    de = de * slope
    return {"y": out, "final": final if s["init"] is not None else None, "dx": dx, "ddt": de, "dA": dA.view(C, S), "dB": dB,
            "dC": dC, "dD": (dy * x).sum(0), "dz": dz, "dbias": de.sum(0) if s["bias"] is not None else None, "dinit": dinit}


def _exact_norm(case, s):
    act = {"sigmoid": torch.sigmoid, "silu": _silu64, "plain": lambda v: v, "": None}[case["gate"]]

    def stream(residual, block, gate, post, scale):
        m = block
        if post is not None:
            m = post * m / torch.sqrt((m * m).sum(-1, keepdim=True) / m.shape[-1] + EPS)
        if gate is not None:
            m = m * act(gate)
        return residual + (m if scale is None else m * scale)

    def normed(r, weight):
        return r / torch.sqrt((r * r).sum(-1, keepdim=True) / r.shape[-1] + EPS) * weight

    ins = [_f64(s[k]) for k in ("residual", "block", "gate", "post", "scale")]
    weight = s["weight"].double()
    r = stream(*ins)
    y = normed(r, weight)
    if case["kind"] == "norm":
        return {"y": y, "residual": r}
    # the backward pass starts from the stream as it was stored
    kept = r.to(s["residual"].dtype).double().requires_grad_()
    weight.requires_grad_()
    dr, dweight = torch.autograd.grad(normed(kept, weight), [kept, weight], s["dy"].double())
    dr = dr + s["dr"].double()
    leaves = [None if v is None else v.requires_grad_() for v in ins[1:]]
    got = iter(torch.autograd.grad(stream(ins[0], *leaves), [v for v in leaves if v is not None], dr))
    dblock, dgate, dpost, dscale = (None if v is None else next(got) for v in leaves)
    return {"y": y, "residual": r, "dresidual": dr, "dblock": dblock, "dgate": dgate, "dweight": dweight, "dpost": dpost,
            "dscale": dscale}
