"""The layer operators' main paths at sizes where their loops go round, against the float64 references:
scans over many steps of a cluster (every ring stage and barrier used again and again), several blocks in a
checkpoint row, groups of the norm with several rows each, heads rounded up to whole CTAs."""
import pytest
import torch

import chunked_gated_deltaproduct_gb300 as pkg
from tests import _layer_ref as R
from tests.test_gpu_layer import _as_laid_out, _cu, _gates, _rand

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# lengths, C, types, gate: clusters of 16 (few channels), 8 and 4 CTAs, each over eight steps and more
LONG = [
    ([9000, 0, 5000, 6001], 256, BF16, BF16, "log"),
    ([700, 1, 8000, 3300], 128, BF16, F32, "sigmoid"),
    ([8192], 2048, BF16, BF16, "sigmoid"),
    ([5000, 3192], 2048, F16, F32, "log"),
    ([4000, 77, 4115], 4096, BF16, BF16, "log"),
    ([6000], 1024, F32, F32, "alpha"),
    ([6000], 200, F32, F32, "log"),
    ([3000, 5000], 1027, BF16, BF16, "log"),  # rows off the 16-byte boundaries
]


@pytest.mark.parametrize("lengths,C,xt,gt,kind", LONG)
def test_recurrence_many_steps(cuda_device, lengths, C, xt, gt, kind):
    T, N, dev = sum(lengths), len(lengths), cuda_device
    x, g, s0 = _rand((T, C), 1, xt), _gates(kind, (T, C), 2, gt), _rand((N, C), 3)
    h, fin = pkg.gated_linear_recurrence(x.to(dev), g.to(dev), _cu(lengths, dev), gate=kind, initial_state=s0.to(dev),
                                         output_final_state=True)
    rh, rfin, eh, efin = R.recurrence(x, g, lengths, kind, s0)
    R.check(h, rh, eh, "h")
    R.check(fin, rfin, efin, "final state")


@pytest.mark.parametrize("saved", ["h", "codes"])
@pytest.mark.parametrize("lengths,C,xt,gt,kind", LONG)
def test_recurrence_backward_many_steps(cuda_device, lengths, C, xt, gt, kind, saved):
    T, N, dev = sum(lengths), len(lengths), cuda_device
    x, h, dh = (_rand((T, C), i, xt) for i in (1, 3, 4))
    g, s0, dfin = _gates(kind, (T, C), 2, gt), _rand((N, C), 5), _rand((N, C), 6)
    if saved == "codes":
        codes, scales, values = R.quantize(h.view(T, 1, C))  # one row of C channels: several blocks of 128
        h_in, href = pkg.ActivationCheckpoint(codes.to(dev), scales.float().to(dev)), values.view(T, C)
    else:
        h_in, href = h.to(dev), h
    got = pkg.gated_linear_recurrence_backward(g.to(dev), h_in, dh.to(dev), _cu(lengths, dev), gate=kind,
                                               x=x.to(dev) if kind == "sigmoid" else None, initial_state=s0.to(dev),
                                               d_final_state=dfin.to(dev))
    dx, dg, dinit, ex, eg, einit = R.recurrence_backward(g, href, dh, lengths, kind, x, s0, dfin)
    R.check(got["dx"], dx, ex, "dx")
    R.check(got["dg"], dg, eg + 2.0 ** -23 * dg.abs(), "dg")
    R.check(got["d_initial_state"], dinit, einit, "d_initial_state")


@pytest.mark.parametrize("C,H", [(384, 2), (400, 2), (640, 5), (260, 1), (2304, 3)])
def test_recurrence_backward_from_rows_of_several_blocks(cuda_device, C, H):
    """Checkpoint rows of 192, 200, 128, 260 and 768 channels: tiles of 64 channels inside one block, or across
    blocks and rows."""
    lengths, dev = [300, 0, 411], cuda_device
    T = sum(lengths)
    h, dh, g = _rand((T, C), 3, BF16), _rand((T, C), 4, BF16), _gates("log", (T, C), 2, BF16)
    codes, scales, values = R.quantize(h.view(T, H, C // H) * torch.logspace(-2, 2, C // H).to(BF16))
    got = pkg.gated_linear_recurrence_backward(
        g.to(dev), pkg.ActivationCheckpoint(codes.to(dev), scales.float().to(dev)), dh.to(dev), _cu(lengths, dev))
    dx, dg, _, ex, eg, _ = R.recurrence_backward(g, values.view(T, C), dh, lengths, "log")
    R.check(got["dx"], dx, ex, "dx")
    R.check(got["dg"], dg, eg + 2.0 ** -23 * dg.abs(), "dg")


# T, H, D, type, gated, activation, centred, bias, per head, layout.  On 152 SMs a row's group of 4, 8, 16 or 32
# lanes, or its CTA, gets three rows and more in the forward pass as in the backward.
MANY = [
    (12000, 8, 64, BF16, True, "silu", False, True, False, "dense"),
    (6000, 8, 128, BF16, True, "silu", False, False, False, "dense"),
    (6000, 7, 128, F16, True, "sigmoid", True, True, True, "slice"),
    (1200, 37, 128, BF16, True, "silu", False, True, True, "dense"),  # heads rounded up to whole CTAs
    (1200, 37, 128, BF16, False, "silu", True, True, False, "dense"),
    (5000, 5, 127, BF16, True, "silu", True, True, False, "odd"),
    (3000, 8, 200, BF16, True, "silu", False, True, True, "dense"),
    (3000, 4, 256, F32, True, "silu", False, False, False, "dense"),
    (5000, 2, 500, F16, False, "silu", True, True, False, "dense"),
    (5000, 2, 512, BF16, True, "sigmoid", True, True, True, "dense"),
    (2500, 3, 321, BF16, True, "silu", False, True, True, "odd"),
    (4000, 1, 1024, BF16, True, "silu", False, True, False, "dense"),
    (4000, 1, 1024, BF16, True, "silu", True, True, False, "slice"),
    (2000, 2, 1001, F16, True, "silu", True, True, True, "odd"),
    (1500, 1, 4096, BF16, True, "silu", True, True, True, "dense"),
    (1500, 1, 4096, F32, False, None, False, False, False, "dense"),
    (1200, 1, 8192, BF16, True, "sigmoid", False, True, False, "dense"),
    (1200, 1, 2501, F32, True, "silu", True, True, False, "odd"),
]


def _inputs(case):
    T, H, D, dt, gated, act, center, bias, per_head, layout = case
    o = _rand((T, H, D), 1, sigma=2.0)
    if center:
        o += 3.0
    o *= torch.logspace(-1, 1, T)[:, None, None]  # every row its own size: a stale row would show
    shape = (H, D) if per_head else (D,)
    return (o.to(dt), _rand((T, H, D), 2, dt, 2.0) if gated else None, 1 + _rand(shape, 3, sigma=0.3),
            _rand(shape, 4, sigma=0.3) if bias else None, _rand((T, H, D), 5, dt))


def _spread(c):
    """The scale of every code, in 64 bits."""
    return c.scales.cpu().double().repeat_interleave(pkg.CHECKPOINT_BLOCK, -1)[..., :c.codes.shape[-1]]


@pytest.mark.parametrize("case", MANY)
def test_group_norm_many_rows(cuda_device, case):
    dev, layout = cuda_device, case[-1]
    o, z, w, b, dy = _inputs(case)
    on = lambda t: None if t is None else t.to(dev)  # noqa: E731
    how = dict(eps=1e-5, center=case[6], activation=case[5])
    od, zd = _as_laid_out(o, layout, dev), None if z is None else _as_laid_out(z, layout, dev)
    y, kept = pkg.gated_group_norm(od, on(w), zd, on(b), save_checkpoint=True, **how)
    R.check(y, *R.group_norm(o, w, z, b, 1e-5, case[6], case[5]), "y")
    for name, c, v in (("o", kept.o, o), ("z", kept.z, z)):
        if v is not None:
            codes, scales, _ = R.quantize(v)
            # an fp32 value times the inverse scale is rounded: a code next to a tie may move
            assert int((c.codes.cpu().int() - codes.int()).abs().max()) <= (0 if v.dtype != F32 else 1), name
            assert torch.equal(c.scales.cpu(), scales.float()), name
    dyd = _as_laid_out(dy, layout, dev)
    for saved in ("tensors", "checkpoint"):
        if saved == "checkpoint":
            o, z = (None if c is None else c.codes.cpu().double() * _spread(c) for c in kept)
        got = pkg.gated_group_norm_backward(dyd, kept if saved == "checkpoint" else (od, zd), on(w), on(b), **how)
        ref = R.group_norm_backward(dy, o, w, z, b, 1e-5, case[6], case[5])
        for name in ("do", "dz", "dweight", "dbias"):
            if got[name] is not None:
                R.check(got[name], *ref[name], f"{name} from {saved}")


def test_group_norm_past_32_bit_offsets(cuda_device):
    """More than 2^31 elements, rows of many places against the reference."""
    dev, D = cuda_device, 128
    T = (1 << 24) + 4099
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    gen = torch.Generator(device=dev).manual_seed(1)
    o, z, dy = (torch.empty((T, 1, D), dtype=BF16, device=dev).normal_(generator=gen) for _ in range(3))
    w = 1 + _rand((D,), 3, sigma=0.3)
    y, kept = pkg.gated_group_norm(o, w.to(dev), z, save_checkpoint=True)
    d = pkg.gated_group_norm_backward(dy, kept, w.to(dev))
    rows = torch.cat([torch.arange(0, 200), torch.arange(T // 2, T // 2 + 200), torch.arange(T - 4400, T)]).to(dev)
    part = lambda t: t[rows].cpu()  # noqa: E731
    R.check(part(y), *R.group_norm(part(o), w, part(z)), "y")
    ko, kz = (part(c.codes).double() * part(c.scales).double() for c in kept)
    ref = R.group_norm_backward(part(dy), ko, w, kz)
    for name in ("do", "dz"):
        R.check(part(d[name]), *ref[name], name)
