"""examples/recurrent_mixer.py: the operators together, as a training step and a serving loop use them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_mixer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("recurrent_mixer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss(cuda_device, example):
    losses = example.train(steps=15)
    assert losses[-1] < 0.8 * losses[0] and all(b < a * 1.02 for a, b in zip(losses, losses[1:]))


def test_serving_equals_one_pass(cuda_device, example):
    got, want = example.serve()
    # both are roundings to bf16 (2^-8 relative) of values of order one, through four rounded stages each
    assert float((got.float() - want.float()).abs().max()) <= 8 * 2.0 ** -8 * max(1.0, float(want.float().abs().max()))


def test_layer_gradient_against_differences(cuda_device, example):
    """The whole layer's gradient along a direction of the gate parameter and of a norm weight against a
    difference of the loss (8-bit checkpoints and bf16 stages: a few per cent)."""
    H, D = 2, 64
    model = example.Mixer(H, D, cuda_device, seed=5)
    batch = example.make_batch([150, 60], H, D, cuda_device, seed=6)
    d_out = torch.randn(210, H, D, generator=torch.Generator().manual_seed(7)).to(cuda_device, torch.bfloat16)
    out, saved = model.forward(*batch)
    grads = model.backward(saved, d_out)

    def loss():
        return float((model.forward(*batch, keep=False)[0].double() * d_out.double()).sum())

    for name, step in (("gate", 0.25), ("w1", 0.125), ("w2", 0.125)):
        v = getattr(model, name)
        direction = grads[name] / grads[name].norm()
        vals = []
        for s in (step, -step):
            setattr(model, name, v + s * direction * v.numel() ** 0.5 * 0.25)
            vals.append(loss())
        setattr(model, name, v)
        slope = (vals[0] - vals[1]) / (2 * step * v.numel() ** 0.5 * 0.25)
        assert abs(slope - float(grads[name].norm())) < 0.08 * abs(slope), (name, slope, float(grads[name].norm()))
