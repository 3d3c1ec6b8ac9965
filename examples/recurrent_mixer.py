"""A small recurrent mixer trained and served with the library's operators.

One layer: a gated linear recurrence over the width, its grouped norm with an activated gate, then the
Gated DeltaProduct recurrence over the normed rows and a second grouped norm.  The norms keep 8-bit
checkpoints, and the backward passes read only those: no 16-bit activation of either recurrence is kept
(the Gated DeltaProduct's backward recomputes its forward from q, k, v, which are the normed rows here).

  train_step   forward, loss, backward, one SGD step on the gates and the norm weights
  serve        the same layer over a prompt, then token by token over the state caches

Run on a GPU: python examples/recurrent_mixer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_deltaproduct_gb300 as gdp  # noqa: E402


class Mixer:
    """H heads of D channels; parameters are the recurrence's gate logits per channel and the norms' weights."""

    def __init__(self, H: int, D: int, device, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        self.H, self.D, self.device = H, D, device
        self.gate = torch.full((H * D,), 2.0) + 0.5 * torch.randn(H * D, generator=gen)
        self.gate = self.gate.to(device)  # decays sigmoid(2) = 0.88 and around
        self.w1, self.w2 = torch.ones(D, device=device), torch.ones(H, D, device=device)

    def _logits(self, x):
        """Gate logits of every token: the channel's own plus half the input (any projection in a real model)."""
        return (self.gate + 0.5 * x.float()).to(x.dtype)

    def forward(self, x, z, g, beta, cu, keep=True):
        """x, z [T, H*D] bf16 (packed); g [T, H] decay logs, beta [T, H].  Returns the output and what the
        backward pass needs."""
        T, H, D = x.shape[0], self.H, self.D
        logits = self._logits(x)
        h = gdp.gated_linear_recurrence(x, logits, cu, gate="sigmoid")
        y, c1 = gdp.gated_group_norm(h.view(T, H, D), self.w1, z.view(T, H, D), save_checkpoint=True)
        o = gdp.chunk_gated_delta_product(y, y, y, g, beta, cu, 1, use_qk_l2norm_in_kernel=True)
        out, c2 = gdp.gated_group_norm(o, self.w2, center=True, save_checkpoint=True)
        return out, (x, logits, y, g, beta, cu, c1, c2) if keep else None

    def backward(self, saved, d_out):
        """Gradients of the gate logits' parameter and of both norms' weights, and of x."""
        x, logits, y, g, beta, cu, c1, c2 = saved
        T, H, D = y.shape
        n2 = gdp.gated_group_norm_backward(d_out, c2, self.w2, center=True)
        r2 = gdp.chunk_gated_delta_product_backward(y, y, y, g, beta, cu, 1, n2["do"], use_qk_l2norm_in_kernel=True)
        dy = (r2["dq"] + r2["dk"] + r2["dv"]).to(y.dtype)
        n1 = gdp.gated_group_norm_backward(dy, c1, self.w1)
        r1 = gdp.gated_linear_recurrence_backward(logits, c1.o, n1["do"].view(T, H * D), cu, gate="sigmoid", x=x)
        dg = r1["dg"].float()
        return {"gate": dg.sum(0), "w1": n1["dweight"], "w2": n2["dweight"], "x": r1["dx"].float() + 0.5 * dg,
                "z": n1["dz"].view(T, H * D)}

    def prefill(self, x, z, g, beta, cu, rec_cache, gdp_cache, slots):
        """The forward over prompts, states written into the two caches at ``slots``."""
        T, H, D = x.shape[0], self.H, self.D
        h = gdp.gated_linear_recurrence(x, self._logits(x), cu, gate="sigmoid", state=rec_cache, state_indices=slots)
        y = gdp.gated_group_norm(h.view(T, H, D), self.w1, z.view(T, H, D))
        o = gdp.chunk_gated_delta_product(y, y, y, g, beta, cu, 1, use_qk_l2norm_in_kernel=True, state=gdp_cache,
                                          state_indices=slots)
        return gdp.gated_group_norm(o, self.w2, center=True)

    def step(self, x, z, g, beta, rec_cache, gdp_cache, slots):
        """One token per request: x, z [N, H*D], g, beta [N, H]."""
        N, H, D = x.shape[0], self.H, self.D
        h = gdp.gated_linear_recurrence_decode(x, self._logits(x), gate="sigmoid", state=rec_cache, state_indices=slots)
        y = gdp.gated_group_norm(h.view(N, H, D), self.w1, z.view(N, H, D))
        o = gdp.gated_delta_product_decode(y, y, y, g, beta, 1, use_qk_l2norm_in_kernel=True, state=gdp_cache,
                                           state_indices=slots)
        return gdp.gated_group_norm(o, self.w2, center=True)


def make_batch(lengths, H, D, device, seed):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lengths)
    x, z = (torch.randn(T, H * D, generator=gen).to(device, torch.bfloat16) for _ in range(2))
    g = (-0.05 * torch.rand(T, H, generator=gen)).to(device)
    beta = torch.sigmoid(torch.randn(T, H, generator=gen)).to(device)
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=device)
    return x, z, g, beta, cu


def train(steps=20, lengths=(200, 77, 300), H=2, D=64, device="cuda", lr=0.2):
    """Fits the layer to a teacher of other parameters; returns the losses."""
    teacher, model = Mixer(H, D, device, seed=1), Mixer(H, D, device, seed=2)
    teacher.w1 = teacher.w1 * 1.5
    batch = make_batch(list(lengths), H, D, device, seed=3)
    target = teacher.forward(*batch, keep=False)[0].float()
    losses = []
    for _ in range(steps):
        out, saved = model.forward(*batch)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        grads = model.backward(saved, (2.0 * diff).to(out.dtype))
        for name in ("gate", "w1", "w2"):
            grad = grads[name] / out.shape[0]
            setattr(model, name, getattr(model, name) - lr * grad)
    return losses


def serve(lengths=(40, 3, 129), new_tokens=4, H=2, D=64, device="cuda"):
    """Prompt over the caches, then token by token; returns those outputs and the same from one whole pass."""
    model = Mixer(H, D, device, seed=1)
    whole = [n + new_tokens for n in lengths]
    x, z, g, beta, cu = make_batch(whole, H, D, device, seed=4)
    reference = model.forward(x, z, g, beta, cu, keep=False)[0]
    starts = cu.tolist()[:-1]
    prompt = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lengths)]).to(device)
    pcu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=device)
    slots = torch.arange(len(lengths), dtype=torch.int32, device=device).flip(0).contiguous()
    rec_cache = torch.zeros((len(lengths) + 1, H * D), device=device)
    gdp_cache = torch.zeros((len(lengths) + 1, H, D, D), device=device)
    model.prefill(x[prompt], z[prompt], g[prompt], beta[prompt], pcu, rec_cache, gdp_cache, slots)
    outs, refs = [], []
    for i in range(new_tokens):
        at = torch.tensor([s + n + i for s, n in zip(starts, lengths)], device=device)
        outs.append(model.step(x[at], z[at], g[at], beta[at], rec_cache, gdp_cache, slots))
        refs.append(reference[at])
    return torch.stack(outs), torch.stack(refs)


if __name__ == "__main__":
    losses = train()
    print("training loss %.4f -> %.4f" % (losses[0], losses[-1]))
    got, want = serve()
    print("decode after prefill against one pass: largest difference %.4f" % float((got.float() - want.float()).abs().max()))
