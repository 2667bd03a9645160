"""A RoSA adapter trained and served with this package's operators.

    python examples/rosa_finetune_and_serve.py

Training: a frozen two-layer MLP whose projections carry a low-rank and a sparse update
(RosaLinear: csr_add into the weight, lora_add beside the projection; lora_grad and sddmm
backward), the gradients clipped by their global norm (clip_grads on a GradSet of fixed buffers)
and applied by masked_adam to fp32 master copies; once more with the frozen weights in 4 bits
(mx4_linear, mx4_linear_grad) and dropout in front of the low-rank factors. Serving: one batch of requests with several
adapters, their prompts first and then one token each, through lora_add.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unstructured_sparse_linear_gb300 as sp  # noqa: E402


def random_mask(out_features, in_features, density, gen, device):
    """A uniform CSR mask (row_offsets int32, col_idx int16)."""
    keep = torch.rand(out_features, in_features, generator=gen, device=device) < density
    row_offsets = torch.zeros(out_features + 1, dtype=torch.int32, device=device)
    row_offsets[1:] = keep.sum(1).cumsum(0).to(torch.int32)
    return row_offsets, keep.nonzero()[:, 1].to(torch.int16).contiguous()


def rosa_layer(out_features, in_features, rank, gen, device, dtype, four_bits=False, dropout=0.0):
    w = torch.randn(out_features, in_features, generator=gen, device=device).mul_(in_features ** -0.5).to(dtype)
    if four_bits:  # the low-rank part only: beside a sparse one the weight is formed in every pass
        return sp.RosaLinear(sp.mx4_quantize(w), rank, scale=2.0, dropout=dropout)
    row_offsets, col_idx = random_mask(out_features, in_features, 0.01, gen, device)
    values = torch.zeros(col_idx.numel(), dtype=dtype, device=device)
    return sp.RosaLinear(w, rank, scale=2.0, row_offsets=row_offsets, col_idx=col_idx, values=values, dropout=dropout)


class Trainer:
    """fp32 master copies, fixed gradient buffers in one GradSet, masked_adam."""

    def __init__(self, params, lr=1e-2, max_norm=1.0):
        self.params = list(params)
        self.master = [p.detach().float().reshape(-1).clone() for p in self.params]
        self.state = [(torch.zeros_like(m), torch.zeros_like(m)) for m in self.master]
        for p in self.params:
            p.grad = torch.zeros_like(p)
        self.set = sp.GradSet([p.grad for p in self.params])
        self.lr, self.max_norm, self.steps = lr, max_norm, 0

    def step(self):
        norm = sp.clip_grads(self.set, self.max_norm)
        self.steps += 1
        for p, m, (a, b) in zip(self.params, self.master, self.state):
            sp.masked_adam(m, a, b, p.grad.reshape(-1), self.steps, lr=self.lr)
            p.data.copy_(m.reshape(p.shape))
            p.grad.zero_()  # (autograd adds to the same buffer)
        return norm


def train(steps=20, tokens=1000, hidden=256, inner=512, rank=8, dtype=torch.bfloat16, device="cuda", four_bits=False,
          dropout=0.0):
    """Fits the MLP to a target that differs from it; returns the losses and gradient norms. four_bits: the frozen
    weights are kept in 4 bits; dropout: in front of the low-rank factors."""
    gen = torch.Generator(device=device).manual_seed(0)
    torch.manual_seed(0)  # (the layers' dropout draws its states from torch's generator)
    up, down = (rosa_layer(n_out, n_in, rank, gen, device, dtype, four_bits, dropout)
                for n_out, n_in in ((inner, hidden), (hidden, inner)))
    X = torch.randn(tokens, hidden, generator=gen, device=device).to(dtype)
    target = torch.randn(tokens, hidden, generator=gen, device=device).to(dtype)
    trainer = Trainer([*up.parameters(), *down.parameters()])
    losses, norms = [], []
    for _ in range(steps):
        loss = (down(torch.relu(up(X))) - target).float().square().mean()
        loss.backward()
        norms.append(trainer.step())
        losses.append(loss.detach())
    return [float(x) for x in losses], [float(x) for x in norms]


def serve(prompts=(7, 130, 64, 1, 300), adapters=4, hidden=256, out=512, rank=16, dtype=torch.bfloat16, device="cuda"):
    """A batch of prompts, then one token per request, each request with its adapter (the last one
    without): the outputs of both steps and what they were computed from."""
    gen = torch.Generator(device=device).manual_seed(1)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=device).mul_(std).to(dtype)

    W, A, B = randn(out, hidden, std=hidden ** -0.5), randn(adapters, rank, hidden, std=hidden ** -0.5), \
        randn(adapters, out, rank, std=0.1)
    which = [i % adapters for i in range(len(prompts) - 1)] + [-1]
    steps = []
    for lengths in (list(prompts), [1] * len(prompts)):
        ids = torch.tensor([a for a, n in zip(which, lengths) for _ in range(n)], dtype=torch.int32, device=device)
        plan = sp.lora_plan(ids, adapters)  # one plan serves every projection of every layer
        X = randn(len(ids), hidden)
        Y = X @ W.t()
        sp.lora_add(X, A, B, plan, base=Y, scale=0.5, out=Y)
        steps.append(dict(X=X, ids=ids, Y=Y))
    return dict(W=W, A=A, B=B, scale=0.5, steps=steps)


def main():
    losses, norms = train()
    print("loss", " ".join(f"{x:.3f}" for x in losses))
    print("gradient norm", " ".join(f"{x:.3f}" for x in norms))
    losses, _ = train(four_bits=True, dropout=0.1)
    print("loss, frozen weights in 4 bits and dropout", " ".join(f"{x:.3f}" for x in losses))
    for s in serve()["steps"]:
        print(f"served {len(s['ids'])} tokens of {int(s['ids'].max()) + 1} adapters:", tuple(s["Y"].shape))


if __name__ == "__main__":
    main()
