"""A training step of an expert layer, through the library's grouped products and Newton-Schulz.

``python -m fp64_gemm_emulation_gb300.run_experts --tokens 4096 --experts 8 --k 512 --n 768 --steps 10``

Tokens are routed to one expert each (sorted by expert; the row offsets stay on the device).
A step is the forward product, the loss against a fixed teacher layer, the gradients in the
tokens and in the weights, a momentum, and the orthogonalised momentum as the update.
Prints the loss of each step.
"""
from __future__ import annotations

import argparse


def route(choice, experts: int):
    """Sorts tokens by expert: (order, offsets) with offsets int32 (experts + 1), all on the device."""
    import torch

    order = torch.argsort(choice, stable=True)
    counts = torch.zeros(experts, dtype=torch.int64, device=choice.device).scatter_add_(0, choice, torch.ones_like(choice))
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=choice.device)
    offsets[1:] = counts.cumsum(0)
    return order, offsets


class ExpertLayer:
    """W (experts, n, k) with a bfloat16 momentum, updated by its Newton-Schulz orthogonalisation."""

    def __init__(self, W, lr: float = 0.02, momentum: float = 0.9):
        import torch

        self.W, self.lr, self.momentum = W, lr, momentum
        self.M = torch.zeros_like(W)

    def step(self, X, offsets, target):
        """One step on tokens X (rows, k) sorted by expert: (loss, gradient in X)."""
        from . import ozaki as oz

        Y = oz.ozaki_grouped_gemm(X, self.W, offsets)
        diff = Y.float() - target.float()
        rows = max(1, X.shape[0])
        loss = 0.5 * diff.square().sum() / rows
        dY = (diff / rows).to(X.dtype)
        dX = oz.ozaki_grouped_gemm_dgrad(dY, self.W, offsets)
        dW = oz.ozaki_grouped_gemm_wgrad(dY, X, offsets)
        self.M.mul_(self.momentum).add_(dW)
        update = oz.ozaki_newton_schulz(self.M)
        self.W.sub_(self.lr * update)
        return loss, dX


def train(tokens: int, experts: int, k: int, n: int, steps: int, seed: int = 0, lr: float = 0.02) -> list[float]:
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

    from . import ozaki as oz

    X = randn(tokens, k)
    order, offsets = route(torch.randint(experts, (tokens,), generator=gen, device="cuda"), experts)
    X = X[order].contiguous()
    teacher = randn(experts, n, k, scale=k ** -0.5)
    target = oz.ozaki_grouped_gemm(X, teacher, offsets)
    layer = ExpertLayer((teacher.float() + torch.randn(teacher.shape, generator=gen, device="cuda") * k ** -0.5).to(torch.bfloat16), lr)
    losses = []
    for _ in range(steps):
        loss, _ = layer.step(X, offsets, target)
        losses.append(float(loss))
    status = oz.ozaki_get_device_status()
    if status != oz.OZ_OK:
        raise RuntimeError(f"device status {oz.ozaki_status_string(status)}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--k", type=int, default=512)
    ap.add_argument("--n", type=int, default=768)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--lr", type=float, default=0.02)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.tokens, a.experts, a.k, a.n, a.steps, a.seed, a.lr)):
        print(f"step {i}: loss {loss:.4f}")


if __name__ == "__main__":
    main()
