"""Experts that the fused layer does not have, built from its pieces, on one GPU: one
matrix in, a squared ReLU, one matrix out.  The stacked expert weights are trained with
the Muon rule (momentum, then the orthogonalised update of every expert's matrix), the
router with Adam.

    python examples/open_experts.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dispatch_grouped_gemm_gb300 as hmm  # noqa: E402


class Muon(torch.optim.Optimizer):
    """p -= lr * sqrt(max(1, M / N)) * orthogonalize(g + momentum * m), m = momentum * m + g,
    for stacks [..., M, N] of matrices."""

    def __init__(self, params, lr=0.02, momentum=0.95, steps=5):
        super().__init__(params, dict(lr=lr, momentum=momentum, steps=steps))

    @torch.no_grad()
    def step(self):
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if not state:
                    state["momentum"] = torch.zeros_like(p, dtype=torch.float32)
                m = state["momentum"].mul_(group["momentum"]).add_(p.grad)
                M, N = p.shape[-2:]
                update = hmm.orthogonalize(m * group["momentum"] + p.grad, steps=group["steps"],
                                           scale=max(1.0, M / N) ** 0.5, out_dtype=torch.bfloat16)
                p.add_(update, alpha=-group["lr"])


class OpenExperts(torch.nn.Module):
    """y = experts(x) with K of E experts per token."""

    def __init__(self, H, I, E, K, device="cuda"):
        super().__init__()
        self.K, self.E = K, E

        def weight(*shape):
            w = torch.randn(shape, device=device) * shape[-2] ** -0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.router = weight(H, E)
        self.up, self.down = weight(E, H, I), weight(E, I, H)

    def experts(self, x, ids, w):
        routing = hmm.moe_route(ids, self.E)
        rows = hmm.moe_dispatch(x, routing)
        h = torch.relu(hmm.moe_grouped_mm(rows, self.up, routing.offsets)).square()
        return hmm.moe_combine(hmm.moe_grouped_mm(h, self.down, routing.offsets), routing, w)

    def forward(self, x):
        ids, w = hmm.moe_gate(x @ self.router, self.K, renormalize=True)
        return self.experts(x, ids, w)


def main(steps=10, T=512, H=512, I=768, E=16, K=2):
    """Returns (losses of the training steps, the layer)."""
    torch.manual_seed(0)
    layer, target = OpenExperts(H, I, E, K), OpenExperts(H, I, E, K)
    muon = Muon([layer.up, layer.down])
    adam = torch.optim.Adam([layer.router], lr=1e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            want = target(x).float()
        loss = (layer(x).float() - want).square().mean()
        muon.zero_grad()
        adam.zero_grad()
        loss.backward()
        muon.step()
        adam.step()
        losses.append(loss.item())
    return losses, layer


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=10)
    print("loss: " + " ".join(f"{v:.4f}" for v in main(ap.parse_args().steps)[0]))
