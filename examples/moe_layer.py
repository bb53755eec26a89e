"""A mixture-of-experts layer end to end on one GPU: a grouped sigmoid router
with a balance bias in front of the fused experts, a few training steps in bf16,
then the same layer served with 4-bit experts.

    python examples/moe_layer.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dispatch_grouped_gemm_gb300 as hmm  # noqa: E402

ROUTER = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, renormalize=True, scale=1.0)


class MoELayer(torch.nn.Module):
    """y = experts(x) with K of E experts per token."""

    def __init__(self, H, I, E, K, device="cuda"):
        super().__init__()
        self.K, self.E = K, E

        def weight(*shape):
            w = torch.randn(shape, device=device) * shape[-2] ** -0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.router = weight(H, E)
        self.up, self.down = weight(E, H, 2 * I), weight(E, I, H)
        # moved in small steps against the load, not by the loss
        self.register_buffer("bias", torch.zeros(E, device=device))
        self.up4 = self.down4 = None

    def route(self, x, return_scores=False):
        return hmm.moe_gate(x @ self.router, self.K, bias=self.bias, return_scores=return_scores,
                            **ROUTER)

    def forward(self, x):
        ids, w, p = self.route(x, return_scores=True)
        load = torch.bincount(ids.flatten(), minlength=self.E).float() / ids.numel()
        balance = self.E * (load * (p / p.sum(1, keepdim=True)).mean(0)).sum()
        with torch.no_grad():
            self.bias += 1e-3 * torch.sign(1.0 / self.E - load)
        return hmm.moe_ffn(x, ids, w, self.up, self.down), balance

    def quantize(self):
        """4-bit experts for serving (4.25 bits a weight)."""
        self.up4 = hmm.mx4_quantize_experts(self.up.detach(), gate_up=True)
        self.down4 = hmm.mx4_quantize_experts(self.down.detach())

    @torch.no_grad()
    def serve(self, x):
        ids, w = self.route(x)
        return hmm.moe_ffn_mx4(x, ids, w, self.up4, self.down4)


def main(steps=10, T=512, H=1024, I=512, E=32, K=4):
    """Returns (losses of the training steps, relative distance of the 4-bit
    layer's outputs from the bf16 layer's)."""
    torch.manual_seed(0)
    layer = MoELayer(H, I, E, K)
    target = MoELayer(H, I, E, K)
    opt = torch.optim.Adam(layer.parameters(), lr=1e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            want = target(x)[0].float()
        y, balance = layer(x)
        loss = (y.float() - want).square().mean() + 1e-2 * balance
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    layer.quantize()
    with torch.no_grad():
        x = torch.randn((64, H), device="cuda").to(torch.bfloat16)
        ids, w = layer.route(x)
        want = hmm.moe_ffn(x, ids, w, layer.up, layer.down).float()
        got = layer.serve(x).float()
        one = layer.serve(x[:1].contiguous()).float()  # a single token: the same row
        assert torch.equal(one, got[:1])
    return losses, ((got - want).norm() / want.norm()).item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=10)
    losses, off = main(ap.parse_args().steps)
    print("loss: " + " ".join(f"{v:.4f}" for v in losses))
    print(f"4-bit experts: outputs {off:.3f} (relative) from the bf16 experts'")
