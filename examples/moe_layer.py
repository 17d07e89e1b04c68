"""A Mixture-of-Experts layer from this package's operators: training step and serving.

    python examples/moe_layer.py [--tokens 4096 --hidden 2048 --ffn 1536 --experts 64 --top-k 8 --fp8]

A token's router logits choose its experts (moe_route); the plan (moe_plan) sorts
the chosen rows by expert; every expert is up [F, H], SiLU, down [H, F]; the
results come back weighted (moe_combine).  Training adds the balance loss to the
loss of the task.  Products run in bf16 (cake_grouped_det_mm) or in 8 bits
(grouped_fp8_mm); serving keeps the weights in 8 bits and routes without autograd.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_ragged_bf16_amd as mdg  # noqa: E402


class MoeLayer(torch.nn.Module):
    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, *, fp8: bool = False, device="cuda"):
        super().__init__()
        make = lambda *s: torch.nn.Parameter(
            (torch.randn(s, device=device) / s[-1] ** 0.5).to(torch.bfloat16))
        self.gate = make(experts, hidden)
        self.up = make(experts, ffn, hidden)
        self.down = make(experts, hidden, ffn)
        self.top_k, self.experts = top_k, experts
        self.product = mdg.grouped_fp8_mm if fp8 else mdg.cake_grouped_det_mm

    def forward(self, x: torch.Tensor, token_mask=None):
        """(out [T, H], balance loss, counts [E]) of x [T, H]; masked tokens get zeros."""
        logits = (x @ self.gate.t()).float()
        route = mdg.moe_route(logits, self.top_k, token_mask=token_mask)
        plan = mdg.moe_plan(route.idx, self.experts)
        rows = mdg.moe_dispatch(x, plan)
        hidden = torch.nn.functional.silu(self.product(rows, self.up, plan.offs))
        y = self.product(hidden, self.down, plan.offs)
        return mdg.moe_combine(y, route.weight, plan), route.loss, route.counts


class MoeServer:
    """The layer's serving form: weights in 8 bits, laid out once."""

    def __init__(self, layer: MoeLayer):
        self.gate, self.top_k, self.experts = layer.gate.detach(), layer.top_k, layer.experts
        self.up = mdg.quantize_fp8_weight(layer.up.detach())
        self.down = mdg.quantize_fp8_weight(layer.down.detach())

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        route = mdg.moe_route_fwd((x @ self.gate.t()).float(), self.top_k)
        plan = mdg.moe_plan(route.idx, self.experts)
        rows = mdg.moe_dispatch_fwd(x, plan)
        hidden = torch.nn.functional.silu(mdg.grouped_fp8_gemm_fwd(rows, self.up.q, self.up.scale, plan.offs))
        y = mdg.grouped_fp8_gemm_fwd(hidden, self.down.q, self.down.scale, plan.offs)
        return mdg.moe_combine_fwd(y, route.weight, plan)


def train_step(layer: MoeLayer, x: torch.Tensor, target: torch.Tensor, balance: float = 0.01):
    out, loss, _ = layer(x)
    total = torch.nn.functional.mse_loss(out.float(), target.float()) + balance * loss
    total.backward()
    return total.detach()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 2048), ("ffn", 1536), ("experts", 64), ("top-k", 8), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--fp8", action="store_true", help="training products in 8 bits")
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = MoeLayer(a.hidden, a.ffn, a.experts, a.top_k, fp8=a.fp8)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    target = torch.randn_like(x)
    opt = torch.optim.SGD(layer.parameters(), lr=1.0)

    def timed(f):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            r = f()
        torch.cuda.synchronize()
        return r, (time.perf_counter() - t) / a.steps

    def step():
        opt.zero_grad()
        r = train_step(layer, x, target)
        opt.step()
        return r

    loss, s = timed(step)
    print(f"training step ({'8 bits' if a.fp8 else 'bf16'}): {s * 1e3:.3f} ms, loss {float(loss):.4f}")
    server = MoeServer(layer)
    for tokens in (a.tokens, 1):
        _, s = timed(lambda: server(x[:tokens]))
        print(f"serving {tokens} tokens: {s * 1e3:.3f} ms")


if __name__ == "__main__":
    main()
