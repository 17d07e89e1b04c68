"""Transformer half-blocks of gated experts from this package's operators: a training
step with clipped gradients, and serving.

    python examples/moe_block.py [--tokens 4096 --hidden 2048 --ffn 1536 --experts 64 --top-k 8 --layers 2]

A layer takes the residual stream and what the layer before added to it.  One
call adds them (with the norm after a block, a gate for each token and a scale)
and norms the sum for the router and the experts (block_norm); each token's
rows go to its experts (moe_route, moe_plan, moe_dispatch), which are gated
feed-forwards (grouped_gated_ffn), and come back weighted (moe_combine).  The
experts' weight gradients are added into fp32 main_grads by the products'
epilogue; clip_grads clips all gradients by their norm before the update.
Serving runs the single calls, which record nothing for autograd.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_ragged_bf16_amd as mdg  # noqa: E402


class MoeBlock(torch.nn.Module):
    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, *, scale: float = 0.5, device="cuda"):
        super().__init__()
        make = lambda *s: torch.nn.Parameter((torch.randn(s, device=device) / s[-1] ** 0.5).to(torch.bfloat16))
        ones = lambda: torch.nn.Parameter(torch.ones(hidden, device=device))
        self.norm, self.post_norm = ones(), ones()          # fp32, before and after the block
        self.router, self.token_gate = make(experts, hidden), make(1, hidden)
        self.gate_up, self.down = make(experts, 2 * ffn, hidden), make(experts, hidden, ffn)
        self.top_k, self.experts, self.scale = top_k, experts, scale
        for w in (self.gate_up, self.down):
            w.main_grad = torch.zeros(w.shape, device=device)

    def add(self, residual, y, weight):
        """The residual stream with this block's y added, and its norm for the next block."""
        gate = torch.sigmoid((y @ self.token_gate.t()).float()).flatten()
        return mdg.block_norm(residual, y, post_weight=self.post_norm, gate=gate, scale=self.scale, weight=weight)

    def forward(self, n: torch.Tensor):
        """(y [T, H], balance loss) of normed rows n [T, H]."""
        route = mdg.moe_route((n @ self.router.t()).float(), self.top_k)
        plan = mdg.moe_plan(route.idx, self.experts)
        rows = mdg.grouped_gated_ffn(mdg.moe_dispatch(n, plan), self.gate_up, self.down, plan.offs,
                                     fuse_wgrad_accumulation=True)
        return mdg.moe_combine(rows, route.weight, plan), route.loss

    @torch.no_grad()
    def serve(self, n: torch.Tensor) -> torch.Tensor:
        route = mdg.moe_route_fwd((n @ self.router.t()).float(), self.top_k)
        plan = mdg.moe_plan(route.idx, self.experts)
        h = mdg.grouped_gated_gemm_fwd(mdg.moe_dispatch_fwd(n, plan), self.gate_up, plan.offs).h
        return mdg.moe_combine_fwd(mdg.grouped_det_gemm_fwd(h, self.down, plan.offs), route.weight, plan)


class MoeStack(torch.nn.Module):
    def __init__(self, layers: int, hidden: int, *args, device="cuda", **kw):
        super().__init__()
        self.blocks = torch.nn.ModuleList(MoeBlock(hidden, *args, device=device, **kw) for _ in range(layers))
        self.final = torch.nn.Parameter(torch.ones(hidden, device=device))

    def weights(self):
        """The norm weight before each block but the first, and the last one."""
        return [b.norm for b in self.blocks[1:]] + [self.final]

    def forward(self, x: torch.Tensor):
        """(normed output [T, H], balance loss)."""
        stream, n = mdg.block_norm(x, weight=self.blocks[0].norm)
        loss = 0.0
        for block, weight in zip(self.blocks, self.weights()):
            y, balance = block(n)
            loss = loss + balance
            stream, n = block.add(stream, y, weight)
        return n, loss

    @torch.no_grad()
    def serve(self, x: torch.Tensor) -> torch.Tensor:
        stream, n = mdg.block_norm_fwd(x, weight=self.blocks[0].norm)[:2]
        for block, weight in zip(self.blocks, self.weights()):
            stream, n = block.add(stream, block.serve(n), weight)
        return n

    def gradients(self):
        """Every parameter's gradient: main_grad where it has one."""
        return [p.main_grad if hasattr(p, "main_grad") else p.grad for p in self.parameters()]


def train_step(stack: MoeStack, x: torch.Tensor, target: torch.Tensor, *, balance: float = 0.01, max_norm: float = 1.0,
               lr: float = 0.0):
    """One step; returns the loss and the gradients' norm before clipping (on the device)."""
    for p in stack.parameters():
        p.grad = None
        if hasattr(p, "main_grad"):
            p.main_grad.zero_()
    n, loss = stack(x)
    total = torch.nn.functional.mse_loss(n.float(), target.float()) + balance * loss
    total.backward()
    grads = stack.gradients()
    norm = mdg.clip_grads(grads, max_norm)
    if lr:
        with torch.no_grad():
            for p, g in zip(stack.parameters(), grads):
                p.sub_(g.to(p.dtype), alpha=lr)
    return total.detach(), norm


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 2048), ("ffn", 1536), ("experts", 64), ("top-k", 8), ("layers", 2),
                          ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    torch.manual_seed(0)
    stack = MoeStack(a.layers, a.hidden, a.ffn, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    target = torch.randn_like(x)

    def timed(f):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            r = f()
        torch.cuda.synchronize()
        return r, (time.perf_counter() - t) / a.steps

    (loss, norm), s = timed(lambda: train_step(stack, x, target, lr=0.1))
    print(f"training step: {s * 1e3:.3f} ms, loss {float(loss):.4f}, gradient norm {float(norm):.4f}")
    for tokens in (a.tokens, 1):
        _, s = timed(lambda: stack.serve(x[:tokens]))
        print(f"serving {tokens} tokens: {s * 1e3:.3f} ms")


if __name__ == "__main__":
    main()
