"""examples/moe_block.py: norms, routing, gated experts, residual and clipping together.

The stack's output and every gradient against the same mathematics in plain torch
operations in 64 bits, with the routing choices of the run.  Bound: a value passes
at most 12 roundings to bf16 a layer (the stream, its norm, the projections, h, the
experts' rows, their sum, and the gradients of each), each off by 2^-8 of the value at most,
so 24 * 2^-8 of the 2-norm for two layers."""
import os
import sys

import pytest
import torch

import moe_ragged_bf16_amd as mdg

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, F, E, K, LAYERS = 96, 128, 64, 6, 2, 2
BOUND = 24 * 2.0 ** -8


def make(seed=0):
    torch.manual_seed(seed)
    stack = moe_block.MoeStack(LAYERS, H, F, E, K)
    with torch.no_grad():
        for p in stack.parameters():
            if p.dim() == 1:
                p.add_(0.2 * torch.randn_like(p))
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    return stack, x, torch.randn((T, H), device=DEV).to(torch.bfloat16)


def rms(v, w):
    return v / torch.sqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * w


def plain(p, x, choices, target, balance):
    """The stack in plain operations on fp64 leaves p (by name) and the choices [T, K] of each layer."""
    stream, loss = x, 0.0
    n = rms(stream, p["blocks.0.norm"])
    for i in range(LAYERS):
        q = lambda name: p[f"blocks.{i}.{name}"]
        logits = n @ q("router").t()
        idx = choices[i].long()
        prob = torch.softmax(logits, dim=1)
        weight = torch.softmax(logits.gather(1, idx), dim=1)
        counts = torch.bincount(idx.flatten(), minlength=E).double()
        loss = loss + (E / (K * T * T) * counts * prob.sum(dim=0)).sum()
        y = 0
        for j in range(K):
            gu, down = q("gate_up")[idx[:, j]], q("down")[idx[:, j]]
            ab = torch.einsum("tfh,th->tf", gu, n)
            h = torch.nn.functional.silu(ab[:, :F]) * ab[:, F:]
            y = y + weight[:, j:j + 1] * torch.einsum("thf,tf->th", down, h)
        gate = torch.sigmoid(y @ q("token_gate").t())
        stream = stream + 0.5 * gate * rms(y, q("post_norm"))
        n = rms(stream, p[f"blocks.{i + 1}.norm"] if i + 1 < LAYERS else p["final"])
    return n, torch.nn.functional.mse_loss(n, target) + balance * loss


def near(got, want):
    return float((got.double().cpu() - want.cpu()).norm()) <= BOUND * float(want.norm())


def test_training_step_and_serving():
    stack, x, target = make()
    choices = []
    real = mdg.moe_plan
    mdg.moe_plan = lambda idx, experts: (choices.append(idx), real(idx, experts))[1]
    try:
        loss, norm = moe_block.train_step(stack, x, target, max_norm=1e9)
    finally:
        mdg.moe_plan = real
    assert len(choices) == LAYERS and all(int(c.min()) >= 0 for c in choices)
    leaves = {k: v.detach().double().cpu().requires_grad_() for k, v in stack.named_parameters()}
    n, want = plain(leaves, x.double().cpu(), [c.cpu() for c in choices], target.double().cpu(), 0.01)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= BOUND * want
    assert near(stack.serve(x), n.detach())
    grads = dict(zip((k for k, _ in stack.named_parameters()), stack.gradients()))
    for k, g in grads.items():
        assert near(g, leaves[k].grad), (k, float((g.double().cpu() - leaves[k].grad).norm() / leaves[k].grad.norm()))
    total = sum(float(g.double().square().sum()) for g in grads.values()) ** 0.5
    assert abs(float(norm) - total) <= 2.0 ** -23 * total       # (max_norm 1e9: the gradients are as they were)
    # the same step clipped: the same bits before, each gradient scaled by one factor after
    before = [g.clone() for g in stack.gradients()]
    _, again = moe_block.train_step(stack, x, target, max_norm=0.25 * float(norm))
    assert torch.equal(again, norm)
    by = torch.tensor(0.25 * float(norm), device=DEV).double() / (norm.double() + 1e-6)
    for g, b in zip(stack.gradients(), before):
        assert torch.allclose(g.double(), b.double() * by, rtol=2.0 ** -7, atol=0)


def test_repeats_bit_for_bit_and_serves_single_tokens():
    stack, x, target = make(1)
    runs = []
    for _ in range(2):
        _, norm = moe_block.train_step(stack, x, target)
        runs.append([norm] + [g.clone() for g in stack.gradients()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert torch.equal(stack.serve(x), stack.serve(x)) and stack.serve(x[:1]).shape == (1, H)
    one = stack.serve(x[:1]).double()
    assert float((one - stack.serve(x)[:1].double()).norm()) <= BOUND * float(one.norm())


def test_runs_as_a_program():
    import subprocess
    # (a child process of its own: it uses the GPU beside this one)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_block.py"), "--tokens", "64", "--hidden", "256",
                        "--ffn", "128", "--experts", "8", "--top-k", "2", "--steps", "2"], capture_output=True, text=True,
                       timeout=110, cwd=root)
    assert r.returncode == 0, r.stderr[-500:]
    assert "training step" in r.stdout and "serving 1 tokens" in r.stdout
