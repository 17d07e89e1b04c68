"""The operators together, as examples/moe_layer.py runs them: output, balance loss
and gradients against the layer written out in fp32, and the serving form.

Tolerances: every bf16 rounding on the way (rows, hidden, y, out: 2^-8 each, of
values whose errors average over the sums) adds at most 2^-8 in the 2-norm; the
chain is 5 roundings forward and 9 to a weight's gradient: 5 and 9 times 2^-8.
8 bits: an e4m3 value is off by at most 2^-4 of itself, both operands of both
products: 4 * 2^-4 forward.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def plain(layer, x, mask):
    """The layer in fp32 on the CPU, expert by expert, with its own autograd."""
    p = [t.detach().float().cpu().requires_grad_() for t in (x, layer.gate, layer.up, layer.down)]
    xf, gate, up, down = p
    # the router's logits as the layer has them (bf16 product): the choice of experts is discrete
    logits = (x @ layer.gate.t()).float().detach().cpu() + (xf @ gate.t() - (xf @ gate.t()).detach())
    keep = torch.ones(x.shape[0], dtype=torch.bool) if mask is None else mask.cpu()
    prob = torch.softmax(logits, dim=1)
    top = torch.topk(logits, layer.top_k, dim=1)
    w = torch.softmax(top.values, dim=1)
    out = torch.zeros_like(xf)
    counts = torch.zeros(layer.experts)
    for e in range(layer.experts):
        t, j = torch.nonzero((top.indices == e) & keep[:, None], as_tuple=True)
        counts[e] = len(t)
        y = torch.nn.functional.silu(xf[t] @ up[e].t()) @ down[e].t()
        out = out.index_add(0, t, y * w[t, j][:, None])
    R = int(keep.sum())
    loss = layer.experts / (layer.top_k * R * R) * (counts * prob[keep].sum(dim=0)).sum()
    return p, out, loss, counts


def rel(a, b):
    return float((a.float().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_against_plain(fp8):
    torch.manual_seed(0)
    T, H, F, E, k = 203, 256, 208, 12, 3
    layer = moe_layer.MoeLayer(H, F, E, k, fp8=fp8)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16).requires_grad_()
    mask = torch.rand(T, device="cuda") > 0.1
    dout = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    out, loss, counts = layer(x, mask)
    p, want, wloss, wcounts = plain(layer, x, mask)
    fwd, bwd = (4 * 2.0 ** -4, 8 * 2.0 ** -4) if fp8 else (5 * 2.0 ** -8, 9 * 2.0 ** -8)
    assert torch.equal(counts.cpu(), wcounts.int())
    assert abs(float(loss) - float(wloss)) <= 2.0 ** -10 * float(wloss)
    assert rel(out, want.detach()) <= fwd
    assert torch.all(out[~mask] == 0)
    ((out.float() * dout.float()).sum() + 0.5 * loss).backward()
    ((want * dout.float().cpu()).sum() + 0.5 * wloss).backward()
    for got, ref in zip((x, layer.gate, layer.up, layer.down), p):
        assert rel(got.grad, ref.grad) <= bwd


def test_serving_form_and_single_tokens():
    torch.manual_seed(1)
    T, H, F, E, k = 65, 256, 208, 12, 3
    layer = moe_layer.MoeLayer(H, F, E, k)
    server = moe_layer.MoeServer(layer)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    _, want, _, _ = plain(layer, x, None)
    got = server(x)
    assert rel(got, want.detach()) <= 4 * 2.0 ** -4
    for t in (0, 17):
        assert rel(server(x[t:t + 1]), want[t:t + 1].detach()) <= 2 * 4 * 2.0 ** -4


def test_training_steps_reduce_the_loss():
    torch.manual_seed(2)
    for fp8 in (False, True):
        layer = moe_layer.MoeLayer(128, 128, 8, 2, fp8=fp8)
        x = torch.randn((256, 128), device="cuda").to(torch.bfloat16)
        target = torch.tanh(x.float() * 0.5).to(torch.bfloat16)
        opt = torch.optim.SGD(layer.parameters(), lr=2.0)
        losses = []
        for _ in range(12):
            opt.zero_grad()
            losses.append(float(moe_layer.train_step(layer, x, target)))
            opt.step()
        assert losses[-1] < 0.95 * losses[0], losses
