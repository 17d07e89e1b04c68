"""The layer of examples/moe_layer.py in 8 bits (and in bf16), stage by stage and
element by element: each stage is checked on the values that it really got, so
nothing is left to average out.

Products and their gradients are compared with 64 bits on the quantised operands
(straight-through: the gradient by x is that of the product with the quantised
weight, by w the product of the unquantised operands).  Tolerances: in 8 bits
7 * 2^-13 * sum over groups of 8 of 2^E plus (K + 8) u sum |products|, u = 2^-24; in bf16
and for weight gradients (n + 8) u sum |products| of n terms; a bf16 result has to lie
between the bf16 roundings of the interval's ends.  Everything between the products
has to have the bits of the package's single calls, or of torch, on those values.
"""
import os
import sys

import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import fp8 as ref
from test_gpu_fp8 import U, group_bound, h, inside

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check_product(a, w, ends, got, fp8):
    """got = a @ w[e]^T by group, of what the operands stand for (fp64 arrays a [M, K], w [E, N, K])."""
    K = a.shape[1]
    bound = 0.0
    if fp8:
        (qa, ca), (qw, cw) = ref.quantize_rows(a), ref.quantize_weight(w)
        bound = group_bound(qa, ca, qw, cw, ends)
        a, w = ref.dequantize(qa, ca, (1, 128)), ref.dequantize(qw, cw, (128, 128))
    want = ref.grouped_product(a, w, ends)
    size = ref.grouped_product(np.abs(a), np.abs(w), ends)
    assert inside(got, want, (K + 8) * U * size + bound)
    assert np.all(h(got[int(ends[-1]):]) == 0)


def check_wgrad(dy, x, ends, got):
    start = 0
    for e, end in enumerate(ends):
        g, v = dy[start:end], x[start:end]
        assert inside(got[e], g.T @ v, (len(g) + 8) * U * (np.abs(g).T @ np.abs(v))), e
        start = end


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("T,H,F,E,k", [(203, 256, 208, 12, 3), (5, 128, 264, 8, 2), (700, 136, 640, 5, 2)])
def test_every_stage(T, H, F, E, k, fp8):
    torch.manual_seed(T)
    layer = moe_layer.MoeLayer(H, F, E, k, fp8=fp8, device=DEV)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16).requires_grad_()
    mask = torch.rand(T, device=DEV) > 0.1
    dout = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    seen, inner = [], layer.product

    def product(rows, w, offs):
        y = inner(rows, w, offs)
        rows.retain_grad()
        y.retain_grad()
        seen.append((rows, w, offs, y))
        return y

    layer.product = product
    out, loss, counts = layer(x, mask)
    (out * dout).sum().backward(retain_graph=True)
    (rows, up, offs, y1), (hidden, down, _, y2) = seen
    ends = offs.cpu().numpy()
    t = int(ends[-1])
    assert t == int(mask.sum()) * k == int(counts.sum())

    # forward: the rows in, the products, the rows out
    logits = (x @ layer.gate.t()).float().detach()
    route = mdg.moe_route_fwd(logits, k, token_mask=mask)
    plan = mdg.moe_plan(route.idx, E)
    assert torch.equal(plan.offs, offs) and torch.equal(route.loss, loss)
    assert torch.equal(rows, mdg.moe_dispatch_fwd(x.detach(), plan))
    check_product(h(rows), h(up), ends, y1.detach(), fp8)
    assert torch.equal(hidden, torch.nn.functional.silu(y1))
    check_product(h(hidden), h(down), ends, y2.detach(), fp8)
    assert torch.equal(out, mdg.moe_combine_fwd(y2.detach(), route.weight, plan))

    # backward
    dy2, dweight = mdg.moe_combine_bwd(dout, y2.detach(), route.weight, plan)
    assert torch.equal(y2.grad, dy2)
    check_product(h(y2.grad), h(down).transpose(0, 2, 1), ends, hidden.grad, fp8)
    check_wgrad(h(y2.grad), h(hidden), ends, down.grad)
    leaf = y1.detach().clone().requires_grad_()
    torch.nn.functional.silu(leaf).backward(hidden.grad)
    assert torch.equal(y1.grad, leaf.grad)
    check_product(h(y1.grad), h(up).transpose(0, 2, 1), ends, rows.grad, fp8)
    check_wgrad(h(y1.grad), h(rows), ends, up.grad)
    dlogits = mdg.moe_route_bwd(dweight, None, logits, route)
    xg, gate = x.detach().clone().requires_grad_(), layer.gate.detach().clone().requires_grad_()
    (xg @ gate.t()).float().backward(dlogits)
    assert torch.equal(layer.gate.grad, gate.grad)
    assert torch.equal(x.grad, xg.grad + mdg.moe_dispatch_bwd(rows.grad, plan))

    # the balance loss reaches the gate (and x) through the logits only
    before = [p.grad.clone() for p in (layer.up, layer.down)]
    x.grad = layer.gate.grad = None
    (0.5 * loss).backward()
    dlogits = mdg.moe_route_bwd(None, torch.full((), 0.5, device=DEV), logits, route)
    gate.grad = xg.grad = None
    (xg @ gate.t()).float().backward(dlogits)
    assert torch.equal(layer.gate.grad, gate.grad) and torch.equal(x.grad, xg.grad)
    assert all(torch.equal(p.grad, b) for p, b in zip((layer.up, layer.down), before))


@pytest.mark.parametrize("tokens", [1, 3, 120])
def test_every_stage_of_serving(tokens, monkeypatch):
    """The server's products on what they got, its other stages bit by bit."""
    H, F, E, k = 256, 208, 12, 3
    torch.manual_seed(tokens)
    layer = moe_layer.MoeLayer(H, F, E, k, device=DEV)
    server = moe_layer.MoeServer(layer)
    x = torch.randn((tokens, H), device=DEV).to(torch.bfloat16)
    seen, fwd = [], mdg.grouped_fp8_gemm_fwd

    def product(rows, wq, ws, offs):
        y = fwd(rows, wq, ws, offs)
        seen.append((rows, offs, y))
        return y

    monkeypatch.setattr(mdg, "grouped_fp8_gemm_fwd", product)
    out = server(x)
    (rows, offs, y1), (hidden, _, y2) = seen
    route = mdg.moe_route_fwd((x @ layer.gate.detach().t()).float(), k)
    plan = mdg.moe_plan(route.idx, E)
    ends = offs.cpu().numpy()
    assert int(ends[-1]) == tokens * k and torch.equal(plan.offs, offs)
    assert torch.equal(rows, mdg.moe_dispatch_fwd(x, plan))
    check_product(h(rows), h(layer.up), ends, y1, True)
    assert torch.equal(hidden, torch.nn.functional.silu(y1))
    check_product(h(hidden), h(layer.down), ends, y2, True)
    assert torch.equal(out, mdg.moe_combine_fwd(y2, route.weight, plan))
