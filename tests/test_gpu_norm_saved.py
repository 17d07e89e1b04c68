"""What a differentiable block norm keeps for its gradient: not out where only a norm
of it would read it."""
import gc

import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H = 512, 1024


def rows(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn((T, H), generator=g, device=DEV).bfloat16()


CASES = [dict(), dict(gate=True), dict(post=True), dict(gate=True, post=True)]


def call(how, weight=False):
    leaves = {"residual": rows(1), "y": rows(2)}
    if how.get("gate"):
        leaves["gate"] = rows(3)[:, 0].float()
    if how.get("post"):
        leaves["post_weight"] = rows(4)[0].float()
    if weight:
        leaves["weight"] = rows(5)[0].float()
    leaves = {k: t.clone().requires_grad_() for k, t in leaves.items()}
    out, normed = mdg.block_norm(scale=0.5, **leaves)
    return leaves, out, normed


@pytest.mark.parametrize("how", CASES)
def test_out_may_change_in_place_without_a_norm_of_it(how):
    (a, out, _), (b, changed, _) = call(how), call(how)
    after = changed * 1.0
    with torch.no_grad():
        changed.mul_(3.0)
    out.backward(rows(6))
    after.backward(rows(6))
    assert all(torch.equal(a[k].grad, b[k].grad) for k in a)


def test_out_is_kept_where_its_norm_reads_it():
    _, out, normed = call({}, weight=True)
    with torch.no_grad():
        out.mul_(3.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        normed.backward(rows(6))


def test_out_is_freed():
    call({})
    leaves, out, _ = call({})
    after = out * 1.0
    gc.collect()
    held = torch.cuda.memory_allocated()
    del out
    assert torch.cuda.memory_allocated() == held - T * H * 2
    after.backward(rows(6))
    assert torch.equal(leaves["residual"].grad, rows(6)) and torch.equal(leaves["y"].grad, rows(6) * 0.5)
