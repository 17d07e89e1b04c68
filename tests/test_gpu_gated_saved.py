"""What the differentiable gated feed-forward computes and keeps for its gradient: what
the wanted gradients read, whichever they are."""
import gc
import itertools

import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
M, K, F, N, E = 1024, 64, 512, 128, 4
NAMES = ("x", "w", "w_down")
WANTED = [w for w in itertools.product((False, True), repeat=3) if any(w)]
#: elements each of the operands has, and what each wanted gradient reads
SIZES = {"x": M * K, "w": E * 2 * F * K, "w_down": E * N * F, "h": M * F, "gate_up": 2 * M * F}
READ = {"x": {"w", "w_down", "gate_up"}, "w": {"x", "w_down", "gate_up"}, "w_down": {"h"}}


def inputs():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()
    return {"x": r(M, K), "w": r(E, 2 * F, K), "w_down": r(E, N, F)}, r(M, N)


OFFS = torch.tensor([300, 300, 700, 1000], dtype=torch.int32, device=DEV) if torch.cuda.is_available() else None


def leaves(wanted):
    v, dy = inputs()
    return {k: t.requires_grad_(on) for (k, t), on in zip(v.items(), wanted)}, dy


def run(v, **kw):
    return mdg.grouped_gated_ffn(v["x"], v["w"], v["w_down"], OFFS, **kw)


@pytest.mark.parametrize("wanted", WANTED)
def test_the_wanted_gradients_are_those_of_all(wanted):
    every, dy = leaves((True,) * 3)
    run(every).backward(dy)
    v, _ = leaves(wanted)
    y = run(v)
    asked = torch.autograd.grad(y, [v[k] for k in NAMES if v[k].requires_grad], dy, retain_graph=True)
    assert all(torch.equal(g, every[k].grad) for g, k in zip(asked, [k for k in NAMES if v[k].requires_grad]))
    y.backward(dy)
    for k in NAMES:
        assert v[k].grad is None if not v[k].requires_grad else torch.equal(v[k].grad, every[k].grad)
    # one of them at a time, from a graph that keeps what all need
    y = run(every)
    for k in NAMES:
        g, = torch.autograd.grad(y, every[k], dy, retain_graph=True)
        assert torch.equal(g, every[k].grad)


@pytest.mark.parametrize("wanted", WANTED)
def test_added_into_main_grad(wanted):
    got = []
    for on in ((True,) * 3, wanted):
        v, dy = leaves(on)
        for k in ("w", "w_down"):
            v[k].main_grad = torch.ones(v[k].shape, device=DEV)
        run(v, fuse_wgrad_accumulation=True).backward(dy)
        got.append(v)
    every, v = got
    assert v["x"].grad is None if not wanted[0] else torch.equal(v["x"].grad, every["x"].grad)
    for k, on in zip(("w", "w_down"), wanted[1:]):
        assert torch.equal(v[k].main_grad, every[k].main_grad if on else torch.ones_like(v[k].main_grad))


@pytest.mark.parametrize("wanted", WANTED)
def test_only_what_they_read_is_kept(wanted):
    """Of the inputs: changed in place, the others do not matter.  Of the call's own: the
    memory held behind it."""
    read = set().union(*(READ[k] for k, on in zip(NAMES, wanted) if on))
    run(leaves(wanted)[0])
    v, dy = leaves(wanted)
    gc.collect()
    before = torch.cuda.memory_allocated()
    y = run(v)
    held = torch.cuda.memory_allocated() - before - y.numel() * 2
    assert held == 2 * sum(SIZES[k] for k in ("h", "gate_up") if k in read)
    want = torch.autograd.grad(y, [t for t in v.values() if t.requires_grad], dy, retain_graph=True)
    with torch.no_grad():
        for k in NAMES:
            if k not in read:
                v[k].fill_(float("nan"))
    got = torch.autograd.grad(y, [t for t in v.values() if t.requires_grad], dy, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():
        for k in NAMES:
            if k in read:
                v[k].mul_(1.0)
    if read & set(NAMES):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward(dy)
