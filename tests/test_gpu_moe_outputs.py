"""The outputs of a routing call or a plan are tensors of their own: they can be
saved together, one that is kept keeps nothing else, and what is done to one's
storage does not reach another."""
import io

import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def outputs(T, E, k):
    r = mdg.moe_route_fwd(torch.randn((T, E), device=DEV), k)
    return list(r) + list(mdg.moe_plan(r.idx, E))


SIZES = [(1, 256, 8), (3, 8, 2), (5000, 64, 8)]


@pytest.mark.parametrize("T,E,k", SIZES)
def test_outputs_can_be_saved_together(T, E, k):
    out = outputs(T, E, k)
    f = io.BytesIO()
    torch.save(out, f)
    f.seek(0)
    back = torch.load(f, weights_only=True)
    assert len(back) == len(out)
    for a, b in zip(out, back):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("T,E,k", SIZES)
def test_an_output_keeps_only_its_own_memory(T, E, k):
    out = outputs(T, E, k)
    for t in out:
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
    assert len({t.untyped_storage().data_ptr() for t in out}) == len(out)


def test_freeing_one_storage_leaves_the_others():
    out = outputs(5, 16, 3)
    kept = [t.clone() for t in out]
    sizes = [t.untyped_storage().nbytes() for t in out]
    out[0].untyped_storage().resize_(0)
    # (on the host first: a value is read only where its memory is still there)
    assert [t.untyped_storage().nbytes() for t in out[1:]] == sizes[1:] and all(sizes[1:])
    for t, u in zip(out[1:], kept[1:]):
        assert torch.equal(t, u)


@pytest.mark.parametrize("T,E,k", SIZES)
def test_differentiable_outputs_too(T, E, k):
    l = torch.randn((T, E), device=DEV, requires_grad=True)
    r = mdg.moe_route(l, k)
    assert r.loss.untyped_storage().nbytes() == 4
    f = io.BytesIO()
    torch.save([t.detach() for t in r], f)
    (r.weight.square().sum() + r.loss).backward()
    assert torch.isfinite(l.grad).all()
