"""Gradient lists whose partial sums are more than a scaling workgroup's threads load at
once (four each): several launches, whole in the first ones.  Bounds: test_gpu_clip.py's."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from test_gpu_clip import DEV, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[60_000] * 400, [40_000, 60_001, 3, 100_000] * 260, [17_000] * 1100])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_more_partial_sums_than_four_a_thread(lengths, max_norm):
    grads = make(lengths, len(lengths))
    before = [t.clone() for t in grads]
    outs = [torch.full_like(t, 7.0) for t in grads]
    norm = mdg.grad_norm(grads)
    got = mdg.clip_grads(grads, max_norm, out=outs)
    assert torch.equal(got, norm)
    check(before, outs, got, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert torch.equal(mdg.clip_grads(grads, max_norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_a_captured_list_of_many_launches():
    grads = make([30_000] * 700, 3)
    outs = [torch.empty_like(t) for t in grads]
    mdg.clip_grads(grads, 1.0, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mdg.clip_grads(grads, 1.0, out=outs)
    for i in range(3):
        for t, n in zip(grads, make([30_000] * 700, 10 + i)):
            t.copy_(n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept, now = [t.clone() for t in outs], norm.clone()
        want = [torch.empty_like(t) for t in grads]
        assert torch.equal(mdg.clip_grads(grads, 1.0, out=want), now)
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def launches(f, name):
    f()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        f()
        torch.cuda.synchronize()
    return sum(name in e.name for e in prof.events())


@pytest.mark.parametrize("lengths,adds", [([60_000] * 100, 0), ([500] * 700, 0), ([60_000] * 400, 1), ([17_000] * 1100, 1)])
def test_many_sums_are_added_up_once(lengths, adds):
    """Not by every workgroup of every scaling launch, whose cost would grow with the list's square."""
    grads = make(lengths, 1)
    outs = [torch.empty_like(t) for t in grads]
    for call in (lambda: mdg.clip_grads(grads, 1.0), lambda: mdg.clip_grads(grads, 1.0, out=outs)):
        assert launches(call, "clip_finish_kernel") == adds
