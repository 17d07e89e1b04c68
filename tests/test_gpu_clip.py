"""The gradients' norm and clipping on the GPU against 64 bits: lists of every length
around the launches' limits, tensors of any size that start anywhere, both types
mixed, values whose squares overflow or vanish in fp32, norms that are not finite,
streams, graphs.

Tolerances (u = 2^-24): the norm is a sum in 64 bits rounded once, so u and a little.  The factor
is rounded once and so is each product in fp32: 2 u, then bf16's rounding (monotone: the
result lies between the roundings of the interval's ends).
"""
import math

import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import norm as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def make(lengths, seed, scale=1.0):
    """Tensors of these lengths, bf16 and fp32 in turn, starting anywhere in flat buffers."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for dt in (BF, FP):
        mine = [n for i, n in enumerate(lengths) if (i % 2 == 1) == (dt == FP)]
        flat = (torch.randn(sum(mine) + 1, generator=g, device=DEV) * scale).to(dt)[1:]
        out.append(list(torch.split(flat, mine)) if mine else [])
    return [out[i % 2][i // 2] for i in range(len(lengths))]


def check(before, after, got, max_norm, norm=None):
    want = ref.total_norm([f64(t) for t in before])
    if norm is None:
        assert abs(float(got) - want) <= 1.01 * U * want
        norm = want
    for a, b in zip(before, after):
        v = ref.clipped(f64(a), norm, max_norm)
        tol = 2.1 * U * np.abs(v)
        lo = np.nextafter((v - tol).astype(np.float32), np.float32(-np.inf))
        hi = np.nextafter((v + tol).astype(np.float32), np.float32(np.inf))
        if b.dtype == BF:
            lo, hi = (torch.from_numpy(x).to(BF).float().numpy() for x in (lo, hi))
        g = b.float().cpu().numpy()
        assert np.all((lo <= g) & (g <= hi))


@pytest.mark.parametrize("lengths", [
    [1], [0], [0, 0, 5], [7, 8], [1, 2, 3, 4, 5, 6, 7, 8, 9], [16384], [8192, 8192], [16383, 8191], [16385, 8193, 0, 40],
    [100_003, 1, 77], [3] * 163, [5] * 164, [3, 40] * 82 + [9], [7] * 246, [1] * 247, [1] * 300, [2] * 201, [6] * 202, [3, 1] * 168, [5] * 337, [1] * 673, [4] * 493, [2_000_003, 999], [40_000_001]])
@pytest.mark.parametrize("max_norm", [0.25, 1e9])
def test_clipped_in_place_and_into_others(lengths, max_norm):
    grads = make(lengths, len(lengths))
    before = [t.clone() for t in grads]
    norm = mdg.grad_norm(grads)
    outs = [torch.full_like(t, 7.0) for t in grads]
    got = mdg.clip_grads(grads, max_norm, out=outs)
    assert torch.equal(got, norm) and got.dtype == FP and got.dim() == 0
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check(before, outs, got, max_norm)
    assert torch.equal(mdg.clip_grads(grads, max_norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    if max_norm > 1e8:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_neighbours_in_a_flat_buffer_are_left():
    flat = torch.ones(100_000, device=DEV)
    half = torch.ones(100_000, dtype=BF, device=DEV)
    mine = [flat[3:40_000], flat[40_001:40_002], half[1:7], half[9:70_000]]
    mdg.clip_grads(mine, 1.0)
    for t, parts in ((flat, (slice(0, 3), slice(40_000, 40_001), slice(40_002, None))),
                     (half, (slice(0, 1), slice(7, 9), slice(70_000, None)))):
        for p in parts:
            assert torch.all(t[p] == 1.0)
    assert all(torch.all(t < 0.01) for t in mine)


def test_squares_that_overflow_or_vanish_in_fp32():
    big = torch.tensor([3e38, -3e37, 1e30], device=DEV)
    norm = mdg.clip_grads([big], 2.0)
    assert abs(float(norm) - math.sqrt(3e38 ** 2 + 3e37 ** 2 + 1e60)) <= 1e-6 * 3e38
    assert abs(float(big[0]) - 2.0 * 3e38 / float(norm)) < 1e-5
    small = torch.full((1000,), 1e-40, device=DEV)                      # subnormal
    assert abs(float(mdg.grad_norm([small])) - math.sqrt(1000) * float(small[0].double())) <= 1e-44
    low = torch.full((10,), 1e-30, dtype=BF, device=DEV)
    assert abs(float(mdg.grad_norm([low])) - math.sqrt(10) * float(low[0])) <= 1e-36
    # a norm past fp32's largest value is infinite: nothing is scaled
    huge = torch.full((100,), 3e38, device=DEV)
    assert float(mdg.clip_grads([huge], 1.0)) == float("inf") and torch.all(huge == 3e38)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    grads = make([1000, 40_001, 5], 3)
    grads[1][77] = bad
    before = [t.clone() for t in grads]
    outs = [torch.zeros_like(t) for t in grads]
    norm = mdg.clip_grads(grads, 0.1, out=outs)
    assert not math.isfinite(float(norm))
    mdg.clip_grads(grads, 0.1)
    for a, b, c in zip(grads, before, outs):
        bits = torch.int16 if a.dtype == BF else torch.int32
        assert torch.equal(a.view(bits), b.view(bits)) and torch.equal(c.view(bits), b.view(bits))


def test_zeros_and_the_smallest_and_largest_limits():
    zeros = [torch.zeros(10, device=DEV), torch.zeros(5, dtype=BF, device=DEV)]
    assert float(mdg.clip_grads(zeros, 0.0)) == 0.0 and all(torch.all(z == 0) for z in zeros)
    grads = make([100, 33], 1)
    before = [t.clone() for t in grads]
    mdg.clip_grads(grads, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    mdg.clip_grads(grads, 0)
    assert all(torch.all(t == 0) for t in grads)


def test_norm_of_several_lists():
    """Two lists as two processes would hold them: the norm of all, then each clipped by it."""
    parts = [make([1000, 300], 1), make([77, 50_000, 3], 2)]
    before = [[t.clone() for t in p] for p in parts]
    total = torch.stack([mdg.grad_norm(p).double() ** 2 for p in parts]).sum().sqrt().float()
    for p, b in zip(parts, before):
        assert mdg.clip_grads(p, 0.5, norm=total) is total
        check(b, p, total, 0.5, norm=float(total))


def test_shapes_strides_versions_and_sequences():
    g = torch.randn((64, 40), device=DEV)
    t = torch.randn((16, 24), device=DEV).t()                    # dense, in another order
    cl = torch.randn((2, 8, 4, 4), device=DEV).contiguous(memory_format=torch.channels_last)
    scalar = torch.randn((), device=DEV)
    p = torch.nn.Parameter(torch.randn(30, device=DEV))
    before = [x.detach().clone() for x in (g, t, cl, scalar, p)]
    versions = [x._version for x in (g, t, cl, scalar, p)]
    norm = mdg.clip_grads((x for x in (g, t, cl, scalar, p)), 1.0)
    want = torch.sqrt(sum(x.double().square().sum() for x in before))
    assert abs(float(norm) - float(want)) <= 1.01 * U * float(want)
    for x, b, v in zip((g, t, cl, scalar, p), before, versions):
        assert torch.allclose(x.detach(), b * (1.0 / want.float()), rtol=1e-6, atol=0) and x._version == v + 1
    grads = make([40, 50], 7)
    assert torch.equal(mdg.grad_norm(grads), mdg.grad_norm(tuple(grads)))
    twice = mdg.grad_norm([grads[0], grads[0]])                  # (each listed tensor counts)
    assert abs(float(twice) - math.sqrt(2) * ref.total_norm([f64(grads[0])])) <= 2 * U * float(twice)


def test_same_as_torch():
    params = [torch.nn.Parameter(torch.zeros(n, device=DEV)) for n in (1000, 37, 20_000)]
    for i, p in enumerate(params):
        p.grad = torch.randn(p.shape, device=DEV) * (i + 1)
    mine = [p.grad.clone() for p in params]
    norm = mdg.clip_grads(mine, 3.0)
    want = torch.nn.utils.clip_grad_norm_(params, 3.0)
    assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
    assert all(torch.allclose(a, p.grad, rtol=3e-6, atol=0) for a, p in zip(mine, params))


def test_other_stream_and_graph_replay():
    grads = make([5000, 70_001, 3, 9], 5)
    start = [t.clone() for t in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in grads]
    with torch.cuda.stream(side):
        norm = mdg.clip_grads(grads, 1.0, out=outs)
    side.synchronize()
    check(start, outs, norm, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gnorm = mdg.clip_grads(grads, 1.0, out=outs)
        mdg.clip_grads(grads, 0.5, norm=gnorm)
    for i in range(4):
        for t, n in zip(grads, make([5000, 70_001, 3, 9], 30 + i)):
            t.copy_(n)
        before = [t.clone() for t in grads]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(before, outs, gnorm, 1.0)
        check(before, grads, gnorm, 0.5)


def test_tensors_of_more_than_4_gib():
    n = 1_300_000_000
    g = torch.zeros(n, device=DEV)
    g[-5:] = 2.0
    g[0] = 1.0
    norm = mdg.clip_grads([g, torch.zeros(3, device=DEV)], 1.0)
    assert float(norm) == float(np.float32(math.sqrt(21.0)))
    by = np.float32(1.0 / (math.sqrt(21.0) + 1e-6))
    assert torch.all(g[-5:] == float(np.float32(2.0) * by)) and float(g[0]) == float(by) and int((g != 0).sum()) == 6


def test_refusals_on_the_device():
    a, b = torch.randn(64, device=DEV), torch.randn(64, dtype=BF, device=DEV)
    for error, call in (
            (ValueError, lambda: mdg.grad_norm([])),
            (ValueError, lambda: mdg.clip_grads([], 1.0)),
            (TypeError, lambda: mdg.grad_norm(a)),
            (TypeError, lambda: mdg.grad_norm([a, None])),
            (TypeError, lambda: mdg.grad_norm([a.half()])),
            (TypeError, lambda: mdg.grad_norm([a.double()])),
            (TypeError, lambda: mdg.grad_norm(5)),
            (ValueError, lambda: mdg.grad_norm([a, b.cpu()])),
            (ValueError, lambda: mdg.grad_norm([a[::2]])),
            (ValueError, lambda: mdg.grad_norm([a[:1].expand(9)])),
            (ValueError, lambda: mdg.clip_grads([a], -1.0)),
            (TypeError, lambda: mdg.clip_grads([a], float("nan"))),
            (TypeError, lambda: mdg.clip_grads([a], "1")),
            (TypeError, lambda: mdg.clip_grads([a], 1.0, norm=2.0)),
            (ValueError, lambda: mdg.clip_grads([a], 1.0, norm=torch.ones(1, device=DEV))),
            (ValueError, lambda: mdg.clip_grads([a, b], 1.0, out=[torch.empty_like(a)])),
            (ValueError, lambda: mdg.clip_grads([a], 1.0, out=[torch.empty_like(b)])),
            (ValueError, lambda: mdg.clip_grads([a.view(8, 8)], 1.0, out=[torch.empty_like(a).view(8, 8).t()])),
            (mdg.MdgError, lambda: mdg.clip_grads([a, a], 1.0)),
            (mdg.MdgError, lambda: mdg.clip_grads([a[:40], a[39:]], 1.0)),
            (mdg.MdgError, lambda: mdg.clip_grads([a[:32], a[32:]], 1.0, out=[a[32:], a[:32]])),
            (mdg.MdgError, lambda: mdg.clip_grads([a], 1.0, norm=a[3]))):
        before = a.clone()
        with pytest.raises(error):
            call()
        assert torch.equal(a, before)
