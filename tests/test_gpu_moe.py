"""Routing, the plan, dispatch and combine on the GPU against the 64-bit oracle:
sizes around every layout change of the kernels, ties, masked rows and experts,
NaN and infinities, gradients against the formula and against differences.

Tolerances (u = 2^-24, the fp32 rounding unit): a softmax entry carries the
rounding of l - max (|l - max| <= 40 here: 40 u relative), exp and division (8 u)
and a sum over at most 22 partial steps: 80 u.  The loss adds at most 2^11
terms in sequence: 2048 u + 80 u.  A sum of n fp32 products is off by at most
(n + 2) u sum |products|.  A bf16 result has to lie between the bf16 roundings of
the two ends of that interval (rounding is monotone).
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import moe as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
P_TOL, LOSS_TOL = 80 * U, 2128 * U


def inside(got, want, tol):
    """got (bf16 or fp32 tensor) within tol of want (fp64), rounded as got's type rounds."""
    lo = np.nextafter((want - tol).astype(np.float32), np.float32(-np.inf))
    hi = np.nextafter((want + tol).astype(np.float32), np.float32(np.inf))
    if got.dtype == torch.bfloat16:
        lo, hi = (torch.from_numpy(v).to(torch.bfloat16).float().numpy() for v in (lo, hi))
    g = got.float().cpu().numpy()
    return bool(np.all((lo <= g) & (g <= hi)))


def make_logits(T, E, dtype, seed, grid=None, masked=False):
    rng = np.random.default_rng(seed)
    l = rng.normal(0, 2, (T, E)) + rng.normal(0, 1, (1, E))
    if grid:                                   # many equal logits
        l = np.round(l * grid) / grid
    if masked:
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[rng.random(T) < 0.2] = -np.inf
    return torch.from_numpy(l).to(dtype).to(DEV)


def check_route(logits, k, normalize, mask, r):
    host = logits.float().cpu().numpy()
    w, idx, counts, loss, balance = ref.route(host, k, normalize, None if mask is None else mask.cpu().numpy())
    assert np.array_equal(r.idx.cpu().numpy(), idx)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    got = r.weight.cpu().numpy()
    assert np.all(np.abs(got - w) <= P_TOL * np.abs(w) + 1e-37)
    assert np.all(np.abs(r.balance.cpu().numpy() - balance) <= 2 * U * balance)
    assert abs(float(r.loss) - loss) <= LOSS_TOL * abs(loss)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (7, 3, 3), (130, 8, 8), (1000, 9, 4), (65, 16, 16), (333, 30, 30), (200, 32, 32), (61, 60, 6),
    (999, 64, 8), (257, 128, 4), (1, 256, 8), (515, 256, 32), (100, 257, 7), (40, 512, 8), (33, 513, 8),
    (70, 1000, 3), (129, 1024, 32), (8193, 8, 2), (4099, 64, 8), (3001, 256, 8), (2050, 600, 2)])
def test_route_sizes(T, E, k, dtype):
    for masked, normalize in ((False, True), (True, False)):
        logits = make_logits(T, E, dtype, T + E, grid=4 if T % 2 else None, masked=masked)
        mask = None
        if masked:
            mask = torch.from_numpy(np.random.default_rng(1).random(T) > 0.2).to(DEV)
        r = mdg.moe_route_fwd(logits, k, normalize=normalize, token_mask=mask)
        check_route(logits, k, normalize, mask, r)
        again = mdg.moe_route_fwd(logits, k, normalize=normalize, token_mask=mask)
        for a, b in zip(r, again):
            assert torch.equal(a, b)


def test_route_no_tokens_and_nothing_routed():
    r = mdg.moe_route_fwd(torch.empty((0, 16), device=DEV), 2)
    assert r.weight.shape == (0, 2) and int(r.counts.abs().sum()) == 0 and float(r.loss) == 0.0
    assert float(r.balance.abs().sum()) == 0.0
    logits = torch.full((9, 16), float("-inf"), device=DEV)
    r = mdg.moe_route_fwd(logits, 3)
    assert torch.all(r.idx == -1) and torch.all(r.weight == 0) and float(r.loss) == 0.0
    dl = mdg.moe_route_bwd(torch.full((9, 3), float("nan"), device=DEV), torch.ones((), device=DEV), logits, r)
    assert torch.all(dl == 0)
    r = mdg.moe_route_fwd(torch.randn((9, 16), device=DEV), 3, token_mask=torch.zeros(9, dtype=torch.bool, device=DEV))
    assert torch.all(r.idx == -1) and int(r.counts.sum()) == 0


@pytest.mark.parametrize("E", [8, 24, 256, 1024])
def test_route_special_values(E):
    """The type's lowest value is an ordinary logit, zeros of both signs tie, and
    a NaN or +inf stays in its row (and in the loss)."""
    low = torch.finfo(torch.float32).min
    l = torch.randn((6, E), device=DEV)
    l[0] = low
    l[1, :] = low
    l[1, E // 2] = float("-inf")
    l[2, 0::2] = 0.0
    l[2, 1::2] = -0.0
    r = mdg.moe_route_fwd(l, 4)
    check_route(l, 4, True, None, r)
    assert r.idx[2].tolist() == [0, 1, 2, 3] and r.idx[0].tolist() == [0, 1, 2, 3]
    l[3, 5] = float("nan")
    l[4, 2] = float("inf")
    r = mdg.moe_route_fwd(l, 4)
    assert r.idx[3, 0] == 5 and r.idx[4, 0] == 2
    assert torch.isnan(r.weight[3]).all() and torch.isnan(r.weight[4, 0])
    assert torch.isfinite(r.weight[[0, 1, 2, 5]]).all() and torch.isnan(r.loss)
    dl = mdg.moe_route_bwd(torch.randn((6, 4), device=DEV), None, l, r)
    assert torch.isfinite(dl[[0, 1, 2, 5]]).all() and torch.isnan(dl[3]).any()


def grad_bound(host, k, dw, g, normalize, mask):
    """Sum of the magnitudes of a gradient entry's parts."""
    w, idx, _, _, a = ref.route(host, k, normalize, mask)
    p = ref._softmax(host, mask)[2]
    inner = np.abs(w * dw).sum(axis=1, keepdims=True)
    m = p * (g * a + g * (p * a).sum(axis=1, keepdims=True) + inner)
    for t in range(host.shape[0]):
        s = idx[t] >= 0
        m[t, idx[t][s]] += w[t][s] * (np.abs(dw[t][s]) + inner[t])
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 3, 2), (300, 8, 2), (77, 12, 9), (64, 30, 30), (129, 64, 8), (200, 128, 4),
                                   (131, 256, 8), (50, 300, 17), (40, 513, 8), (33, 1024, 32), (2049, 60, 6)])
def test_route_gradient(T, E, k, dtype):
    rng = np.random.default_rng(E)
    for masked, normalize in ((False, True), (True, False), (True, True)):
        logits = make_logits(T, E, dtype, T * E, masked=masked)
        mask = torch.from_numpy(rng.random(T) > 0.2).to(DEV) if masked else None
        r = mdg.moe_route_fwd(logits, k, normalize=normalize, token_mask=mask)
        dw = rng.normal(size=(T, k)).astype(np.float32)
        g = 0.37
        dl = mdg.moe_route_bwd(torch.from_numpy(dw).to(DEV), torch.full((), g, device=DEV), logits, r,
                               normalize=normalize)
        host, hm = logits.float().cpu().numpy(), None if mask is None else mask.cpu().numpy()
        want = ref.route_grad(host, k, dw, float(np.float32(g)), normalize, hm)
        tol = 4 * P_TOL * grad_bound(host, k, dw, g, normalize, hm)
        assert inside(dl, want, tol)
        none = mdg.moe_route_bwd(None, None, logits, r, normalize=normalize)
        assert torch.all(none == 0)


def test_route_gradient_against_differences():
    """Central differences of the GPU's own forward (fp32: step 2^-6, so the
    difference quotient is good to about its third-order term, 2^-12 relative to
    the parts, and the forward's rounding over the step, 80 u * 2^7)."""
    T, E, k = 6, 16, 3
    h = 2.0 ** -6
    for normalize in (True, False):
        l = make_logits(T, E, torch.float32, 6)
        top = torch.sort(l, dim=1, descending=True).values
        assert float((top[:, :-1] - top[:, 1:])[:, k - 1].min()) > 2 * h      # the choice does not change
        c = torch.randn((T, k), device=DEV)

        def f(x):
            r = mdg.moe_route_fwd(x, k, normalize=normalize)
            order = torch.argsort(r.idx, dim=1)                               # a slot may swap with its neighbour
            return float((torch.gather(r.weight, 1, order) * c).sum() + 0.5 * r.loss)

        x = l.clone().requires_grad_()
        r = mdg.moe_route(x, k, normalize=normalize)
        order = torch.argsort(r.idx, dim=1)
        ((torch.gather(r.weight, 1, order) * c).sum() + 0.5 * r.loss).backward()
        for t, e in [(0, 0), (1, 5), (2, int(r.idx[2, 0])), (3, int(r.idx[3, 1])), (5, 15), (4, int(r.idx[4, 2]))]:
            d = torch.zeros_like(l)
            d[t, e] = h
            got = (f(l + d) - f(l - d)) / (2 * h)
            assert abs(got - float(x.grad[t, e])) <= 2.0 ** -10 * float(c.abs().sum())


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (3, 2, 8), (64, 1, 1), (100, 8, 64), (511, 8, 9), (513, 8, 256), (2049, 2, 8),
                                   (1025, 8, 1024), (5000, 4, 600), (9000, 1, 3), (4100, 32, 77)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + k)
    for case in ("mixed", "one", "none"):
        idx = rng.integers(-2, E + 2, (T, k)) if case == "mixed" else np.full((T, k), E - 1 if case == "one" else -1)
        offs, dest = ref.plan(idx, E)
        pl = mdg.moe_plan(torch.from_numpy(idx.astype(np.int32)).to(DEV), E)
        assert np.array_equal(pl.offs.cpu().numpy(), offs)
        assert np.array_equal(pl.dest.cpu().numpy(), dest)


ROW_CASES = [(1, 1, 8, 1), (3, 2, 4096, 8), (5, 3, 16, 4), (70, 8, 2048, 64), (33, 2, 1000, 7), (129, 4, 2056, 16),
             (17, 9, 512, 20), (66, 32, 264, 40), (9, 8, 7168, 128), (255, 1, 64, 3)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H,E", ROW_CASES)
def test_rows_forward_and_gradients(T, k, H, E, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(T * k + H)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)
    idx = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    w = rnd(T, k)
    x, dout = rnd(T, H).to(dtype), rnd(T, H).to(dtype)
    y, dxp = rnd(T * k, H).to(dtype), rnd(T * k, H).to(dtype)
    pl = mdg.moe_plan(idx, E)
    end = int(pl.offs[-1])
    y[end:] = float("nan")                              # rows no slot has are never read
    dxp[end:] = float("nan")
    dest = pl.dest.cpu().numpy()
    h = lambda t: t.double().cpu().numpy()

    xp = mdg.moe_dispatch_fwd(x, pl)
    assert np.array_equal(h(xp), ref.dispatch(h(x), dest))

    def close(got, want, size, n):
        assert inside(got, want, (n + 2) * U * size)

    yz = np.nan_to_num(h(y))
    out = mdg.moe_combine_fwd(y, w, pl)
    close(out, ref.combine(yz, h(w), dest), ref.combine(np.abs(yz), np.abs(h(w)), dest), k)
    dx = mdg.moe_dispatch_bwd(dxp, pl)
    dz = np.nan_to_num(h(dxp))
    close(dx, ref.dispatch_grad(dz, dest), ref.dispatch_grad(np.abs(dz), dest), k)
    dy, dw = mdg.moe_combine_bwd(dout, y, w, pl)
    want_dy, want_dw = ref.combine_grad(h(dout), yz, h(w), dest)
    close(dy, want_dy, np.abs(want_dy), 1)
    size = ref.combine_grad(np.abs(h(dout)), np.abs(yz), h(w), dest)[1]
    assert np.all(np.abs(h(dw) - want_dw) <= (H + 2) * U * size)
    for a, b in ((out, mdg.moe_combine_fwd(y, w, pl)), (dw, mdg.moe_combine_bwd(dout, y, w, pl)[1])):
        assert torch.equal(a, b)


def test_rows_autograd_and_differences():
    T, k, H, E = 12, 3, 40, 5
    idx = torch.randint(-1, E, (T, k), device=DEV, dtype=torch.int32)
    pl = mdg.moe_plan(idx, E)
    x = torch.randn((T, H), device=DEV, requires_grad=True)
    w = torch.rand((T, k), device=DEV, requires_grad=True)
    c = torch.randn((T, H), device=DEV)
    f = lambda x, w: (mdg.moe_combine(torch.tanh(mdg.moe_dispatch(x, pl)), w, pl) * c).sum()
    f(x, w).backward()
    h = 2.0 ** -7                                        # the third-order term: h^2 / 6 of the parts
    with torch.no_grad():
        for t, i in [(0, 0), (3, 17), (11, 39)]:
            d = torch.zeros_like(x)
            d[t, i] = h
            got = float(f(x + d, w) - f(x - d, w)) / (2 * h)
            assert abs(got - float(x.grad[t, i])) <= 2e-3 * (1 + abs(float(x.grad[t, i])))
        for t, j in [(0, 0), (5, 1), (11, 2)]:
            d = torch.zeros_like(w)
            d[t, j] = h
            got = float(f(x, w + d) - f(x, w - d)) / (2 * h)
            assert abs(got - float(w.grad[t, j])) <= 2e-3 * (1 + abs(float(w.grad[t, j])))


def test_malformed_plan_stays_in_bounds():
    """dest entries outside the rows are slots without one; offs are clamped."""
    T, k, H = 4, 2, 64
    dest = torch.tensor([[0, 99], [-7, 1], [2, 2 ** 30], [8, 3]], dtype=torch.int32, device=DEV)
    x = torch.randn((T, H), device=DEV, dtype=torch.bfloat16)
    for end, zero_from in ((4, 4), (2 ** 30, 8), (8, 8)):
        pl = mdg.MoePlan(torch.tensor([1, end], dtype=torch.int32, device=DEV), dest)
        rows = mdg.moe_dispatch_fwd(x, pl)
        assert torch.equal(rows[:4], x[[0, 1, 2, 3]]) and torch.all(rows[zero_from:] == 0)
        out = mdg.moe_combine_fwd(rows, torch.ones((T, k), device=DEV), pl)
        assert torch.equal(out, x)


def test_other_stream_and_graph_replay():
    """The calls run on the current stream and, captured, give the eager bits on
    every replay with new values in the same tensors."""
    T, E, k, H = 300, 64, 8, 256
    s = torch.cuda.Stream()
    logits = torch.randn((T, E), device=DEV)
    x = torch.randn((T, H), device=DEV, dtype=torch.bfloat16)

    def layer():
        r = mdg.moe_route_fwd(logits, k)
        pl = mdg.moe_plan(r.idx, E)
        rows = mdg.moe_dispatch_fwd(x, pl)
        return r.weight, r.loss, pl.offs, rows, mdg.moe_combine_fwd(rows, r.weight, pl)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for seed in range(3):
        torch.manual_seed(seed)
        logits.copy_(torch.randn_like(logits))
        x.copy_(torch.randn((T, H), device=DEV).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, layer()):
            assert torch.equal(a, b)


def test_rows_of_more_than_4_gib():
    """Copies against indexing, sums at sampled tokens against fp64."""
    T, k, E, H = 42_000, 8, 16, 7168
    assert T * k * H * 2 > 2 ** 32
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    idx = torch.randint(-1, E, (T, k), generator=gen, device=DEV, dtype=torch.int32)
    weight = torch.rand((T, k), generator=gen, device=DEV)
    x = torch.randn((T, H), generator=gen, device=DEV, dtype=torch.bfloat16)
    plan = mdg.moe_plan(idx, E)
    have = plan.dest >= 0
    assert torch.equal(have, idx >= 0) and int(plan.offs[-1]) == int(have.sum())
    rows = mdg.moe_dispatch_fwd(x, plan)
    for j in range(k):
        t = have[:, j].nonzero()[:, 0]
        assert torch.equal(rows[plan.dest[t, j].long()], x[t])
    assert not rows[int(plan.offs[-1]):].any()

    y = rows
    out, dx = mdg.moe_combine_fwd(y, weight, plan), mdg.moe_dispatch_bwd(y, plan)
    dy, dweight = mdg.moe_combine_bwd(x, y, weight, plan)
    assert not dy[int(plan.offs[-1]):].any()
    at = torch.cat([torch.arange(0, T, 691, device=DEV), torch.arange(T - 40, T, device=DEV)])
    d, wt, xt = plan.dest[at], weight[at].double().cpu().numpy(), x[at].double().cpu().numpy()
    real = (d >= 0).cpu().numpy()
    ys = y[d.clamp(min=0).long()].double().cpu().numpy() * real[:, :, None]
    terms = wt[:, :, None] * ys
    assert inside(out[at], terms.sum(axis=1), (k + 2) * U * np.abs(terms).sum(axis=1))
    assert inside(dx[at], ys.sum(axis=1), (k + 2) * U * np.abs(ys).sum(axis=1))
    prod = xt[:, None, :] * ys
    assert inside(dweight[at], prod.sum(axis=2), (H + 2) * U * np.abs(prod).sum(axis=2))
    got = dy[d.clamp(min=0).long()]
    want = (wt[:, :, None] * xt[:, None, :])
    tol = 2 * U * np.abs(want)
    got[~torch.from_numpy(real).to(DEV)] = 0
    assert inside(got, want * real[:, :, None], tol * real[:, :, None])


def test_binding_refusals_on_the_device():
    l = torch.randn((6, 8), device=DEV)
    x = torch.randn((6, 64), device=DEV)
    r = mdg.moe_route_fwd(l, 2)
    plan = mdg.moe_plan(r.idx, 8)
    y = mdg.moe_dispatch_fwd(x, plan)
    other = mdg.moe_plan(r.idx[:5].contiguous(), 8)
    mask = torch.ones(6, dtype=torch.bool, device=DEV)
    strided = torch.randn((64, 6), device=DEV).t()
    for kind, match, f in (
            (ValueError, "top_k must be between 1", lambda: mdg.moe_route_fwd(l, 9)),
            (ValueError, "top_k must be between 1", lambda: mdg.moe_route_fwd(l, 0)),
            (TypeError, "top_k must be an int", lambda: mdg.moe_route_fwd(l, 2.0)),
            (TypeError, "top_k must be an int", lambda: mdg.moe_route_fwd(l, True)),
            (TypeError, "normalize must be a bool", lambda: mdg.moe_route_fwd(l, 2, normalize=1)),
            (ValueError, "2-D, got shape \\(8,\\)", lambda: mdg.moe_route_fwd(l[0], 2)),
            (ValueError, "6 entries", lambda: mdg.moe_route_fwd(l, 2, token_mask=mask[:5])),
            (TypeError, "torch.bool, got torch.int32", lambda: mdg.moe_route_fwd(l, 2, token_mask=mask.int())),
            (ValueError, "ROCm device", lambda: mdg.moe_route_fwd(l, 2, token_mask=mask.cpu())),
            (ValueError, "contiguous", lambda: mdg.moe_route_fwd(l[:, ::2], 2)),
            (ValueError, "does not belong", lambda: mdg.moe_route_bwd(r.weight, r.loss, l[:5], r)),
            (ValueError, "dweight must have shape \\(6, 2\\)", lambda: mdg.moe_route_bwd(r.weight[:5], None, l, r)),
            (ValueError, "dloss must be 0-D", lambda: mdg.moe_route_bwd(None, r.balance, l, r)),
            (TypeError, "num_experts must be an int", lambda: mdg.moe_plan(r.idx, 8.0)),
            (ValueError, "at least one", lambda: mdg.moe_plan(r.idx, 0)),
            (mdg.MdgError, "status 2", lambda: mdg.moe_plan(r.idx, 5000)),
            (OverflowError, None, lambda: mdg.moe_plan(r.idx, 1 << 70)),
            (mdg.MdgError, "status 2", lambda: mdg.moe_plan(r.idx, 1 << 40)),
            (TypeError, "torch.int32, got torch.int64", lambda: mdg.moe_plan(r.idx.long(), 8)),
            (TypeError, "bfloat16 or float32, got torch.float64", lambda: mdg.moe_dispatch_fwd(x.double(), plan)),
            (ValueError, "x must have 5 rows, got 6", lambda: mdg.moe_dispatch_fwd(x, other)),
            (ValueError, "contiguous", lambda: mdg.moe_dispatch_fwd(strided, plan)),
            (mdg.MdgError, "status 2", lambda: mdg.moe_dispatch_fwd(x[:, :3].contiguous(), plan)),
            (ValueError, "drows must have 10 rows", lambda: mdg.moe_dispatch_bwd(y, other)),
            (ValueError, "weight must have shape \\(6, 2\\)", lambda: mdg.moe_combine_fwd(y, r.weight[:5], plan)),
            (TypeError, "weight must be torch.float32", lambda: mdg.moe_combine_fwd(y, r.weight.bfloat16(), plan)),
            (TypeError, "dout must be torch.float32, got torch.bfloat16",
             lambda: mdg.moe_combine_bwd(x.bfloat16(), y, r.weight, plan)),
            (ValueError, "dout must have shape \\(6, 64\\)", lambda: mdg.moe_combine_bwd(x[:5], y, r.weight, plan))):
        with pytest.raises(kind, match=match):
            f()
    assert isinstance(r, mdg.MoeRoute) and isinstance(plan, mdg.MoePlan)
    torch.cuda.synchronize()


def test_outputs_are_tensors_of_their_own():
    """The small outputs share an allocation, not their values or versions."""
    l = torch.randn((5, 3), device=DEV)
    r = mdg.moe_route_fwd(l, 2)
    kept = [t.clone() for t in r]
    for i, t in enumerate(r):
        assert t.data_ptr() % 256 == 0 and t.is_contiguous() and t._version == 0
        t.fill_(1)
        for j, u in enumerate(r):
            assert torch.equal(u, kept[j]) or j <= i
    assert [t._version for t in r] == [1] * 5
    plan = mdg.moe_plan(r.idx, 3)
    dest = plan.dest.clone()
    plan.offs.zero_()
    assert torch.equal(plan.dest, dest) and plan.dest._version == 0
