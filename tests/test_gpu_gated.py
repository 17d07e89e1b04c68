"""The gated feed-forward on the GPU against the 64-bit oracle: every output element at
sizes around the kernels' tiles and stages, empty groups, rows of no group, special
values, gradients against the formula and against differences, streams, graphs.
Bounds: tests/_gated.py."""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import gated as ref
from _gated import DEV, U, bf16, check_dgrad, check_fwd, f64, inside, offsets, variant_of

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def operands(sizes, f, k, n, seed, pad=0):
    g, m, e = gen(seed), sum(sizes) + pad, len(sizes)
    return (bf16((m, k), g), bf16((e, 2 * f, k), g, 2 / k ** 0.5), bf16((m, n), g), bf16((e, n, f), g, 1 / f ** 0.5),
            offsets(sizes))


SIZES = [
    ([1], 8, 8, 8), ([2, 0, 3], 16, 24, 40), ([0, 0], 32, 32, 32), ([7, 1, 0, 30], 136, 72, 64), ([16, 17], 64, 128, 8),
    ([33, 64, 65, 0, 1], 72, 200, 136), ([300, 0, 257, 1], 128, 96, 264), ([256, 512], 256, 64, 256),
    ([255, 0, 0, 513], 264, 1000, 520), ([1] * 40 + [0] * 20 + [3] * 4, 40, 64, 72), ([600], 1000, 136, 1000),
    ([2, 100, 1, 0, 48], 520, 2000, 2000), ([3000], 128, 64, 64), ([2100, 2050], 384, 512, 128),
]

# sizes whose tiles fill the GPU: the 256-row tile kernels in all of their forms
RAGGED = [513, 0, 1100, 1, 700, 257]
SIZES += [(RAGGED, 1608, 40, 24), (RAGGED, 1608, 64, 96), (RAGGED, 1672, 200, 64), ([2100, 300], 2048, 96, 40),
          ([2100, 0, 1900], 2056, 32, 8), ([255, 260, 256, 770], 2568, 328, 264), ([2600], 2176, 1000, 64), ([90, 20], 72, 40, 2056),
          (RAGGED, 1608, 1056, 2080), (RAGGED, 1608, 1064, 2056), ([8200], 2312, 40, 24), ([130, 65], 328, 72, 2600)]
# the middle kernel's two tiles, whole and partial, in one group and several
SIZES += [([64], 32, 64, 64), ([65, 0, 63, 128], 96, 136, 128), ([129], 40, 328, 72), ([64, 64, 1], 264, 2048, 192),
          ([1500, 700, 3], 1096, 136, 264), ([1281], 1928, 200, 128)]
FORMS = {("fwd", "small"), ("fwd", "mid", 64), ("fwd", "mid", 128), ("dgrad", "mid", 64), ("dgrad", "mid", 128)} | {
    ("fwd", "tile", False, False), ("fwd", "tile", False, True), ("fwd", "tile", True, True),
    ("dgrad", "tile", False, True), ("dgrad", "tile", True, True)}


def test_the_sizes_reach_every_form():
    got = set()
    for sizes, f, k, n in SIZES:
        got |= {variant_of("fwd", sum(sizes), len(sizes), k, f), variant_of("dgrad", sum(sizes), len(sizes), n, f)}
    assert FORMS <= got, FORMS - got


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("sizes,f,k,n", SIZES)
def test_products(sizes, f, k, n, name):
    x, w, dy, w2, offs = operands(sizes, f, k, n, sum(sizes) + f)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=True)
    check_fwd(x, w, offs, name, r.h, r.gate_up, sum(sizes))
    alone = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name)
    assert alone.gate_up is None and torch.equal(alone.h, r.h)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs, activation=name)
    check_dgrad(dy, w2, r.gate_up, offs, name, d, sum(sizes))
    again = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=True)
    assert torch.equal(again.h, r.h) and torch.equal(again.gate_up, r.gate_up)
    assert torch.equal(mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs, activation=name), d)


def test_random_sizes():
    rng = np.random.default_rng(11)
    for i in range(24):
        e = int(rng.integers(1, 24))
        sizes = (rng.integers(0, 2, e) * np.exp(rng.uniform(0, 6, e))).astype(int).tolist()
        f, k, n = (8 * int(np.exp(rng.uniform(0, 4.5))) for _ in range(3))
        x, w, dy, w2, offs = operands(sizes, f, k, n, i)
        r = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
        check_fwd(x, w, offs, "silu", r.h, r.gate_up, sum(sizes))
        d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs)
        check_dgrad(dy, w2, r.gate_up, offs, "silu", d, sum(sizes))


@pytest.mark.parametrize("sizes", [[3, 0, 2], [40, 0, 300], [30_000, 0, 20_300], [60_000, 0, 40_000]])
def test_rows_of_no_group_are_left_and_any_form_of_offsets(sizes):
    f, k, n, m = 72, 64, 40, sum(sizes)
    x, w, dy, w2, offs = operands(sizes, f, k, n, 3, pad=21)
    indptr = torch.cat([offs.new_zeros(1), offs])
    h = torch.full((m + 21, f), 7.0, dtype=torch.bfloat16, device=DEV)
    got = mdg.grouped_gated_gemm_fwd(x, w, offs, out=h)
    assert got.h is h and torch.all(h[m:] == 7.0)
    check_fwd(x, w, offs, "silu", h, None, m)
    r = mdg.grouped_gated_gemm_fwd(x, w, indptr, keep=True)
    assert torch.equal(r.h[:m], h[:m])
    d = torch.full((m + 21, 2 * f), 7.0, dtype=torch.bfloat16, device=DEV)
    assert mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, indptr, out=d) is d
    assert torch.all(d[m:] == 7.0)
    check_dgrad(dy, w2, r.gate_up, offs, "silu", d, m)
    # offsets that fall, are negative or past the rows act as their clamped form
    bad = torch.tensor([sizes[0], -5, 10 ** 6], dtype=torch.int32, device=DEV)
    good = torch.tensor([sizes[0], sizes[0], m + 21], dtype=torch.int32, device=DEV)
    assert torch.equal(mdg.grouped_gated_gemm_fwd(x, w, bad).h, mdg.grouped_gated_gemm_fwd(x, w, good).h)


@pytest.mark.parametrize("m", [0, 1, 300])
def test_no_rows_and_no_groups_with_rows(m):
    x, w, dy, w2, _ = operands([m], 16, 24, 32, 1)
    w, w2 = w.expand(3, -1, -1).contiguous(), w2.expand(3, -1, -1).contiguous()
    offs = torch.zeros(3, dtype=torch.int32, device=DEV)
    h = torch.full((m, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    mdg.grouped_gated_gemm_fwd(x, w, offs, out=h)
    assert torch.all(h == 7.0)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, torch.zeros((m, 32), dtype=torch.bfloat16, device=DEV), offs)
    assert d.shape == (m, 32)
    xs, ws, w2s = x.clone().requires_grad_(), w.clone().requires_grad_(), w2.clone().requires_grad_()
    y = mdg.grouped_gated_ffn(xs, ws, w2s, offs)
    assert torch.all(y == 0)
    y.backward(dy)
    assert torch.all(xs.grad == 0) and torch.all(ws.grad == 0) and torch.all(w2s.grad == 0)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [4, 300, 50_000])
def test_special_values_stay_where_they_belong(rows, name):
    """Projections of any size, zeros of both signs and values that are not finite: each
    reaches its own h, da and db only, and far tails are exact zeros or the value itself."""
    f, k = 64, 64
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    w = torch.zeros((1, 2 * f, k), dtype=torch.bfloat16, device=DEV)
    a = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 100.0, -100.0, 1e4, -1e4, 3e19, -3e19, 3e38, -3e38,
                      float("inf"), float("-inf"), float("nan"), 1.0, -1.0, 0.5], device=DEV).to(torch.bfloat16)
    w[0, :20, 0], w[0, f:, 0] = a, 1.5
    w[0, f + 30, 0], w[0, 30, 0] = float("inf"), 1.0
    offs = offsets([rows])
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=True)
    assert torch.equal(r.gate_up[:, :20].isnan(), a.isnan().expand(rows, -1))
    h = r.h.float()
    want = torch.from_numpy(ref.act(f64(a), name) * 1.5).to(DEV)
    fine = torch.isfinite(want) & (want.abs() < 3e38)
    assert torch.allclose(h[:, :20][:, fine].double(), want[fine].expand(rows, -1), rtol=2.0 ** -8, atol=1e-35)
    assert torch.all(h[:, 14] == float("inf")) and h[:, 15:17].isnan().all() and torch.all(h[:, 30] == float("inf"))
    others = [i for i in range(f) if i not in (12, 13, 14, 15, 16, 30)]
    assert torch.isfinite(h[:, others]).all()
    dy = torch.ones((rows, 8), dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros((1, 8, f), dtype=torch.bfloat16, device=DEV)
    w2[0, 0] = 2.0
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs, activation=name).double()
    av = f64(a)
    da = torch.from_numpy(2 * 1.5 * ref.act_grad(av, name)).to(DEV)
    db = torch.from_numpy(2 * ref.act(av, name)).to(DEV)
    ok = torch.isfinite(a) & (a.abs() < 1e38)   # (the oracle's cubes overflow past that)
    small = ok & (a.abs() < 1e5)
    assert torch.allclose(d[:, :20][:, small], da[small].expand(rows, -1), rtol=2.0 ** -8, atol=1e-35)
    assert torch.allclose(d[:, f:f + 20][:, small], db[small].expand(rows, -1), rtol=2.0 ** -8, atol=1e-35)
    assert torch.all(d[:, [10, 12]] == 3.0) and torch.all(d[:, [11, 13]] == 0.0)
    clean = [i for i in range(2 * f) if i % f not in (12, 13, 14, 15, 16, 30)]
    assert torch.isfinite(d[:, clean]).all()


@pytest.mark.parametrize("sizes,f", [([20, 300, 5], 136), ([900, 1100, 700], 1608), ([20, 300, 5], 40_008),
                                     ([3000, 2600, 2700], 2056)])
def test_nan_in_one_row_or_weight_stays_there(sizes, f):
    k, n, m, last = 96, 72, sum(sizes), sum(sizes[:2])
    x, w, dy, w2, offs = operands(sizes, f, k, n, 9)
    base = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
    x2, w_ = x.clone(), w.clone()
    x2[30, 5] = float("nan")
    w_[2, f + 3, 1] = float("inf")
    r = mdg.grouped_gated_gemm_fwd(x2, w_, offs, keep=True)
    hit = torch.zeros_like(base.h, dtype=torch.bool)
    hit[30] = True
    hit[last:, 3] = True
    assert torch.equal(r.h[~hit], base.h[~hit]) and not torch.isfinite(r.h[hit]).any()
    dy2 = dy.clone()
    dy2[last - 1, 2] = float("inf")
    d0 = mdg.grouped_gated_gemm_dgrad(dy, w2, base.gate_up, offs)
    d = mdg.grouped_gated_gemm_dgrad(dy2, w2, base.gate_up, offs)
    rows = torch.arange(m, device=DEV) != last - 1
    assert torch.equal(d[rows], d0[rows]) and not torch.isfinite(d[last - 1]).any()


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("sizes,f,k,n", [([3, 0, 2], 16, 24, 40), ([40, 300, 0, 9], 136, 72, 64)])
def test_block_gradients_against_the_formula(sizes, f, k, n, name):
    """Each stage of the block against the oracle on the operands that stage got."""
    m = sum(sizes)
    x, w, dy, w2, offs = operands(sizes, f, k, n, 5, pad=3)
    xs, ws, w2s = (t.clone().requires_grad_() for t in (x, w, w2))
    y = mdg.grouped_gated_ffn(xs, ws, w2s, offs, activation=name)
    y.backward(dy)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=True)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs, activation=name)
    o = offs.cpu().numpy()
    h, dn, dyn = f64(r.h)[:m], f64(d)[:m], f64(dy)[:m]
    inside(y[:m], ref.down(h, f64(w2), o), (f + 2) * U * ref.down(np.abs(h), np.abs(f64(w2)), o), "y")
    for got, left, g, rows, weight in ((ws.grad, xs.grad, dn, f64(x)[:m], f64(w)), (w2s.grad, None, dyn, h, f64(w2))):
        dx, dw = ref.product_grads(g, rows, weight, o)
        tx, tw = ref.product_grads(np.abs(g), np.abs(rows), np.abs(weight), o)
        inside(got, dw, (m + 2) * U * tw, "dw")
        if left is not None:
            inside(left[:m], dx, (2 * f + 2) * U * tx, "dx")
    assert torch.all(y[m:] == 0) and torch.all(xs.grad[m:] == 0)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_block_gradients_against_differences(name):
    """Derivatives along random directions against central differences of the oracle's
    block in 64 bits.  The gradients are sums of terms rounded to bf16 (2^-8 each, kept
    projections, h, d(gate_up) and the results: 4 of them) with random signs, and the
    directional derivative a sum of many: 4 * 2^-8 of the norm is far outside its error."""
    sizes, f, k, n = [30, 0, 34], 48, 40, 56
    x, w, dy, w2, offs = operands(sizes, f, k, n, 6)
    leaves = [t.clone().requires_grad_() for t in (x, w, w2)]
    mdg.grouped_gated_ffn(*leaves, offs, activation=name).backward(dy)
    o, base, g = offs.cpu().numpy(), [f64(t) for t in (x, w, w2)], f64(dy)

    def value(x, w, w2):
        return float((ref.down(ref.hidden(*ref.projections(x, w, o), name), w2, o) * g).sum())

    rng = np.random.default_rng(0)
    for i in range(3):
        v = [np.zeros_like(b) for b in base]
        v[i] = rng.normal(size=base[i].shape)
        e = 1e-5
        want = (value(*[b + e * d for b, d in zip(base, v)]) - value(*[b - e * d for b, d in zip(base, v)])) / (2 * e)
        got = float((f64(leaves[i].grad) * v[i]).sum())
        assert abs(got - want) <= 4 * 2.0 ** -8 * np.linalg.norm(f64(leaves[i].grad)), (i, got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_adds_into_main_grad(dtype):
    sizes, f, k, n = [30, 0, 270], 72, 64, 40
    x, w, dy, w2, offs = operands(sizes, f, k, n, 7)
    leaves = [t.clone().requires_grad_() for t in (w, w2)]
    start = [torch.randn(t.shape, device=DEV).to(dtype) for t in leaves]
    for t, s in zip(leaves, start):
        t.main_grad, t.grad_added_to_main_grad = s.clone(), False
    y = mdg.grouped_gated_ffn(x, *leaves, offs, fuse_wgrad_accumulation=True)
    y.backward(dy)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs)
    for t, s, g, rows in zip(leaves, start, (d, dy), (x, r.h)):
        assert t.grad_added_to_main_grad
        assert torch.equal(t.main_grad, s + mdg.grouped_det_gemm_wgrad(g, rows, offs, out_dtype=dtype))
    frozen = [w.clone(), w2.clone().requires_grad_()]
    frozen[1].main_grad = torch.zeros(w2.shape, device=DEV)
    mdg.grouped_gated_ffn(x, *frozen, offs, fuse_wgrad_accumulation=True).backward(dy)
    assert torch.equal(frozen[1].main_grad, mdg.grouped_det_gemm_wgrad(dy, r.h, offs, out_dtype=torch.float32))
    del frozen[1].main_grad
    with pytest.raises(ValueError, match="grouped_gated_ffn.*main_grad"):
        mdg.grouped_gated_ffn(x, *frozen, offs, fuse_wgrad_accumulation=True)


def test_no_double_backward_and_needed_gradients_only():
    x, w, dy, w2, offs = operands([5, 30], 24, 16, 8, 8)
    xs = x.clone().requires_grad_()
    y = mdg.grouped_gated_ffn(xs, w, w2, offs)
    with pytest.raises(NotImplementedError, match="double backward"):
        torch.autograd.grad(y, xs, dy, create_graph=True)
    y = mdg.grouped_gated_ffn(xs, w, w2, offs)
    only_x, = torch.autograd.grad(y, xs, dy)
    w2s = w2.clone().requires_grad_()
    only_down, = torch.autograd.grad(mdg.grouped_gated_ffn(x, w, w2s, offs), w2s, dy)
    all_ = [t.clone().requires_grad_() for t in (x, w, w2)]
    mdg.grouped_gated_ffn(*all_, offs).backward(dy)
    assert torch.equal(only_x, all_[0].grad) and torch.equal(only_down, all_[2].grad)
    assert not mdg.grouped_gated_ffn(x, w, w2, offs).requires_grad


@pytest.mark.parametrize("sizes", [[2, 0, 3], [300, 0, 40], [12_000, 0, 9000], [45_000, 0, 30_001]])
def test_other_stream_and_graph_replay(sizes):
    f, k, n = 136, 200, 72
    x, w, dy, w2, offs = operands(sizes, f, k, n, 12)
    want = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
    dwant = mdg.grouped_gated_gemm_dgrad(dy, w2, want.gate_up, offs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
        d = mdg.grouped_gated_gemm_dgrad(dy, w2, got.gate_up, offs)
    side.synchronize()
    assert torch.equal(got.h, want.h) and torch.equal(got.gate_up, want.gate_up) and torch.equal(d, dwant)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
        dg = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs)
    for i in range(4):
        x.copy_(bf16(tuple(x.shape), gen(100 + i)))
        if i == 2:
            offs.copy_(offsets(sizes[::-1]))
        torch.cuda.synchronize()
        graph.replay()
        want = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
        dwant = mdg.grouped_gated_gemm_dgrad(dy, w2, want.gate_up, offs)
        torch.cuda.synchronize()
        assert torch.equal(r.h, want.h) and torch.equal(r.gate_up, want.gate_up) and torch.equal(dg, dwant)


def test_workspace_given_and_refusals():
    x, w, dy, w2, offs = operands([5, 30], 24, 16, 8, 8)
    need = mdg.gated_gemm_fwd_workspace_bytes(35, 24, 16, 2)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True, workspace=ws)
    assert torch.equal(r.h, mdg.grouped_gated_gemm_fwd(x, w, offs).h)
    need = mdg.gated_gemm_dgrad_workspace_bytes(35, 8, 24, 2)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    assert torch.equal(d, mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs))
    fwd, dgrad = mdg.grouped_gated_gemm_fwd, mdg.grouped_gated_gemm_dgrad
    for error, call in (
            (ValueError, lambda: fwd(x, w, offs, workspace=ws[:256])),
            (ValueError, lambda: fwd(x, w, offs, activation="relu")),
            (TypeError, lambda: fwd(x.float(), w, offs)),
            (TypeError, lambda: fwd(x, w.float(), offs)),
            (TypeError, lambda: fwd(x, w, offs.long())),
            (TypeError, lambda: fwd(x, w, offs, keep=1)),
            (ValueError, lambda: fwd(x[:, :8], w, offs)),
            (ValueError, lambda: fwd(x, w[:, :, :8].contiguous(), offs)),
            (ValueError, lambda: fwd(x, w[:, :47].contiguous(), offs)),
            (ValueError, lambda: fwd(x, w, offs[:1])),
            (ValueError, lambda: fwd(x.cpu(), w, offs)),
            (ValueError, lambda: fwd(x, w, offs, out=r.h[:, :16].contiguous())),
            (mdg.MdgError, lambda: fwd(x, w[:, :4].contiguous(), offs)),
            (mdg.MdgError, lambda: fwd(x, w, offs, out=w.view(-1)[:35 * 24].view(35, 24))),
            (ValueError, lambda: dgrad(dy, w2, r.gate_up[:, :24].contiguous(), offs)),
            (ValueError, lambda: dgrad(dy[:, :4].contiguous(), w2, r.gate_up, offs)),
            (mdg.MdgError, lambda: dgrad(dy, w2, r.gate_up, offs, out=r.gate_up)),
            (ValueError, lambda: mdg.grouped_gated_ffn(x, w, w2[:1], offs)),
            (ValueError, lambda: mdg.grouped_gated_ffn(x, w, w2, offs, fuse_wgrad_accumulation=1))):
        with pytest.raises(error):
            call()


def test_tensors_of_more_than_4_gib():
    """Rows whose offsets pass 32 bits: the last group's against the same rows alone."""
    m, f, k, n = 140_000, 8192, 64, 64          # gate_up: 4.6 GB
    x, w, dy, w2, offs = operands([m - 300, 300], f, k, n, 2)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
    d = mdg.grouped_gated_gemm_dgrad(dy, w2, r.gate_up, offs)
    last = slice(m - 300, m)
    gu = r.gate_up[last].clone()
    check_fwd(x[last], w[1:], offsets([300]), "silu", r.h[last], gu, 300)
    check_dgrad(dy[last], w2[1:], gu, offsets([300]), "silu", d[last], 300)
