"""Calls of the gated feed-forward, the norms and clipping in other surroundings than a
plain eager one: compiled, captured with their gradients, on two streams at once, with
outputs or inputs left out, in inference mode, with inputs that are one tensor."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings(
    "ignore::DeprecationWarning", "ignore:Dynamo does not know:UserWarning", "ignore::FutureWarning")]
DEV = "cuda:0"
T, H, F, E = 40, 64, 48, 4


def inputs(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    return {"x": r(T, H).bfloat16(), "w": (r(E, 2 * F, H) / 8).bfloat16(), "w2": (r(E, H, F) / 8).bfloat16(),
            "res": r(T, H).bfloat16(), "n": 1 + r(H) / 4, "p": 1 + r(H) / 4, "gate": r(T)}


OFFS = torch.tensor([10, 10, 30, 40], dtype=torch.int32, device=DEV) if torch.cuda.is_available() else None


def run(v):
    out, n = mdg.block_norm(v["res"] * 2, v["x"], weight=v["n"], post_weight=v["p"], gate=v["gate"], scale=0.5)
    y = mdg.grouped_gated_ffn(n, v["w"], v["w2"], OFFS, activation="gelu_tanh")
    return mdg.block_norm(out, torch.tanh(y), weight=v["n"])[1] * 3


def test_compiled_gives_the_eager_bits():
    torch._dynamo.reset()
    compiled = torch.compile(run, backend="eager")
    for seed in (1, 2):
        a, b = [{k: t.clone().requires_grad_() for k, t in inputs(seed).items()} for _ in range(2)]
        ya, yb = compiled(a), run(b)
        assert torch.equal(ya, yb)
        for y in (ya, yb):
            y.float().square().sum().backward()
        assert all(torch.equal(a[k].grad, b[k].grad) for k in a)
    clip = torch.compile(lambda g: mdg.clip_grads([t * 2 for t in g], 1.0) + 1, backend="eager")
    g = [inputs(3)["res"], inputs(3)["gate"]]
    assert torch.equal(clip(g), mdg.grad_norm([t * 2 for t in g]) + 1)
    torch._dynamo.reset()


def test_captured_with_its_gradients():
    v = {k: t.clone().requires_grad_() for k, t in inputs(1).items()}
    dy = torch.randn((T, H), device=DEV).bfloat16()

    def step():
        grads = torch.autograd.grad(run(v), list(v.values()), dy)
        outs = [torch.empty_like(g) for g in grads]
        return list(grads) + outs + [mdg.clip_grads(grads, 0.5, out=outs)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(4):
        new = inputs(10 + seed)
        with torch.no_grad():
            for k, t in v.items():
                t.copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got_now = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got_now, want))


def test_two_streams_at_once():
    vs = [inputs(i) for i in range(2)]
    big = [torch.randn(3_000_000, device=DEV) for _ in range(2)]
    with torch.no_grad():
        want = [(run(v), mdg.grad_norm([b])) for v, b in zip(vs, big)]
    streams = [torch.cuda.Stream() for _ in vs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s), torch.no_grad():
                got[i].append((run(vs[i]), mdg.grad_norm([big[i]])))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, want[i][0]) and torch.equal(n, want[i][1]) for a, n in got[i])


def test_autograd_with_parts_left_out():
    v = {k: t.clone().requires_grad_() for k, t in inputs(4).items()}
    dout = torch.randn((T, H), device=DEV).bfloat16()
    out, normed = mdg.block_norm(v["res"], v["x"], gate=v["gate"], scale=0.3)
    assert normed is None
    out.backward(dout)
    r = mdg.block_norm_fwd(v["res"].detach(), v["x"].detach(), gate=v["gate"].detach(), scale=0.3)
    g = mdg.block_norm_bwd(dout, None, r, v["x"].detach(), gate=v["gate"].detach(), scale=0.3)
    assert torch.equal(v["x"].grad, g.dy) and torch.equal(v["gate"].grad, g.dgate) and torch.equal(v["res"].grad, dout)
    # nothing but the sum: y's gradient needs neither y nor out
    x, res = (inputs(4)[k].requires_grad_() for k in ("x", "res"))
    out, _ = mdg.block_norm(res, x, scale=-2.0)
    out.sum().backward()
    assert torch.all(x.grad == -2.0) and torch.all(res.grad == 1.0)
    # one tensor as both inputs
    both = inputs(5)["x"].requires_grad_()
    out, n = mdg.block_norm(both, both, weight=inputs(5)["n"], scale=0.5)
    n.backward(dout)
    a, b = (inputs(5)["x"].requires_grad_() for _ in range(2))
    mdg.block_norm(a, b, weight=inputs(5)["n"], scale=0.5)[1].backward(dout)
    assert torch.equal(both.grad, a.grad + b.grad)


def test_inference_mode_and_no_grad():
    v = inputs(6)
    with torch.inference_mode():
        y = run(v)
        g = [torch.ones(10, device=DEV)]
        mdg.clip_grads(g, 1.0)
    assert torch.equal(y, run(v)) and abs(float(g[0].square().sum()) - 1.0) < 1e-5
    with torch.no_grad():
        assert not mdg.grouped_gated_ffn(v["x"].requires_grad_(), v["w"], v["w2"], OFFS).requires_grad


def test_without_grad_mode_nothing_is_kept():
    """Trained weights in a serving call: no projections, so the memory of weights that are not."""
    x = torch.randn((4096, H), device=DEV).bfloat16()
    offs = torch.tensor([1000, 1500, 1500, 4096], dtype=torch.int32, device=DEV)
    w, w2 = (torch.randn(s, device=DEV).bfloat16() for s in ((E, 1024, H), (E, H, 512)))
    peaks, ys = [], []
    for trained in (False, False, True):  # (the first call fills the allocator)
        ws = [t.requires_grad_(trained) for t in (w, w2)]
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with torch.no_grad():
            y = mdg.grouped_gated_ffn(x, *ws, offs)
        peaks.append(torch.cuda.max_memory_allocated() - before)
        ys.append(y)
    assert peaks[2] == peaks[1]
    assert torch.equal(ys[2], ys[1]) and not ys[2].requires_grad


def test_retained_graph_gives_the_same_gradients_twice():
    v = {k: t.clone().requires_grad_() for k, t in inputs(7).items()}
    y = run(v)
    dy = torch.ones_like(y)
    a = torch.autograd.grad(y, list(v.values()), dy, retain_graph=True)
    b = torch.autograd.grad(y, list(v.values()), dy)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_checkpointed_block_gives_the_same_gradients():
    a, b = [{k: t.clone().requires_grad_() for k, t in inputs(8).items()} for _ in range(2)]
    run(a).float().sum().backward()
    torch.utils.checkpoint.checkpoint(run, b, use_reentrant=False).float().sum().backward()
    assert all(torch.equal(a[k].grad, b[k].grad) for k in a)


def test_gradients_of_summed_and_transposed_outputs():
    """Output gradients that are expanded or strided."""
    v = {k: t.clone().requires_grad_() for k, t in inputs(9).items()}
    y = mdg.grouped_gated_ffn(v["x"], v["w"], v["w2"], OFFS)
    y.sum().backward()
    w = {k: t.clone().requires_grad_() for k, t in inputs(9).items()}
    mdg.grouped_gated_ffn(w["x"], w["w"], w["w2"], OFFS).backward(torch.ones((T, H), device=DEV).bfloat16())
    assert all(torch.equal(v[k].grad, w[k].grad) for k in ("x", "w", "w2"))
    y = mdg.grouped_gated_ffn(v["x"], v["w"], v["w2"], OFFS)
    g = torch.randn((H, T), device=DEV).bfloat16()
    gx, = torch.autograd.grad(y.t(), v["x"], g)
    y = mdg.grouped_gated_ffn(v["x"], v["w"], v["w2"], OFFS)
    assert torch.equal(gx, torch.autograd.grad(y, v["x"], g.t().contiguous())[0])
