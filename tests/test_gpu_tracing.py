"""The operators around the products under torch.compile and torch.jit.trace: what
does not refuse gives the eager bits, also for inputs it was not recorded with."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings(
    "ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning", "ignore:Dynamo does not know:UserWarning",
    "ignore::FutureWarning")]
DEV = "cuda:0"
T, H, E, K = 40, 64, 8, 2


def inputs(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn((T, E), generator=g, device=DEV), torch.randn((T, H), generator=g, device=DEV)


def single_calls(logits, x):
    r = mdg.moe_route_fwd(logits * 2, K)
    plan = mdg.moe_plan(r.idx, E)
    rows = mdg.moe_dispatch_fwd(x + 1, plan)
    return mdg.moe_combine_fwd(torch.tanh(rows), r.weight, plan) * 3


def autograd_calls(logits, x):
    r = mdg.moe_route(logits * 2, K)
    plan = mdg.moe_plan(r.idx, E)
    rows = mdg.moe_dispatch(x + 1, plan)
    return mdg.moe_combine(torch.tanh(rows), r.weight, plan) * 3 + r.loss


@pytest.mark.parametrize("f", [single_calls, autograd_calls])
def test_compiled_gives_the_eager_bits(f):
    torch._dynamo.reset()
    compiled = torch.compile(f, backend="eager")
    for seed in (1, 2):
        logits, x = inputs(seed)
        assert torch.equal(compiled(logits, x), f(logits, x))
        if f is autograd_calls:
            a, b = [[t.clone().requires_grad_() for t in (logits, x)] for _ in range(2)]
            compiled(*a).square().sum().backward()
            f(*b).square().sum().backward()
            assert all(torch.equal(p.grad, q.grad) for p, q in zip(a, b))
    torch._dynamo.reset()


def test_traced_autograd_forms_follow_new_inputs():
    logits, x = inputs(1)
    plan = mdg.moe_plan(mdg.moe_route_fwd(logits, K).idx, E)
    f = lambda x, w: mdg.moe_combine(torch.tanh(mdg.moe_dispatch(x, plan)), w, plan)
    w = torch.rand((T, K), device=DEV)
    traced = torch.jit.trace(f, (x.clone().requires_grad_(), w.clone().requires_grad_()), check_trace=False)
    new, nw = inputs(2)[1], torch.rand((T, K), device=DEV)
    assert torch.equal(traced(new, nw), f(new, nw))
    route = torch.jit.trace(lambda l: tuple(mdg.moe_route(l, K)), logits.clone().requires_grad_(), check_trace=False)
    for a, b in zip(route(inputs(3)[0]), mdg.moe_route_fwd(inputs(3)[0], K)):
        assert torch.equal(a, b)


def test_single_calls_refuse_tracing():
    with pytest.raises(NotImplementedError, match="moe_route_fwd cannot be traced"):
        torch.jit.trace(single_calls, inputs(1), check_trace=False)
