"""Output gradients that start anywhere in their buffer, as autograd hands them over
behind a flattened concatenation: the same gradients, bit for bit, as from aligned
ones."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, F, E = 24, 64, 48, 3


def inputs():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    return {"x": r(T, H).bfloat16(), "w": (r(E, 2 * F, H) / 8).bfloat16(), "w2": (r(E, H, F) / 7).bfloat16(),
            "res": r(T, H).bfloat16(), "n": r(H), "p": r(H), "gate": r(T), "weight": torch.rand((T, 2), generator=g, device=DEV)}


OFFS = torch.tensor([7, 7, T], dtype=torch.int32, device=DEV) if torch.cuda.is_available() else None


def plan():
    return mdg.moe_plan(torch.arange(2 * T, dtype=torch.int32, device=DEV).view(T, 2) % E, E)


CALLS = {
    "cake_grouped_det_mm": lambda v: mdg.cake_grouped_det_mm(v["x"], v["w"], OFFS),
    "grouped_fp8_mm": lambda v: mdg.grouped_fp8_mm(v["x"], v["w"], OFFS),
    "moe_dispatch": lambda v: mdg.moe_dispatch(v["x"], plan()),
    "moe_combine": lambda v: mdg.moe_combine(torch.cat([v["x"], v["res"]]), v["weight"], plan()),
    "grouped_gated_ffn": lambda v: mdg.grouped_gated_ffn(v["x"], v["w"], v["w2"], OFFS),
    "block_norm": lambda v: mdg.block_norm(v["res"], v["x"], weight=v["n"], post_weight=v["p"], gate=v["gate"])[1],
    "block_norm, out": lambda v: mdg.block_norm(v["res"], v["x"], weight=v["n"], scale=0.5)[0],
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("by", [1, 3])
def test_gradients_that_start_anywhere(name, by):
    a, b = [{k: t.clone().requires_grad_() for k, t in inputs().items()} for _ in range(2)]
    ya, yb = CALLS[name](a), CALLS[name](b)
    dy = torch.randn(ya.shape, device=DEV).to(ya.dtype)
    ya.backward(dy)
    # the gradient of the concatenation's second part is a view `by` elements into its own
    joined = torch.cat([yb.new_zeros(by), yb.flatten()])
    joined.backward(torch.cat([dy.new_ones(by), dy.flatten()]))
    for k in a:
        assert (a[k].grad is None) == (b[k].grad is None)
        assert a[k].grad is None or torch.equal(a[k].grad, b[k].grad), k
