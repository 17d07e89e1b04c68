"""torch.jit.trace records torch's operators only: of a library call it would see the
outputs' allocation and nothing that fills them.  So calls that are not autograd
functions refuse it; those that are stay in the graph as Python calls.

CPU tensors: a call that does not refuse tracing first refuses the device (ValueError).
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from moe_ragged_bf16_amd import _capi

pytestmark = pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning",
                                      "ignore:Dynamo does not know:UserWarning")

T, K, E, H = 3, 2, 4, 16
X = torch.ones((T, H))
B = torch.ones((T, H), dtype=torch.bfloat16)
W = torch.ones((E, 8, H), dtype=torch.bfloat16)
IDX = torch.zeros((T, K), dtype=torch.int32)
OFFS = torch.full((E,), T, dtype=torch.int32)
PLAN = mdg.MoePlan(OFFS, IDX)
WT = torch.ones((T, K))
ROUTE = mdg.MoeRoute(WT, IDX, OFFS, torch.ones(()), torch.ones(E))
Y = torch.ones((T * K, H))

CALLS = {
    "moe_route_fwd": lambda x: mdg.moe_route_fwd(x, K).weight,
    "moe_route_bwd": lambda x: mdg.moe_route_bwd(None, None, x, ROUTE),
    "moe_plan": lambda x: mdg.moe_plan(x.int(), E).dest,
    "moe_dispatch_fwd": lambda x: mdg.moe_dispatch_fwd(x, PLAN),
    "moe_dispatch_bwd": lambda x: mdg.moe_dispatch_bwd(x, PLAN),
    "moe_combine_fwd": lambda x: mdg.moe_combine_fwd(x, WT, PLAN),
    "moe_combine_bwd": lambda x: mdg.moe_combine_bwd(x, Y, WT, PLAN)[0],
    "quantize_fp8_rows": lambda x: mdg.quantize_fp8_rows(x).q,
    "quantize_fp8_weight": lambda x: mdg.quantize_fp8_weight(x[None]).q,
    "grouped_fp8_gemm_fwd": lambda x: mdg.grouped_fp8_gemm_fwd(x, W, W, OFFS),
    "grouped_fp8_gemm_dgrad": lambda x: mdg.grouped_fp8_gemm_dgrad(x, W, W, OFFS),
    "grouped_fp8_mm": lambda x: mdg.grouped_fp8_mm(x.bfloat16(), W, OFFS),
    "grouped_det_gemm_fwd": lambda x: mdg.grouped_det_gemm_fwd(x, W, OFFS),
    "grouped_det_gemm_dgrad": lambda x: mdg.grouped_det_gemm_dgrad(x, W, OFFS),
    "grouped_det_gemm_wgrad": lambda x: mdg.grouped_det_gemm_wgrad(x, B, OFFS),
    "zero_pad_rows": lambda x: mdg.zero_pad_rows(x, OFFS, E),
    "grouped_mm_bf16": lambda x: mdg.grouped_mm_bf16(x, W, torch.zeros(E + 1, dtype=torch.int32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_single_calls_refuse_tracing(name):
    with pytest.raises(NotImplementedError, match="cannot be traced by torch.jit.trace"):
        torch.jit.trace(CALLS[name], X, check_trace=False)


@pytest.mark.parametrize("name", CALLS)
def test_without_tracing_they_check_their_arguments(name):
    with pytest.raises((ValueError, TypeError)):
        CALLS[name](X)


@pytest.mark.parametrize("name", ["moe_plan", "moe_dispatch_fwd", "moe_route_fwd", "quantize_fp8_rows"])
def test_compile_does_not_take_them_into_a_graph(name):
    """torch.compile leaves the call out of its graphs and runs it: it refuses the CPU."""
    with pytest.raises(Exception, match="ROCm device"):
        torch.compile(lambda x: CALLS[name](x * 2), backend="eager")(X)
    torch._dynamo.reset()


def test_autograd_forms_are_python_calls_of_a_trace(monkeypatch):
    """With a stand-in for the library's call, the traced function follows new inputs."""
    def dispatch(x, offs, dest):
        return torch.from_numpy(x.detach().numpy()[np.arange(T * K) // K].copy())
    monkeypatch.setitem(_capi.native.__dict__, "dispatch_fwd", dispatch)
    traced = torch.jit.trace(lambda x: mdg.moe_dispatch(x, PLAN) * 2, X.clone().requires_grad_(), check_trace=False)
    new = torch.randn((T, H))
    assert torch.equal(traced(new), new.repeat_interleave(K, dim=0) * 2)
