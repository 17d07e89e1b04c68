"""The gated feed-forward without a GPU: the C ABI's refusals and workspace rules, the
binding's, tracing, and the oracle's gradients against differences.

Pointers below are fake, aligned addresses: every case returns before any device
access.
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import gated as ref

OK, EINVAL, EUNSUP, EOVERLAP, EWS, EHIP, ENOMEM = range(7)
P = [0x100000000 * i for i in range(1, 12)]


@pytest.fixture(scope="module")
def lib():
    return mdg.load_library()


def caller(fn, order, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a)
        a.update(kw)
        return fn(*[a[n] for n in order])
    return call


def test_fwd_refusals(lib):
    order = "x w offs h gu act M F K E ws wsn stream".split()
    need = lib.grouped_gated_gemm_fwd_workspace_bytes(100, 264, 72, 4)
    assert need > 0
    call = caller(lib.grouped_gated_gemm_fwd, order, dict(
        x=P[0], w=P[1], offs=P[2], h=P[3], gu=P[4], act=0, M=100, F=264, K=72, E=4, ws=P[5], wsn=need, stream=None))
    for kw in (dict(M=-1), dict(F=0), dict(K=0), dict(E=0), dict(act=2), dict(act=-1), dict(x=0), dict(w=0), dict(offs=0),
               dict(h=0), dict(x=P[0] + 8), dict(w=P[1] + 8), dict(offs=P[2] + 2), dict(h=P[3] + 2), dict(gu=P[4] + 8),
               dict(ws=P[5] + 16)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(F=260), dict(K=76), dict(E=1025), dict(M=4000001), dict(F=(1 << 19) + 8), dict(K=(1 << 20) + 8),
               dict(F=1 << 15, K=1 << 15)):
        assert call(**kw) == EUNSUP, kw
    assert call(ws=0) == EWS and call(wsn=need - 1) == EWS
    w_end = P[1] + 4 * 528 * 72 * 2
    for kw in (dict(h=P[0] + 16), dict(h=P[1]), dict(h=w_end - 16), dict(h=P[2]), dict(gu=P[0]), dict(gu=P[1] + 16),
               dict(gu=P[3] + 100 * 264 * 2 - 16), dict(ws=P[0]), dict(ws=P[3]), dict(ws=P[4]), dict(h=P[5] + 32)):
        assert call(**kw) == EOVERLAP, kw
    assert call(M=0, wsn=lib.grouped_gated_gemm_fwd_workspace_bytes(0, 264, 72, 4)) == OK
    assert call(M=0, x=0, h=0, gu=0) == OK and call(M=0, w=0) == EINVAL


def test_dgrad_refusals(lib):
    order = "dy w gu offs d act M N F E ws wsn stream".split()
    need = lib.grouped_gated_gemm_dgrad_workspace_bytes(100, 72, 264, 4)
    assert need > 0
    call = caller(lib.grouped_gated_gemm_dgrad, order, dict(
        dy=P[0], w=P[1], gu=P[2], offs=P[3], d=P[4], act=1, M=100, N=72, F=264, E=4, ws=P[5], wsn=need, stream=None))
    for kw in (dict(M=-1), dict(F=0), dict(N=0), dict(E=0), dict(act=2), dict(dy=0), dict(w=0), dict(offs=0), dict(gu=0),
               dict(d=0), dict(dy=P[0] + 8), dict(gu=P[2] + 8), dict(d=P[4] + 8), dict(offs=P[3] + 1), dict(ws=P[5] + 8)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(F=260), dict(N=76), dict(E=1025), dict(M=4000001), dict(F=1 << 15, N=1 << 15)):
        assert call(**kw) == EUNSUP, kw
    assert call(ws=0) == EWS and call(wsn=need - 1) == EWS
    for kw in (dict(d=P[0]), dict(d=P[1] + 16), dict(d=P[2]), dict(d=P[3] - 16), dict(ws=P[2]), dict(ws=P[4])):
        assert call(**kw) == EOVERLAP, kw
    assert call(M=0, dy=0, gu=0, d=0) == OK


def test_workspace_is_a_function_of_the_sizes(lib):
    fwd, dgrad = lib.grouped_gated_gemm_fwd_workspace_bytes, lib.grouped_gated_gemm_dgrad_workspace_bytes
    for bad in ((-1, 8, 8, 1), (1, 0, 8, 1), (1, 8, 9, 1), (1, 9, 8, 1), (1, 8, 8, 0), (1, 8, 8, 1025)):
        assert fwd(*bad) == 0 and dgrad(bad[0], bad[2], bad[1], bad[3]) == 0
    most = 8192 + 256 * 256 * 256 * 4
    assert fwd(16384, 14336, 4096, 8) == most == dgrad(16384, 4096, 14336, 8)
    assert fwd(1, 8, 8, 1) < most
    assert mdg.gated_gemm_fwd_workspace_bytes(1, 8, 8, 1) == fwd(1, 8, 8, 1)
    assert mdg.gated_gemm_dgrad_workspace_bytes(1, 8, 16, 1) == dgrad(1, 8, 16, 1)


X = torch.ones((3, 16), dtype=torch.bfloat16)
W, W2 = torch.ones((4, 32, 16), dtype=torch.bfloat16), torch.ones((4, 8, 16), dtype=torch.bfloat16)
OFFS = torch.full((4,), 3, dtype=torch.int32)
CALLS = {
    "fwd": lambda x: mdg.grouped_gated_gemm_fwd(x, W, OFFS).h,
    "dgrad": lambda x: mdg.grouped_gated_gemm_dgrad(x[:, :8].contiguous(), W2, torch.cat([x, x], 1), OFFS),
    "ffn": lambda x: mdg.grouped_gated_ffn(x, W, W2, OFFS),
}


@pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning")
@pytest.mark.parametrize("name", CALLS)
def test_refuses_cpu_tensors_and_tracing(name):
    with pytest.raises(ValueError, match="must be on a ROCm device"):
        CALLS[name](X)
    with pytest.raises(NotImplementedError, match="cannot be traced by torch.jit.trace"):
        torch.jit.trace(CALLS[name], X, check_trace=False)


def test_refusals_before_the_device():
    with pytest.raises(ValueError, match="activation must be one of"):
        mdg.grouped_gated_gemm_fwd(X, W, OFFS, activation="relu")
    with pytest.raises(ValueError, match="activation must be one of"):
        mdg.grouped_gated_ffn(X, W, W2, OFFS, activation=None)
    with pytest.raises(TypeError, match="must be torch.bfloat16"):
        mdg.grouped_gated_gemm_fwd(X.float(), W, OFFS)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        mdg.grouped_gated_gemm_dgrad(None, W2, X, OFFS)
    with pytest.raises(ValueError, match="fuse_wgrad_accumulation must be a bool"):
        mdg.grouped_gated_ffn(X, W, W2, OFFS, fuse_wgrad_accumulation=1)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_oracle_gradients_against_differences(name):
    rng = np.random.default_rng(3)
    offs, f = [3, 3, 8], 5
    x, w, w2, g = rng.normal(size=(8, 7)), rng.normal(size=(3, 10, 7)), rng.normal(size=(3, 6, 5)), rng.normal(size=(8, 6))

    def loss(x, w, w2):
        return (ref.down(ref.hidden(*ref.projections(x, w, offs), name), w2, offs) * g).sum()

    a, b = ref.projections(x, w, offs)
    _, d = ref.gate_up_grad(g, w2, a, b, offs, name)
    dx, dw = ref.product_grads(d, x, w, offs)
    _, dw2 = ref.product_grads(g, ref.hidden(a, b, name), w2, offs)
    for i, grad in enumerate((dx, dw, dw2)):
        at = [x, w, w2]
        v = rng.normal(size=at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-6 * v, at[i] - 1e-6 * v
        want = (loss(*hi) - loss(*lo)) / 2e-6
        assert abs((grad * v).sum() - want) <= 1e-7 * abs(grad * v).sum()
    z = rng.normal(size=50) * 5
    t = torch.from_numpy(z).requires_grad_()
    y = torch.nn.functional.silu(t) if name == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    y.sum().backward()
    assert np.allclose(ref.act(z, name), y.detach().numpy(), rtol=1e-9, atol=1e-14)
    assert np.allclose(ref.act_grad(z, name), t.grad.numpy(), rtol=1e-9, atol=1e-13)
