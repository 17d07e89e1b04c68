"""The norms around a block, the gradients' norm and clipping without a GPU: the C ABI's
refusals and workspace rules, the binding's, tracing, and the oracle's gradients
against differences.

Pointers below are fake, aligned addresses: every case returns before any device
access.
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from moe_ragged_bf16_amd._capi import Gradient
from oracle import norm as ref

OK, EINVAL, EUNSUP, EOVERLAP, EWS, EHIP, ENOMEM = range(7)
P = [0x100000000 * i for i in range(1, 24)]
BF16, FP32 = 0, 1


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


def test_norm_fwd_refusals(lib):
    order = "r y w wp gate out n rstd prstd T H dt wdt scale eps stream".split()
    call = caller(lib.block_norm_fwd, order, dict(
        r=P[0], y=P[1], w=P[2], wp=P[3], gate=P[4], out=P[5], n=P[6], rstd=P[7], prstd=P[8], T=10, H=64, dt=BF16,
        wdt=FP32, scale=1.0, eps=1e-6, stream=None))
    for kw in (dict(T=-1), dict(H=0), dict(dt=2), dict(wdt=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(eps=-1.0), dict(eps=float("nan")), dict(r=0), dict(out=0), dict(n=0), dict(rstd=0), dict(w=0),
               dict(prstd=0), dict(wp=0), dict(y=0), dict(y=0, out=0, wp=0, prstd=0), dict(r=P[0] + 8), dict(y=P[1] + 2),
               dict(w=P[2] + 4), dict(wp=P[3] + 8), dict(gate=P[4] + 2), dict(out=P[5] + 8), dict(n=P[6] + 8),
               dict(rstd=P[7] + 1), dict(prstd=P[8] + 2),
               dict(y=0, out=0, wp=0, prstd=0, gate=0, w=0, n=0, rstd=0)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(T=4000001), dict(H=60), dict(H=16392)):
        assert call(**kw) == EUNSUP, kw
    for kw in (dict(out=P[0]), dict(out=P[1] + 16), dict(n=P[0] + 10 * 64 * 2 - 16), dict(n=P[2]), dict(n=P[3] + 240),
               dict(rstd=P[4]), dict(rstd=P[7], prstd=P[7] + 36), dict(out=P[6]), dict(rstd=P[5] + 4)):
        assert call(**kw) == EOVERLAP, kw
    assert call(T=0) == OK and call(T=0, r=0, y=0, gate=0, out=0, n=0, rstd=0, prstd=0) == OK


def test_norm_bwd_refusals(lib):
    order = "d dn out y w wp gate rstd prstd dr dy dw dwp dg T H dt wdt scale ws wsn stream".split()
    need = lib.block_norm_bwd_workspace_bytes(10, 64)
    assert need == 3 * 2 * 64 * 4                              # 4 rows a block
    assert lib.block_norm_bwd_workspace_bytes(10 ** 6, 8192) == 512 * 2 * 8192 * 4
    assert lib.block_norm_bwd_workspace_bytes(10, 60) == 0 and lib.block_norm_bwd_workspace_bytes(0, 64) == 0
    call = caller(lib.block_norm_bwd, order, dict(
        d=P[0], dn=P[1], out=P[2], y=P[3], w=P[4], wp=P[5], gate=P[6], rstd=P[7], prstd=P[8], dr=P[9], dy=P[10], dw=P[11],
        dwp=P[12], dg=P[13], T=10, H=64, dt=FP32, wdt=BF16, scale=0.5, ws=P[14], wsn=need, stream=None))
    for kw in (dict(T=-1), dict(H=0), dict(dt=3), dict(wdt=9), dict(scale=float("nan")), dict(d=0, dn=0), dict(w=0),
               dict(out=0), dict(rstd=0), dict(prstd=0), dict(y=0), dict(wp=0), dict(gate=0), dict(d=P[0] + 4),
               dict(dn=P[1] + 8), dict(out=P[2] + 4), dict(y=P[3] + 4), dict(dr=P[9] + 4), dict(dy=P[10] + 4),
               dict(dw=P[11] + 8), dict(dwp=P[12] + 8), dict(dg=P[13] + 2), dict(rstd=P[7] + 2), dict(ws=P[14] + 64)):
        assert call(**kw) == EINVAL, kw
    assert call(H=20000) == EUNSUP and call(H=12) == EUNSUP
    assert call(ws=0) == EWS and call(wsn=need - 1) == EWS
    for kw in (dict(dr=P[0]), dict(dr=P[1]), dict(dy=P[2]), dict(dy=P[3] + 16), dict(dw=P[4]), dict(dwp=P[5]), dict(dg=P[6]),
               dict(dg=P[7]), dict(dr=P[10]), dict(dw=P[12] + 16), dict(ws=P[9]), dict(ws=P[3])):
        assert call(**kw) == EOVERLAP, kw
    assert call(T=0, dw=0, dwp=0, ws=0, wsn=0) == OK


def table(*rows):
    return (Gradient * len(rows))(*[Gradient(*r, 0) for r in rows])


def test_clip_refusals(lib):
    need = lib.grad_norm_workspace_bytes(2)
    assert need == 1024 * 8 and lib.grad_norm_workspace_bytes(336) == need
    assert lib.grad_norm_workspace_bytes(337) == 2 * need
    assert lib.grad_norm_workspace_bytes(-1) == 0 and lib.grad_norm_workspace_bytes(65537) == 0
    assert lib.grad_norm_workspace_bytes(0) == 0
    ok = ((P[0], P[1], 100, FP32), (P[2], P[2], 100, BF16))

    def norm(rows=ok, n=None, norm=P[5], ws=P[6], wsn=need):
        return lib.grad_norm(table(*rows), len(rows) if n is None else n, norm, ws, wsn, None)

    def clip(rows=ok, n=None, limit=1.0, given=None, norm=P[5], ws=P[6], wsn=need):
        return lib.grad_clip(table(*rows), len(rows) if n is None else n, limit, given, norm, ws, wsn, None)

    for call in (norm, clip):
        assert call(n=-1) == EINVAL and call(norm=P[5] + 2) == EINVAL and call(norm=0) == EINVAL
        assert call(ws=0) == EWS and call(wsn=need - 1) == EWS and call(ws=P[6] + 8) == EINVAL
        for row in ((P[0], P[1], 100, 2), (P[0], P[1], -1, FP32), (0, P[1], 1, FP32), (P[0] + 2, P[1], 1, FP32),
                    (P[0] + 1, P[1], 1, BF16)):
            assert call(rows=(ok[1], row)) == EINVAL, row
        assert call(rows=((P[0], P[1], 2 ** 36 + 1, BF16),), wsn=need) == EUNSUP
        assert call(rows=((P[0], P[1], 2 ** 36, FP32),) * 300, wsn=need) == EUNSUP      # 2.5e9 pieces
        assert call(rows=(ok[1], (P[0] + 2 ** 48, P[1], 1, FP32))) == EINVAL
        assert call(norm=P[0] + 396) == EOVERLAP and call(ws=P[0]) == EOVERLAP and call(norm=P[6]) == EOVERLAP
    assert lib.grad_norm(None, 1, P[5], P[6], need, None) == EINVAL
    assert clip(limit=-1.0) == EINVAL and clip(limit=float("nan")) == EINVAL
    assert clip(given=P[7]) == EINVAL and clip(given=P[7] + 1, norm=None) == EINVAL
    assert clip(rows=((P[0], 0, 1, FP32),)) == EINVAL and clip(rows=((P[0], P[1] + 2, 1, FP32),)) == EINVAL
    for rows in (((P[0], P[0], 100, FP32), (P[0], P[0], 100, FP32)),            # one tensor twice
                 ((P[0], P[0] + 4, 100, FP32),),                               # half over itself
                 ((P[0], P[1], 100, FP32), (P[2], P[0], 1, FP32)),              # an output in another's data
                 ((P[0], P[1], 100, FP32), (P[2], P[1] + 398, 1, BF16)),        # two outputs
                 ((P[3], P[3], 10, FP32), (P[0], P[1], 100, FP32), (P[1] + 396, P[4], 1, FP32))):
        assert clip(rows=rows) == EOVERLAP, rows
    assert clip(rows=((P[0], P[5], 1, FP32),)) == EOVERLAP and clip(rows=((P[0], P[6] + 64, 1, FP32),)) == EOVERLAP
    assert clip(given=P[1] + 4, norm=None, ws=None, wsn=0) == EOVERLAP


X = torch.ones((3, 16))
CALLS = {
    "block_norm_fwd": lambda x: mdg.block_norm_fwd(x, weight=x[0].contiguous()).normed,
    "block_norm_bwd": lambda x: mdg.block_norm_bwd(x, x, mdg.BlockNorm(x, x, None, None), weight=x[0]).dresidual,
    "grad_norm": lambda x: mdg.grad_norm([x]),
    "clip_grads": lambda x: mdg.clip_grads([x], 1.0),
}


@pytest.mark.filterwarnings("ignore::DeprecationWarning", "ignore::torch.jit.TracerWarning")
@pytest.mark.parametrize("name", CALLS)
def test_refuses_cpu_tensors_and_tracing(name):
    with pytest.raises(ValueError, match="must be on a ROCm device"):
        CALLS[name](X)
    with pytest.raises(NotImplementedError, match="cannot be traced by torch.jit.trace"):
        torch.jit.trace(CALLS[name], X, check_trace=False)


def test_clip_refuses_what_is_no_list_of_tensors():
    with pytest.raises(TypeError, match="sequence of tensors"):
        mdg.grad_norm(X)
    with pytest.raises(ValueError, match="no gradients"):
        mdg.clip_grads([], 1.0)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        mdg.grad_norm([1])
    with pytest.raises(ValueError, match="dense"):
        mdg.grad_norm([X.to_sparse()])


@pytest.mark.parametrize("post,gate,weight", [(True, True, True), (False, True, True), (True, False, False), (False, False, True)])
def test_oracle_gradients_against_differences(post, gate, weight):
    rng = np.random.default_rng(5)
    T, H, eps, scale = 5, 7, 1e-3, -0.6
    at = [rng.normal(size=(T, H)), rng.normal(size=(T, H)), rng.normal(size=H) if weight else None,
          rng.normal(size=H) if post else None, rng.normal(size=T) if gate else None]
    do, dn = rng.normal(size=(T, H)), rng.normal(size=(T, H)) if weight else None

    def value(r, y, w, p, g):
        out, normed = ref.block(r, y, w, p, g, scale, eps)
        return (out * do).sum() + (0 if dn is None else (normed * dn).sum())

    out, _ = ref.block(*at, scale, eps)
    grads = ref.block_grad(do, dn, out, *at[1:], scale, eps)
    for i, g in enumerate(grads):
        if at[i] is None:
            assert g is None
            continue
        v = rng.normal(size=at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-6 * v, at[i] - 1e-6 * v
        want = (value(*hi) - value(*lo)) / 2e-6
        assert abs((g * v).sum() - want) <= 1e-7 * np.abs(g * v).sum()
