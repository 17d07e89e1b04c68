"""Routing, plan, dispatch and combine without a GPU: the C ABI's refusals, the
binding's, workspace rules, and the oracle's gradients against differences.

Pointers below are fake, aligned addresses: every case returns before any device
access.
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import moe as ref

OK, EINVAL, EUNSUP, EOVERLAP, EWS, EHIP, ENOMEM = range(7)
P = [0x10000000 * i for i in range(1, 12)]
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


def test_route_fwd_refusals(lib):
    order = "logits dtype mask weight idx counts loss balance T E k norm ws wsn stream".split()
    need = lib.moe_route_fwd_workspace_bytes(100000, 64)
    assert need > 0
    call = caller(lib.moe_route_fwd, order, dict(
        logits=P[0], dtype=BF16, mask=P[1], weight=P[2], idx=P[3], counts=P[4], loss=P[5], balance=P[6],
        T=100000, E=64, k=4, norm=1, ws=P[7], wsn=need, stream=None))
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(dtype=2), dict(logits=0), dict(weight=0), dict(idx=0),
               dict(counts=0), dict(loss=0), dict(balance=0), dict(logits=P[0] + 1), dict(dtype=FP32, logits=P[0] + 2),
               dict(weight=P[2] + 2), dict(idx=P[3] + 1), dict(ws=P[7] + 16)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(E=1025), dict(k=33), dict(k=5, E=4), dict(T=4000001, k=1), dict(T=1000001)):
        assert call(**kw) == EUNSUP, kw
    assert call(ws=0) == EWS and call(wsn=need - 1) == EWS
    for kw in (dict(weight=P[0] + 4), dict(idx=P[2]), dict(counts=P[1]), dict(loss=P[2] + 8), dict(balance=P[4] + 8),
               dict(ws=P[0]), dict(ws=P[3])):
        assert call(**kw) == EOVERLAP, kw


def test_route_bwd_refusals(lib):
    order = "logits dtype weight idx balance dw dl out T E k norm stream".split()
    call = caller(lib.moe_route_bwd, order, dict(
        logits=P[0], dtype=FP32, weight=P[1], idx=P[2], balance=P[3], dw=P[4], dl=P[5], out=P[6], T=9, E=8, k=2, norm=0,
        stream=None))
    for kw in (dict(T=-1), dict(dtype=7), dict(logits=0), dict(weight=0), dict(idx=0), dict(balance=0), dict(out=0),
               dict(out=P[6] + 2), dict(dw=P[4] + 1), dict(dl=P[5] + 2)):
        assert call(**kw) == EINVAL, kw
    assert call(E=2000) == EUNSUP and call(k=9) == EUNSUP
    for a in (P[0], P[1], P[2], P[3], P[4], P[5]):
        assert call(out=a) == EOVERLAP
    assert call(T=0) == OK and call(T=0, logits=0, weight=0, idx=0, out=0, dw=0, dl=0) == OK


def test_plan_refusals(lib):
    order = "idx offs dest T k E ws wsn stream".split()
    need = lib.moe_plan_workspace_bytes(5000, 4, 64)
    assert need == -(-5 * 64 * 4 // 256) * 256           # 20000 slots: 5 blocks of 4096
    assert lib.moe_plan_workspace_bytes(1024, 4, 64) == 0
    call = caller(lib.moe_plan, order, dict(idx=P[0], offs=P[1], dest=P[2], T=5000, k=4, E=64, ws=P[3], wsn=need,
                                            stream=None))
    for kw in (dict(T=-1), dict(k=0), dict(E=0), dict(idx=0), dict(offs=0), dict(dest=0), dict(idx=P[0] + 2),
               dict(ws=P[3] + 4)):
        assert call(**kw) == EINVAL, kw
    assert call(E=1025) == EUNSUP and call(k=33) == EUNSUP and call(T=2000000) == EUNSUP
    assert call(wsn=need - 1) == EWS
    for kw in (dict(dest=P[0]), dict(offs=P[0] + 16), dict(dest=P[1]), dict(ws=P[2])):
        assert call(**kw) == EOVERLAP, kw


def test_rows_refusals(lib):
    fns = {
        "moe_dispatch_fwd": ("x dest offs out T k E H dtype stream", "offs"),
        "moe_dispatch_bwd": ("x dest out T k H dtype stream", None),
        "moe_combine_fwd": ("x weight dest out T k H dtype stream", None),
        "moe_combine_bwd": ("dout x weight dest offs out dweight T k E H dtype stream", "offs"),
    }
    base = dict(x=P[0], dest=P[1], offs=P[2], out=P[3], weight=P[4], dout=P[5], dweight=P[6], T=8, k=2, E=4, H=64,
                dtype=BF16, stream=None)
    for name, (order, _) in fns.items():
        order = order.split()
        call = caller(getattr(lib, name), order, {n: base[n] for n in order})
        ptrs = [n for n in order if n in ("x", "dest", "offs", "out", "weight", "dout", "dweight")]
        for n in ptrs:
            assert call(**{n: 0}) == EINVAL, (name, n)
            assert call(**{n: base[n] + 2}) == EINVAL, (name, n)
            if n not in ("out", "dweight"):
                assert call(out=base[n]) == EOVERLAP, (name, n)
        assert call(T=-1) == EINVAL and call(k=0) == EINVAL and call(H=0) == EINVAL and call(dtype=3) == EINVAL
        assert call(H=4) == EUNSUP and call(H=2, dtype=FP32) == EUNSUP and call(H=(1 << 20) + 8) == EUNSUP
        assert call(k=33) == EUNSUP and call(T=3000000) == EUNSUP
        if "E" in order:
            assert call(E=0) == EINVAL and call(E=1025) == EUNSUP
        if "dweight" in order:
            assert call(dweight=P[3] + 16) == EOVERLAP
        assert call(T=0) == OK


def test_binding_refuses_what_is_not_on_the_device():
    l = torch.zeros((3, 8))
    i = torch.zeros((3, 2), dtype=torch.int32)
    pl = mdg.MoePlan(torch.zeros(8, dtype=torch.int32), i)
    for f in (lambda: mdg.moe_route_fwd(l, 2), lambda: mdg.moe_plan(i, 8), lambda: mdg.moe_dispatch_fwd(l, pl),
              lambda: mdg.moe_dispatch_bwd(l, pl), lambda: mdg.moe_combine_fwd(l, l, pl),
              lambda: mdg.moe_combine_bwd(l, l, l, pl)):
        with pytest.raises(ValueError, match="ROCm device"):
            f()
    with pytest.raises(TypeError):
        mdg.moe_route_fwd(l.double(), 2)
    with pytest.raises(TypeError):
        mdg.moe_route_fwd(None, 2)


def _num_grad(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        if not np.isfinite(x[i]):
            continue
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_route_gradient_is_the_difference_quotient(normalize):
    rng = np.random.default_rng(0)
    l = rng.normal(size=(5, 7))
    l[1, 3] = l[4, :] = -np.inf
    mask = np.array([1, 1, 0, 1, 1], dtype=bool)
    c = rng.normal(size=(5, 3))

    def f(x):
        w, _, _, loss, _ = ref.route(x, 3, normalize, mask)
        return (w * c).sum() + 0.4 * loss

    got = ref.route_grad(l, 3, c, 0.4, normalize, mask)
    # rounding of f (about 10 terms of size 1) over the step: 1e-15 * 10 / 1e-6
    assert np.max(np.abs(np.where(np.isfinite(l), _num_grad(f, l) - got, 0))) < 1e-8
    assert np.all(got[2] == 0) and np.all(got[4] == 0) and got[1, 3] == 0


def test_oracle_rows_gradients_are_the_difference_quotients():
    rng = np.random.default_rng(1)
    idx = rng.integers(-1, 4, (5, 2))
    _, dest = ref.plan(idx, 4)
    x, w, c = rng.normal(size=(5, 3)), rng.normal(size=(5, 2)), rng.normal(size=(5, 3))
    y, cr = rng.normal(size=(10, 3)), rng.normal(size=(10, 3))
    assert np.allclose(_num_grad(lambda v: (ref.dispatch(v, dest) * cr).sum(), x), ref.dispatch_grad(cr, dest), atol=1e-8)
    dy, dw = ref.combine_grad(c, y, w, dest)
    assert np.allclose(_num_grad(lambda v: (ref.combine(v, w, dest) * c).sum(), y), dy, atol=1e-8)
    assert np.allclose(_num_grad(lambda v: (ref.combine(y, v, dest) * c).sum(), w), dw, atol=1e-8)


def test_oracle_plan_by_hand():
    offs, dest = ref.plan(np.array([[2, 0], [-1, 2], [0, 5]]), 3)
    assert offs.tolist() == [2, 2, 4] and dest.tolist() == [[2, 0], [-1, 3], [1, -1]]
