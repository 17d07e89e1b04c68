"""The grouped product in 8 bits without a GPU: the C ABI's refusals, the
binding's, workspace rules, and the oracle against brute force.

Pointers below are fake, aligned addresses: every case returns before any device
access.
"""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import fp8 as ref

OK, EINVAL, EUNSUP, EOVERLAP, EWS, EHIP, ENOMEM = range(7)
BF16, FP32, E4M3 = 0, 1, 2
P = [0x10000000 * i for i in range(1, 10)]


@pytest.fixture(scope="module")
def lib():
    return mdg.load_library()


def caller(fn, order, defaults):
    def call(**kw):
        assert set(kw) <= set(defaults)
        return fn(*[{**defaults, **kw}[n] for n in order])
    return call


def test_quantize_rows_refusals(lib):
    call = caller(lib.grouped_fp8_quantize_rows, "x dtype q scale M K stream".split(),
                  dict(x=P[0], dtype=BF16, q=P[1], scale=P[2], M=100, K=256, stream=None))
    for kw in (dict(M=-1), dict(K=0), dict(dtype=E4M3), dict(dtype=9), dict(x=0), dict(q=0), dict(scale=0),
               dict(x=P[0] + 8), dict(q=P[1] + 4), dict(scale=P[2] + 2)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(K=20), dict(K=(1 << 20) + 16), dict(M=4000001)):
        assert call(**kw) == EUNSUP, kw
    assert call(q=P[0] + 16) == EOVERLAP and call(scale=P[0] + 4) == EOVERLAP and call(scale=P[1] + 100 * 256 - 4) == EOVERLAP
    assert call(M=0) == OK and call(M=0, x=0, q=0, scale=0) == OK


def test_quantize_weight_refusals(lib):
    call = caller(lib.grouped_fp8_quantize_weight, "w dtype q scale qt st E N K stream".split(),
                  dict(w=P[0], dtype=BF16, q=P[1], scale=P[2], qt=P[3], st=P[4], E=4, N=256, K=512, stream=None))
    for kw in (dict(E=0), dict(N=0), dict(K=-16), dict(dtype=E4M3), dict(w=0), dict(q=0), dict(scale=0), dict(qt=0),
               dict(st=0), dict(w=P[0] + 8), dict(q=P[1] + 8), dict(qt=P[3] + 8)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(E=1025), dict(N=260), dict(K=516), dict(N=1 << 17, K=1 << 14)):
        assert call(**kw) == EUNSUP, kw
    for kw in (dict(q=P[0]), dict(qt=P[1]), dict(st=P[2]), dict(scale=P[3] + 5), dict(st=P[0] + 3)):
        assert call(**kw) == EOVERLAP, kw


def test_gemm_refusals_and_workspace(lib):
    wsf = lib.grouped_fp8_gemm_fwd_workspace_bytes
    need = wsf(300, 256, 528, 4, BF16)
    # q, then 5 blocks of scales in 2 words a row
    assert need == -(-(-(-300 * 528 // 256) * 256 + 2 * 300 * 4) // 256) * 256
    assert wsf(300, 256, 528, 4, E4M3) == 0 and wsf(300, 256, 524, 4, BF16) == 0 and wsf(300, 256, 520, 4, BF16) == need and wsf(300, 256, 528, 4, 5) == 0
    call = caller(lib.grouped_fp8_gemm_fwd, "x dt xs w sw offs y M N K E ws wsn stream".split(),
                  dict(x=P[0], dt=BF16, xs=0, w=P[1], sw=P[2], offs=P[3], y=P[4], M=300, N=256, K=528, E=4, ws=P[5],
                       wsn=need, stream=None))
    for kw in (dict(M=-1), dict(N=0), dict(E=0), dict(dt=4), dict(x=0), dict(w=0), dict(sw=0), dict(offs=0), dict(y=0),
               dict(xs=P[6]), dict(dt=E4M3), dict(x=P[0] + 8), dict(w=P[1] + 4), dict(offs=P[3] + 2), dict(y=P[4] + 8),
               dict(dt=E4M3, xs=P[6] + 2), dict(ws=P[5] + 16)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(N=100), dict(K=524), dict(E=1025)):
        assert call(**kw) == EUNSUP, kw
    assert call(ws=0) == EWS and call(wsn=need - 1) == EWS
    for kw in (dict(y=P[0]), dict(y=P[1] + 16), dict(y=P[2]), dict(y=P[3]), dict(y=P[5]), dict(ws=P[0]), dict(ws=P[1]),
               dict(dt=E4M3, xs=P[4] + 8)):
        assert call(**kw) == EOVERLAP, kw
    assert call(M=0, x=0, y=0, wsn=0, ws=0) == OK
    assert call(M=0, dt=E4M3, x=0, y=0, ws=0, wsn=0) == OK


def test_binding_refusals():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((2, 32, 64), dtype=torch.bfloat16)
    offs = torch.zeros(2, dtype=torch.int32)
    for f in (lambda: mdg.quantize_fp8_rows(x), lambda: mdg.quantize_fp8_weight(w),
              lambda: mdg.grouped_fp8_gemm_fwd(x, w, w, offs), lambda: mdg.grouped_fp8_mm(x, w, offs)):
        with pytest.raises(ValueError, match="ROCm device"):
            f()
    with pytest.raises(TypeError):
        mdg.quantize_fp8_rows(x.double())
    with pytest.raises(TypeError):
        mdg.quantize_fp8_weight(w.double())
    with pytest.raises(TypeError):
        mdg.quantize_fp8_weight(w, transpose=1)
    with pytest.raises(TypeError):
        mdg.fp8_gemm_fwd_workspace_bytes(10, 32, 64, 2, torch.float64)
    assert mdg.fp8_gemm_fwd_workspace_bytes(10, 32, 64, 2, torch.float8_e4m3fn) == 0


def test_oracle_rounds_to_the_nearest_e4m3_value():
    """Against all finite e4m3 values, decoded from their bits by definition."""
    v = []
    for b in range(128):
        e, m = b >> 3, b & 7
        if b != 127:
            v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v = np.array(v)
    assert v.max() == 448 and np.all(np.diff(v) > 0)
    rng = np.random.default_rng(0)
    mid = (v[1:] + v[:-1]) / 2
    u = np.concatenate([v, mid, mid * (1 + 1e-12), mid * (1 - 1e-12), rng.uniform(0, 448, 2000), rng.uniform(0, 0.02, 500)])
    got = ref.e4m3(np.concatenate([u, -u]))
    for x, g in zip(u, got):
        d = np.abs(v - x)
        near = np.nonzero(d == d.min())[0]
        assert g == v[near[0] if len(near) == 1 else near[near % 2 == 0][0]], x      # ties: even mantissa
    assert np.array_equal(got[len(u):], -got[:len(u)])


def test_oracle_scales():
    """The smallest power of two with amax <= 448 * scale, searched."""
    for amax in [448.0, np.nextafter(448, 500), 1.0, 1.75, 1.7500001, 3.4e38, 1e-40, 448 * 2.0 ** -127, 0.0, 2.0 ** -149]:
        x = np.zeros((1, 128))
        x[0, 3] = -amax
        q, c = ref.quantize_rows(x)
        want = next(e for e in range(-127, 128) if amax <= 448 * 2.0 ** e)
        assert c[0, 0] == want + 127, amax
        assert abs(q[0, 3]) <= 448
    q, c = ref.quantize_weight(np.full((1, 130, 10), 2.0))
    assert c.shape == (1, 2, 1) and np.all(ref.dequantize(q, c, (128, 128)) == 2.0)


def test_oracle_group_sums_by_hand():
    """256 + 2^-5 keeps, 256 + 2^-6 loses the small product; products in another
    group of 8 are apart; a zero product does not set the alignment."""
    a, b = np.zeros((4, 16)), np.ones((4, 16))
    a[:, 0], b[:, 0] = 16, 16
    a[0, 1], a[1, 1], a[2, 8] = 2.0 ** -5, 2.0 ** -6, 2.0 ** -6
    a[3, 0], a[3, 1] = 0, 2.0 ** -6
    assert ref.group_sums(a, b).sum(axis=1).tolist() == [256 + 2.0 ** -5, 256, 256 + 2.0 ** -6, 2.0 ** -6]


def test_matrix_instructions_keep_their_distance_from_writes_of_their_sources():
    from moe_ragged_bf16_amd import build
    mfma = "\tv_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[8:15], v[16:23], a[0:3], v30, v31 op_sel_hi:[0,0,0]\n"
    bad = lambda pre: build.mfma_source_hazards(pre + mfma)
    assert bad("\tv_mov_b32_e32 v10, v1\n") and bad("\tv_lshrrev_b32_e32 v31, 8, v31\n\ts_nop 0\n")
    assert bad("\tv_accvgpr_write_b32 a2, v1\n\tv_add_u32_e32 v40, v1, v2\n")
    assert not bad("\tv_mov_b32_e32 v10, v1\n\ts_nop 1\n") and not bad("\tv_mov_b32_e32 v24, v10\n")
    assert not bad("\tv_mov_b32_e32 v10, v1\n\tv_mov_b32_e32 v1, v2\n\ts_mov_b32 s0, s1\n")
    assert not bad("\tds_read_b128 v[8:11], v1\n\ts_waitcnt lgkmcnt(0)\n")
    build.check_mfma_sources(build.LIB_PATH)
