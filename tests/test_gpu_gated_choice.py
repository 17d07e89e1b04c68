"""The kernel that takes a gated product, as a trace of the launches names it, against
the rules that tests/_gated.py restates and other tests choose their sizes by."""
import random
import re

import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, variant_of
from test_gpu_gated import SIZES

pytestmark = pytest.mark.gpu
LAUNCH = re.compile(r"gated_(small_|mid_|)kernel<([^>]*)>")


def form_of(name):
    """variant_of()'s form from a kernel's name, None for other kernels."""
    m = LAUNCH.search(name)
    if not m:
        return None
    kind, args = m.group(1), [a.strip().split(")")[-1] for a in m.group(2).split(",")]
    flag = {"true": True, "1": True, "false": False, "0": False}
    if kind == "small_":
        return ("fwd", "small")
    op = {"0": "fwd", "1": "dgrad"}[args[0]]
    return (op, "mid", int(args[2])) if kind == "mid_" else (op, "tile", flag[args[3]], flag[args[4]])


def draw(rng):
    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    while True:
        m, e, f, k = log(1, 20_000), log(1, 1024), 8 * log(1, 400), 8 * log(1, 300)
        if e * f * k <= 6e7 and m * f <= 3e7:
            return m, e, f, k


def test_the_rules_restated_here_are_the_librarys():
    rng = random.Random(5)
    cases = [(sum(s), len(s), f, k) for s, f, k, _ in SIZES] + [(sum(s), len(s), f, n) for s, f, _, n in SIZES]
    cases += [draw(rng) for _ in range(150)]
    flat = torch.zeros(220_000_000, dtype=torch.bfloat16, device=DEV)       # (every operand: only the choice matters)

    def zeros(*shape):
        n = 1
        for s in shape:
            n *= s
        return flat[:n].view(shape)

    want, calls = [], []
    for m, e, f, n in cases:
        if m == 0:
            continue
        offs = torch.full((e,), m, dtype=torch.int32, device=DEV)
        want += [variant_of("fwd", m, e, n, f), variant_of("dgrad", m, e, n, f)]
        calls += [lambda m=m, e=e, f=f, n=n, offs=offs: mdg.grouped_gated_gemm_fwd(zeros(m, n), zeros(e, 2 * f, n), offs),
                  lambda m=m, e=e, f=f, n=n, offs=offs: mdg.grouped_gated_gemm_dgrad(
                      zeros(m, n), zeros(e, n, f), zeros(m, 2 * f), offs)]
    calls[0]()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        for c in calls:
            c()
        torch.cuda.synchronize()
    launched = sorted((e.time_range.start, form_of(e.name)) for e in prof.events() if form_of(e.name))
    assert [f for _, f in launched] == want
    assert len(set(want)) == 10                              # (every form)
