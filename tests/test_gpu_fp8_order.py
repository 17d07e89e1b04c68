"""What the header promises of the order of the 8-bit product's sums, with the same
rows on both sides of the limits between its kernels (which kernel ran is read from
a trace of the launches)."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
SMALL, MIDDLE, TILE = "fp8_small_kernel", "fp8_mid_kernel", "fp8_gemm_kernel"


def draw(shape, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def run(x, w8, sizes):
    ends = torch.tensor(sizes).cumsum(0).to(device=DEV, dtype=torch.int32)
    return mdg.grouped_fp8_gemm_fwd(x, w8.q, w8.scale, ends)


def kernels(f):
    """The 8-bit product kernels that f() launches."""
    f()
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        f()
        torch.cuda.synchronize()
    return {k for k in (SMALL, MIDDLE, TILE) for e in prof.events() if k in e.name}


# rows of the call, its kernel: the first 8 rows are the same ones
CALLS = [(8, SMALL), (96, SMALL), (200, MIDDLE), (4096, TILE)]
N = 5120


@pytest.mark.parametrize("K", [128, 512, 640, 2048, 2056])
def test_the_same_rows_in_calls_of_different_sizes(K):
    """K <= 512: the same bits everywhere.  More: the same in the middle and the tile
    kernel; between those and the small one both sums are fp32 sums of the same groups
    of 8, each off by at most (K + 8) u sum |products|, rounded once."""
    x, w = draw((4096, K), 1), draw((1, N, K), 2)
    w8 = mdg.quantize_fp8_weight(w)
    y = {}
    for rows, kernel in CALLS:
        call = x[:rows].contiguous()
        assert kernels(lambda: run(call, w8, [rows])) == {kernel}
        y[rows] = run(call, w8, [rows])[:8]
    assert torch.equal(y[8], y[96]) and torch.equal(y[200], y[4096])
    if K <= 512:
        assert torch.equal(y[8], y[200])
        return
    # values of the 8-bit operands are within 2^-4 of x and w (and 2^-9 of a block's scale below its normal range)
    size = 1.25 * (x[:8].double().abs() + 0.01) @ (w[0].double().abs() + 0.01).t()
    apart = 2 * (K + 8) * U * size
    a, b = y[8].double(), y[200].double()
    place = 2.0 ** (torch.frexp(torch.maximum(a.abs(), b.abs()) + apart).exponent - 8)  # a bf16 place at their size
    assert torch.all((a - b).abs() <= apart + place)


@pytest.mark.parametrize("rows,kernel", CALLS)
def test_other_rows_and_the_cut_into_groups_do_not_matter(rows, kernel):
    """Another order of rows, other values in the other rows and other group sizes of
    equal weights leave a row's bits."""
    K, n = 1160, 1288 if rows < 4096 else N
    x, one = draw((rows, K), 3), draw((1, n, K), 4)
    w8 = mdg.quantize_fp8_weight(one.expand(2, n, K).contiguous())
    want = run(x, w8, [rows, 0])
    assert torch.equal(run(x, w8, [rows - 3, 3]), want)
    assert torch.equal(run(x, w8, [rows // 3, rows - rows // 3]), want)
    order = torch.randperm(rows, device=DEV)
    assert torch.equal(run(x[order].contiguous(), w8, [5, rows - 5]), want[order])
    other = draw((rows, K), 5)
    other[rows // 2] = x[rows // 2]
    assert torch.equal(run(other, w8, [rows, 0])[rows // 2], want[rows // 2])


def test_the_product_tests_reach_every_kernel():
    """The sizes that the products are tested at: each kernel has several of them
    (a changed limit between the kernels must not leave one untested)."""
    from test_gpu_fp8 import CASES, test_product_of_many_tiles as many
    tiles = [([rows // E] * (E - 1) + [rows - rows // E * (E - 1)], n, k)
             for E, rows, n, k in many.pytestmark[0].args[1]]
    count = {SMALL: 0, MIDDLE: 0, TILE: 0}
    for sizes, n, k in CASES + tiles:
        w8 = mdg.quantize_fp8_weight(torch.zeros((len(sizes), n, k), dtype=torch.bfloat16, device=DEV))
        x = torch.zeros((sum(sizes), k), dtype=torch.bfloat16, device=DEV)
        (kernel,) = kernels(lambda: run(x, w8, sizes))
        count[kernel] += 1
    assert all(c >= 3 for c in count.values()), count
