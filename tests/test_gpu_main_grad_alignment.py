"""main_grads that start anywhere in a flat gradient buffer: the same sums, bit for
bit, as in tensors of their own, and the buffer's other values left alone."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def randn(*s, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(s, generator=g, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("by", [1, 5])
def test_main_grads_in_a_flat_buffer(dtype, by):
    x, dy = randn(50, 40, seed=1).bfloat16(), randn(50, 40, seed=2).bfloat16()
    w, w2 = (randn(2, 48, 40, seed=3) / 6).bfloat16(), (randn(2, 40, 24, seed=4) / 5).bfloat16()
    offs = torch.tensor([20, 50], dtype=torch.int32, device=DEV)
    start = randn(w.numel() + w2.numel() + by + 9, seed=5).to(dtype)
    flat = start.clone()
    cut = by + w.numel()
    for apart in (True, False):
        a, b = (t.clone().requires_grad_() for t in (w, w2))
        a.main_grad, b.main_grad = flat[by:cut].view(w.shape), flat[cut:cut + w2.numel()].view(w2.shape)
        if apart:
            a.main_grad, b.main_grad = a.main_grad.clone(), b.main_grad.clone()
        for _ in range(2):
            mdg.grouped_gated_ffn(x, a, b, offs, fuse_wgrad_accumulation=True).backward(dy)
            mdg.cake_grouped_det_mm(x, a, offs, fuse_wgrad_accumulation=True).sum().backward()
        if apart:
            want = (a.main_grad, b.main_grad)
            assert torch.equal(flat, start)
    assert torch.equal(a.main_grad, want[0]) and torch.equal(b.main_grad, want[1])
    assert torch.equal(flat[:by], start[:by]) and torch.equal(flat[cut + w2.numel():], start[cut + w2.numel():])
