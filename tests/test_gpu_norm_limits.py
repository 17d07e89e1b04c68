"""The block norm at the most rows it takes."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, bf16

pytestmark = pytest.mark.gpu


def test_the_most_rows_of_a_norm():
    """4,000,000 tokens, the limit; one more is refused."""
    t, h = 4_000_000, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x, y = bf16((t + 1, h), g), bf16((t + 1, h), g)
    w = 1 + torch.randn(h, generator=g, device=DEV) / 4
    r = mdg.block_norm_fwd(x[:t], y[:t], weight=w, post_weight=w, scale=0.5)
    d = mdg.block_norm_bwd(x[:t], y[:t], r, y[:t], weight=w, post_weight=w, scale=0.5)
    for rows in (slice(0, 1000), slice(t - 1000, t)):
        a, b = x[rows].contiguous(), y[rows].contiguous()
        one = mdg.block_norm_fwd(a, b, weight=w, post_weight=w, scale=0.5)
        back = mdg.block_norm_bwd(a, b, one, b, weight=w, post_weight=w, scale=0.5)
        assert torch.equal(r.out[rows], one.out) and torch.equal(r.normed[rows], one.normed)
        assert torch.equal(d.dresidual[rows], back.dresidual) and torch.equal(d.dy[rows], back.dy)
    with pytest.raises(mdg.MdgError):
        mdg.block_norm_fwd(x, weight=w)
