"""Rotation and norms at the edges of what their calls are given."""
import pytest
import torch

import learned_kv_cache_gb300 as kvp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [2 ** 31, -2 ** 31 - 1, 2 ** 32 + 7, -2 ** 32, 2 ** 40])
def test_positions_that_do_not_fit_32_bits(start):
    rope = kvp.Rope(64)
    x = torch.randn(1, 2, 3, 64, device="cuda")
    for call in (lambda: kvp.kvp_rope(x, rope, start=start), lambda: kvp.kvp_qk_norm_rope(x, x, rope=rope, start=start),
                 lambda: kvp.kvp_qk_norm_rope_backward(x, x, x, x, rope=rope, start=start)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("start", [2 ** 31 - 3, -2 ** 31])
def test_the_last_positions_that_do(start):
    """The same as with the positions given."""
    rope = kvp.Rope(64, theta=1e6)
    x = torch.randn(1, 2, 3, 64, device="cuda")
    positions = torch.arange(start, start + 3, device="cuda").to(torch.int32)
    assert torch.equal(kvp.kvp_rope(x, rope, start=start), kvp.kvp_rope(x, rope, positions=positions))
    a, b = kvp.kvp_qk_norm_rope(x, x, rope=rope, start=start), kvp.kvp_qk_norm_rope(x, x, rope=rope, positions=positions)
    assert all(torch.equal(*p) for p in zip(a, b))
    a, b = (kvp.kvp_qk_norm_rope_backward(x, x, x, x, rope=rope, **kw) for kw in ({"start": start}, {"positions": positions}))
    assert all(torch.equal(*p) for p in zip(a, b))
