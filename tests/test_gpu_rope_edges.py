"""Rotation and norms at the edges of what their calls are given."""
import pytest
import torch

import learned_kv_cache_gb300 as kvp
from oracle import rope as oracle

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


@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines_everywhere(interleaved):
    """The unit vector turned.  Off by: the angle as a float, 2^-28 of a turn (2.4e-8); its product with 2 pi, half a step of
    pi / 4 and 2 pi's own (7e-8); all of it times sin(pi / 4); the series 1.8e-9 and its last roundings (6e-8): 2^-22.8."""
    D = 128
    gen = torch.Generator("cuda").manual_seed(0)
    first, second = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    rope = kvp.Rope(D, theta=1e6, interleaved=interleaved)

    def turned(positions):
        x = torch.zeros(1, positions.numel(), D, device="cuda")
        x[..., first] = 1.0
        return x, kvp.kvp_rope(x, rope, positions=positions.to(torch.int32))[0].double()

    # up to 2^20 angles in 64 bits (2^-30 of a radian)
    pos = torch.randint(-2 ** 20, 2 ** 20, (40000,), generator=gen, device="cuda")
    y = turned(pos)[1]
    angle = pos.double()[:, None] * torch.tensor(rope.inv_freq, dtype=torch.float64, device="cuda")
    for got, want in ((y[:, first], torch.cos(angle)), (y[:, second], torch.sin(angle))):
        assert ((got - want).abs() <= 2.0 ** -22 + 2.0 ** -30).all(), (got - want).abs().max().item()
    # beyond, whole turns leave in rational numbers
    pos = torch.cat([torch.randint(-2 ** 31, 2 ** 31, (250,), generator=gen, device="cuda"),
                     torch.tensor([2 ** 31 - 1, -2 ** 31], device="cuda")])
    x, y = turned(pos)
    want = oracle.rotate(x[0].double().cpu().numpy(), pos.cpu().numpy(), rope.inv_freq, interleaved)
    assert (y.cpu() - torch.from_numpy(want)).abs().max() <= 2.0 ** -22
