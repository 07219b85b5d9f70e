"""The paged cache at the edges of what its calls are given: infinite keys, rows whose kept tokens are named wrongly."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests.test_gpu_paged import DT, filled, i32, kvp, raises_status, rows_of  # noqa: F401 (kvp is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,G", [(128, 1), (128, 2), (128, 4), (64, 8), (128, 8), (128, 16)])
@pytest.mark.parametrize("sm_scale", [None, 0.31, 0.25, 0.125 / 1.4426950408889634])
def test_keys_of_minus_infinity_weigh_nothing(kvp, dtype, D, G, sm_scale):  # noqa: F811
    """Whatever the scale's float leaves behind: log2(e) times these is a little more, or less, than its float.

    Bound: a logit is off by d = (D + 4) 2^-23 scale sum |q_i k_i| at most, exp2 by 2^-22, a weight's split by 2^-23,
    each of at most n / 16 + 64 sums by 2^-23; weight and normaliser share d."""
    ps = 16
    c = filled(kvp, [100, 700, 3], ps, D, dtype, seed=D + G, scores=True)
    c.score.zero_()
    gen = torch.Generator().manual_seed(G)
    q = (torch.rand(1, 3 * G, D, generator=gen) + 0.1).to(DT[dtype]).cuda()
    gone = {0: [0, 40, 99], 1: list(range(128, 256)) + [699], 2: [0, 1, 2]}
    t = c.table.cpu()
    for r, tokens in gone.items():
        for j in tokens:
            c.k_pool[t[r, j // ps], j % ps, (7 * j) % D] = float("-inf")
    out, lse = kvp.kvp_paged_decode_attn(q, c, sm_scale=sm_scale, return_lse=True, add_scores=True)
    kvp.kvp_check_device_status()
    k, v = rows_of(c)
    kept = [[j for j in range(x.shape[0]) if j not in gone[r]] for r, x in enumerate(k)]
    scale = D ** -0.5 if sm_scale is None else sm_scale
    ref, ref_lse, mass, mag = paged.paged_decode_attn(q, [x[i] for x, i in zip(k, kept)], [x[i] for x, i in zip(v, kept)],
                                                      scale)
    out, lse, score = out.double().cpu().numpy(), lse.double().cpu().numpy(), c.score.double().cpu().numpy()
    for r in range(3):
        h = slice(r * G, (r + 1) * G)
        if not kept[r]:
            assert (out[0, h] == 0).all() and np.isneginf(lse[0, h]).all() and (score[r] == 0).all()
            continue
        n = k[r].shape[0]
        logit = (D + 4) * 2.0 ** -23 * scale * (k[r][kept[r]].double().abs().numpy() @ q[0, h].double().abs().cpu().numpy().T).max()
        eps = 2 * logit + 2.0 ** -21 + 2 * (n / 16 + 64) * 2.0 ** -23
        assert (np.abs(out[0, h] - ref[0, h]) <= eps * mag[0, h] + 2.0 ** -23 * np.abs(ref[0, h])).all(), r
        assert (np.abs(lse[0, h] - ref_lse[0, h]) <= eps + logit + 2.0 ** -22 * (np.abs(ref_lse[0, h]) + 1)).all(), r
        assert (score[r, gone[r]] == 0).all() and (score[r, n:] == 0).all()
        assert (np.abs(score[r, kept[r]] - mass[r]) <= (eps + logit + 2.0 ** -20) * mass[r]).all(), r
