"""Shared-prefix decode at the edges of what its calls are given."""
import math

import pytest
import torch

import learned_kv_cache_gb300 as kvp
from tests.test_gpu_prefix import DT, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("G", [4, 16])
def test_more_work_than_the_plan_has_room_for(dtype, G):
    """128 rows of 2^29 tokens on a few pages, all members of one family of several items: nothing is read, the outputs are
    empty, the status says so; and the next call on the same buffers is served."""
    N, ps, D, pages = 128, 1024, 64, 1 << 19
    pool = [torch.randn(N + 5, ps, D, device="cuda").to(DT[dtype]) for _ in range(2)]
    table = torch.zeros(N, pages, dtype=torch.int32, device="cuda")
    table[:, :4] = torch.arange(4, dtype=torch.int32)
    table[:, 4] = 5 + torch.arange(N, dtype=torch.int32, device="cuda")
    lens = torch.full((N,), ps * pages, dtype=torch.int32, device="cuda")
    cache = kvp.PagedCache(*pool, table, lens, torch.ones(N + 5, dtype=torch.int32, device="cuda"),
                           torch.zeros((N + 36) // 32, dtype=torch.int32, device="cuda"))
    q = torch.randn(N, G, D, device="cuda").to(DT[dtype])
    lead = torch.zeros(N, dtype=torch.int32, device="cuda")
    bytes_ = kvp.load().kvp_paged_prefix_decode_attn_workspace_size(cache._ref, G, 1)
    workspace = torch.full((bytes_,), 0x7f, dtype=torch.uint8, device="cuda")       # as another call may have left it
    out, lse = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True, workspace=workspace)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_check_device_status()
    assert (out == 0).all() and torch.isneginf(lse).all()
    lens.fill_(4 * ps + 100)
    check(q, cache, lead, workspace=workspace)
