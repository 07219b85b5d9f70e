"""Shared-prefix decode at the edges of what its calls are given."""
import math

import pytest
import torch

import learned_kv_cache_gb300 as kvp
from tests.test_gpu_prefix import DT, PART, build, check, family

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


def row_of(cache, r):
    """Where row r's tokens lie: (pages, slots)."""
    t = torch.arange(int(cache.lens[r]), device="cuda")
    return cache.table[r].long()[t // cache.page_size], t % cache.page_size


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scale", [None, 0.31, -0.2])
@pytest.mark.parametrize("members,G", [(3, 1), (10, 4), (40, 4)])
def test_keys_of_minus_infinity_weigh_nothing(dtype, scale, members, G):
    """In the prefix and in own tokens, whole tiles of them among the others; the rest is as if they were not there (the bounds
    are test_gpu_prefix's, of the kept tokens).  A row of them alone is empty."""
    D, ps, n = 64, 32, 700
    rows, leads, shared = family(members, n, lambda i, h: i * 17 % 300, 1, ps)
    rows, leads, shared = rows + [[40]], leads + [members], shared + [[0]]
    q, cache, lead = build(rows, leads, 1, G, D, ps, DT[dtype], 3, shared)
    q = q.abs() + 0.1
    if scale is not None and scale < 0:
        q = -q
    gone = torch.zeros(1100, dtype=torch.bool, device="cuda")
    gone[[0, 5, 640, 702]] = True
    gone[128:384] = True
    kept = []
    for r in range(members + 1):
        page, slot = row_of(cache, r)
        dead = gone[:page.numel()] if r < members else torch.ones(40, dtype=torch.bool, device="cuda")
        cache.k_pool[page[dead], slot[dead], 7] = -math.inf
        kept.append((page[~dead], slot[~dead]))
    out, lse = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, sm_scale=scale, return_lse=True)
    kvp.kvp_check_device_status()
    assert (out[members] == 0).all() and torch.isneginf(lse[members]).all()
    s = D ** -0.5 if scale is None else scale
    for r in range(members):
        k, v = (pool[kept[r]].double() for pool in (cache.k_pool, cache.v_pool))
        x = q[r].double() @ k.T * s
        want_lse = torch.logsumexp(x, 1)
        p = torch.exp(x - want_lse[:, None])
        e = 2.0 ** -21 * abs(s) * (q[r].double().abs() @ k.abs().T).amax(1)
        step = torch.finfo(DT[dtype]).eps / 2
        tol = (4 * e + 2 * PART[DT[dtype]])[:, None] * (p @ v.abs()) + step * (1 + 2 ** -8) * (p @ v).abs()
        assert ((out[r].double() - p @ v).abs() <= tol).all(), r
        assert ((lse[r].double() - want_lse).abs() <= 2 * e + 2.0 ** -20 + 2.0 ** -23 * want_lse.abs()).all(), r


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("members,G", [(4, 4), (40, 4)])
def test_a_key_that_is_no_number_stays_with_its_rows(dtype, members, G):
    rows, leads, shared = family(members, 600, lambda i, h: 50 + i, 2, 64)
    q, cache, lead = build(rows, leads, 2, G, 64, 64, DT[dtype], 3, shared)
    want = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True)
    page, slot = row_of(cache, 2)                          # sequence 1, head 0: one of its own tokens
    cache.k_pool[page[640], slot[640], 3] = math.nan
    got = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True)
    for a, b in zip(got, want):
        assert a[1, :G].isnan().all() and torch.equal(a[1, G:], b[1, G:])
        assert all(torch.equal(a[n], b[n]) for n in range(members) if n != 1)
    page, slot = row_of(cache, 1)                          # the prompt's of head 1: every sequence's
    cache.k_pool[page[100], slot[100], 3] = math.nan
    got = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True)
    for a, b in zip(got, want):
        assert a[:, G:].isnan().all()
        assert all(torch.equal(a[n, :G], b[n, :G]) for n in range(members) if n != 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("members", [2, 12, 40])
def test_a_scale_of_zero_gives_the_mean(dtype, members):
    """Dot products up to 2^126, of either sign, weigh the same."""
    rows, leads, shared = family(members, 300, lambda i, h: i % 5 * 3, 1, 16)
    q, cache, lead = build(rows, leads, 1, 4, 64, 16, DT[dtype], 5, shared)
    cache.k_pool.mul_(2.0 ** 118)
    out, lse = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, sm_scale=0.0, return_lse=True)
    kvp.kvp_check_device_status()
    for r in range(members):
        v = cache.v_pool[row_of(cache, r)].double()
        # weights of 1 and exact parts; sums of some 300 in 32 bits, the tensor cores' cut off at 2^-23 a step
        tol = 2.0 ** -23 * 60 * v.abs().mean(0) + torch.finfo(DT[dtype]).eps / 2 * v.mean(0).abs() * (1 + 2 ** -8)
        assert ((out[r].double() - v.mean(0)).abs() <= tol).all(), r
        assert (lse[r].double() - math.log(v.shape[0])).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("dtype", list(DT))
def test_many_rows_of_which_some_are_empty(dtype):
    """1500 sequences in families of three: leads without a token or shorter than a page, members that share nothing, one page
    or more (too little to save anything)."""
    own = [(n * 131) % 90 + (64 if n % 3 else 0) if n % 7 else 0 for n in range(1500)]
    rows = [[n] for n in own]
    leads = [n - n % 3 for n in range(1500)]
    shared = [[min(own[n], own[l]) // 64 if n != l else 0] for n, l in enumerate(leads)]
    assert 0 in own and [1] in shared and [0] in shared
    check(*build(rows, leads, 1, 8, 64, 64, DT[dtype], 8, shared))
    # the same with prompts that are worth a prefix for some of them
    rows = [[n + (300 if leads[i] % 4 == 0 and n else 0)] for i, n in enumerate(own)]
    shared = [[min(rows[n][0], rows[l][0]) // 64 if n != l else 0] for n, l in enumerate(leads)]
    check(*build(rows, leads, 1, 8, 64, 64, DT[dtype], 9, shared))


@pytest.mark.parametrize("dtype,members", [("f32", 64), ("bf16", 16384), ("f16", 1), ("f32", 16384)])
def test_as_many_sequences_as_a_call_takes(dtype, members):
    """16384 of them, in families of 64, all in one, or each alone."""
    N, ps = 16384, 16
    rows = [[64 + n * 37 % 40 if n % 5 else n * 37 % 40] for n in range(N)]
    leads = [n - n % members for n in range(N)]
    rows = [[max(r[0], 70)] if n % members == 0 else r for n, r in enumerate(rows)]
    shared = [[min(rows[n][0], rows[l][0]) // ps if n != l else 0] for n, l in enumerate(leads)]
    check(*build(rows, leads, 1, 2, 64, ps, DT[dtype], 10, shared))


@pytest.mark.parametrize("dtype", list(DT))
def test_some_rows_of_a_cache(dtype):
    """The rows of four sequences in the middle, on the pages of all."""
    rows, leads, shared = family(8, 700, lambda i, h: i * 23 + h, 2, 32, first=2)
    q, cache, _ = build(rows, leads, 2, 4, 64, 32, DT[dtype], 4, shared)
    check(q[2:6].contiguous(), cache.rows(4, 12), torch.tensor([0, 0, 0, -1], dtype=torch.int32, device="cuda"))
    check(q[5:], cache.rows(10, 16), torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_past_32_bits(dtype):
    """Pages whose first value is number 2^31 and more of the pool, in prefixes and own tokens."""
    ps, D = 1024, 128
    n_pages = 2 ** 31 // (ps * D) + 40
    pool = [torch.empty(n_pages, ps, D, dtype=DT[dtype], device="cuda") for _ in range(2)]
    gen = torch.Generator("cuda").manual_seed(0)
    for p in pool:
        p[-40:].normal_(generator=gen)
    N, G = 9, 4
    table = torch.zeros(N, 8, dtype=torch.int32)
    table[:, :3] = torch.tensor([n_pages - 1, n_pages - 17, n_pages - 5])
    table[:, 3] = n_pages - 30 + torch.arange(N, dtype=torch.int32)
    cache = kvp.PagedCache(*pool, table.cuda(), torch.full((N,), 3 * ps + 333, dtype=torch.int32, device="cuda"),
                           torch.ones(n_pages, dtype=torch.int32, device="cuda"),
                           torch.zeros((n_pages + 31) // 32, dtype=torch.int32, device="cuda"))
    q = torch.randn(N, G, D, generator=gen, device="cuda").to(DT[dtype])
    for lead in (torch.zeros(N, dtype=torch.int32), torch.full((N,), -1, dtype=torch.int32)):
        check(q, cache, lead.cuda())


@pytest.mark.parametrize("dtype", list(DT))
def test_two_captured_calls_take_turns(dtype):
    """Two graphs of one pool of memory, replayed in turn while the cache grows: each has what it needs of its own."""
    rows, leads, shared = family(6, 900, lambda i, h: i * 31, 2, 32)
    q, cache, lead = build(rows, leads, 2, 4, 64, 32, DT[dtype], 4, shared, max_pages=40)
    other = torch.full_like(lead, -1)
    kvp.kvp_paged_prefix_decode_attn(q, cache, lead)
    graphs, outs = [], []
    for l in (lead, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=graphs[0].pool() if outs else None):
            outs.append(kvp.kvp_paged_prefix_decode_attn(q, cache, l, return_lse=True))
    for step in range(4):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (out, lse), l in zip(outs, (lead, other)):
            want, want_lse = kvp.kvp_paged_prefix_decode_attn(q, cache, l, return_lse=True)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        check(q, cache, lead)
        cache.lens[step] -= 100 * step
        q.normal_()
