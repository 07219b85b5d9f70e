"""Decode attention over shared prefixes against the formula in 64 bits, row by row.

Bounds.  A logit is a sum of head_dim products in 32 bits, whose partial sums may drop bits: off by e = 2^-21 of
scale * sum |q k|, one factor 2 for its scaling and for the maximum that is subtracted.  A weight is then off by 2e of
itself and, as two 16-bit parts, by 2^-16 (bf16; f16: 2^-21; fp32: 2^-22, the exponential's own); so is the sum of the
weights, and both errors are relative to sum p |v|.  The output's rounding is half a step of its type.  The log-sum-exp is
off by 2e, by the sum's own 2^-20 and by half a step of a float.
"""
import math

import pytest
import torch

import learned_kv_cache_gb300 as kvp

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PART = {torch.float32: 2.0 ** -22, torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21}


def build(rows, leads, h_kv, G, D, ps, dtype, seed=0, shared=None, max_pages=None, interleaved=False):
    """A cache with rows[n][h] tokens; sequence n has its first shared[n][h] pages in common with its lead's row.  Pages
    anywhere in the pool, NaN in every slot without a token.  (q, cache, lead)"""
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    N = len(rows)
    pages = [[-(-n // ps) for n in r] for r in rows]
    max_pages = max_pages or max(1, max(max(p) for p in pages)) + 1
    owned = sum(p - (shared[n][h] if leads[n] >= 0 and leads[n] != n else 0) for n, r in enumerate(pages) for h, p in enumerate(r))
    n_pages = owned + 5
    free = torch.randperm(n_pages, generator=host).tolist()
    table = torch.full((N, h_kv, max_pages), -1, dtype=torch.int32)
    refs = [0] * n_pages
    for n in sorted(range(N), key=lambda n: leads[n] >= 0 and leads[n] != n):
        for h in range(h_kv):
            follows = leads[n] >= 0 and leads[n] != n
            k = shared[n][h] if follows else 0
            ids = table[leads[n], h, :k].tolist() + [free.pop() for _ in range(pages[n][h] - k)]
            assert -1 not in ids
            for i in ids:
                refs[i] += 1
            table[n, h, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    if interleaved:
        kv = torch.full((n_pages, 2, ps, D), math.nan, dtype=dtype, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
    else:
        k, v = (torch.full((n_pages, ps, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    table = table.reshape(N * h_kv, max_pages).cuda()
    lens = torch.tensor(rows, dtype=torch.int32).reshape(-1).cuda()
    slots = torch.arange(max_pages * ps, device="cuda") < lens[:, None]
    slot = (table.long()[:, :, None] * ps + torch.arange(ps, device="cuda")).reshape(N * h_kv, -1)[slots].unique()
    for pool in (k, v):
        pool[slot // ps, slot % ps] = torch.randn(slot.numel(), D, generator=gen, device="cuda").to(dtype)
    free_mask = torch.zeros((n_pages + 31) // 32, dtype=torch.int32)
    for i, c in enumerate(refs):
        if c == 0:
            free_mask[i // 32] |= -(1 << 31) if i % 32 == 31 else 1 << i % 32
    cache = kvp.PagedCache(k, v, table, lens, torch.tensor(refs, dtype=torch.int32).cuda(), free_mask.cuda())
    q = torch.randn(N, h_kv * G, D, generator=gen, device="cuda").to(dtype)
    return q, cache, torch.tensor(leads, dtype=torch.int32, device="cuda")


def reference(q, cache, scale=None):
    """(out, lse, bound on out, bound on lse), all fp64."""
    N, Hq, D = q.shape
    R = cache.n_rows
    G = N * Hq // R
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(R, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, G), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    q = q.double().reshape(R, G, D)
    for r, n in enumerate(cache.lens.tolist()):
        if n == 0:
            continue
        held = cache.table[r, :(n - 1) // cache.page_size + 1].long()
        k, v = (p[held].reshape(-1, D)[:n].double() for p in (cache.k_pool, cache.v_pool))
        x = q[r] @ k.T * scale
        lse[r] = torch.logsumexp(x, 1)
        p = torch.exp(x - lse[r][:, None])
        out[r] = p @ v
        e = 2.0 ** -21 * abs(scale) * (q[r].abs() @ k.abs().T).amax(1)
        tol[r] = (4 * e + 2 * PART[cache.dtype])[:, None] * (p @ v.abs()) + torch.finfo(cache.dtype).eps / 2 * (1 + 2 ** -8) * out[r].abs()
        tol_lse[r] = 2 * e + 2.0 ** -20 + 2.0 ** -23 * lse[r].abs()
    return out.view(N, Hq, D), lse.view(N, Hq), tol.view(N, Hq, D), tol_lse.view(N, Hq)


def check(q, cache, lead, scale=None, **kw):
    out, lse = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, sm_scale=scale, return_lse=True, **kw)
    kvp.kvp_check_device_status()
    assert out.dtype == cache.dtype
    want, want_lse, tol, tol_lse = reference(q, cache, scale)
    err = (out.double() - want).abs()
    assert bool((err <= tol + torch.finfo(cache.dtype).tiny).all()), (err - tol).max()
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse), empty) and (out[empty] == 0).all()
    err = torch.where(empty, 0.0, (lse.double() - want_lse).abs())
    assert bool((err <= tol_lse).all()), (err - tol_lse).max()
    return out, lse


def family(members, prompt, own, h_kv, ps, first=0):
    """One family whose members share the prompt's whole pages: (rows, leads, shared)."""
    rows = [[prompt + own(n, h) for h in range(h_kv)] for n in range(members)]
    return rows, [first] * members, [[prompt // ps] * h_kv for _ in range(members)]


SHAPES = [  # members, prompt, own tokens, h_kv, G, page size
    (2, 700, 5, 1, 1, 64), (3, 300, 0, 2, 4, 16), (5, 1000, 130, 2, 16, 32), (9, 513, 40, 1, 16, 128), (40, 600, 17, 1, 8, 64),
    (33, 2100, 260, 2, 4, 256), (17, 4096, 1, 1, 16, 1024), (2, 129, 1, 3, 5, 16), (70, 272, 3, 1, 7, 16)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_one_family(dtype, D, shape):
    members, prompt, own, h_kv, G, ps = shape
    rows, leads, shared = family(members, prompt, lambda n, h: (n * 37 + h * 11) % (own + 1), h_kv, ps)
    check(*build(rows, leads, h_kv, G, D, ps, DT[dtype], members, shared))


@pytest.mark.parametrize("dtype", list(DT))
def test_rows_alone(dtype):
    """No families: every length from nothing to a few tiles, one row longer than the rest together."""
    rows = [[n, (n * 7) % 400] for n in (0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 5000)]
    check(*build(rows, [-1] * len(rows), 2, 3, 64, 32, DT[dtype]))
    check(*build(rows, list(range(len(rows))), 2, 4, 128, 64, DT[dtype]))
    check(*build([[0]], [0], 1, 2, 64, 16, DT[dtype]))
    check(*build([[1]], [-1], 1, 16, 128, 16, DT[dtype]))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
def test_families_strays_and_empty_rows(dtype, D):
    """Families of several sizes in any order, their leads anywhere, heads of different lengths, members that have shared
    less since, rows without tokens."""
    ps, h_kv, G = 32, 3, 4
    leads = [3, -1, 3, 3, 8, 3, 6, 8, 8, 3, 8, -1, 3, 8, 3]
    prompt = {3: (900, 64, 2000), 8: (300, 1500, 31)}
    rows, shared = [], []
    for n, l in enumerate(leads):
        if l in prompt:
            rows.append([prompt[l][h] + (n * 53 + h * 19) % 200 for h in range(h_kv)])
            shared.append([prompt[l][h] // ps for h in range(h_kv)])
        else:
            rows.append([0, 77, 0] if n == 11 else [400, 0, 33])
            shared.append([0] * h_kv)
    shared[5] = [4, 0, 60]                                # evicted by itself
    rows[9], shared[9] = [0, 10, 1999], [0, 0, 62]        # cut short: fewer tokens than the prompt
    rows[10], shared[10] = [320, 1500, 0], [9, 46, 0]
    check(*build(rows, leads, h_kv, G, D, ps, DT[dtype], 4, shared))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0, 1e-30, 2.0])
def test_scales(dtype, scale):
    rows, leads, shared = family(6, 400, lambda n, h: n * 30, 2, 32)
    check(*build(rows, leads, 2, 4, 64, 32, DT[dtype], 1, shared), scale=scale)


@pytest.mark.parametrize("dtype", list(DT))
def test_growing_maximum(dtype):
    """Logits that grow along the tokens, so that the running maximum moves again and again; then a sink first."""
    rows, leads, shared = family(10, 3000, lambda n, h: 100 + n, 1, 64)
    for sign in (1, -1):
        q, cache, lead = build(rows, leads, 1, 4, 64, 64, DT[dtype], 2, shared)
        direction = q.double().mean((0, 1))
        direction = direction / direction.norm()
        q.copy_((q.double() + 3 * direction).to(q.dtype))
        for r in range(10):
            n = rows[r][0]
            t = torch.arange(n, device="cuda").double()
            add = (t if sign > 0 else n - 1 - t) / n * 40
            page, slot = cache.table[r].long()[(t // 64).long()], (t % 64).long()
            base = torch.randn(n, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).double()
            cache.k_pool[page, slot] = (base + add[:, None] * direction).to(q.dtype)
        check(q, cache, lead)


def test_pools_side_by_side_and_strided_queries():
    rows, leads, shared = family(7, 500, lambda n, h: n * 9, 2, 64)
    for dtype in DT.values():
        q, cache, lead = build(rows, leads, 2, 4, 128, 64, dtype, 5, shared, max_pages=40, interleaved=True)
        want, lse = check(q, cache, lead)
        wide = torch.zeros(7, 3, 8, 128, dtype=dtype, device="cuda")
        wide[:, 1] = q
        out = torch.empty_like(want)
        got = kvp.kvp_paged_prefix_decode_attn(wide[:, 1], cache, lead, out=out)
        assert got is out and torch.equal(out, want)


@pytest.mark.parametrize("dtype", list(DT))
def test_many_rows_and_a_long_prefix(dtype):
    rows, leads, shared = family(12, 40000, lambda n, h: 500 - n * 40, 2, 128)
    check(*build(rows, leads, 2, 6, 128, 128, DT[dtype], 8, shared))
    rows = [[(n * 131) % 90 + (64 if n % 3 else 0)] for n in range(1500)]
    leads = [n - n % 3 for n in range(1500)]
    rows = [[64 * 3 + (n * 131) % 90] for n in range(1500)]
    shared = [[3]] * 1500
    check(*build(rows, leads, 1, 8, 64, 64, DT[dtype], 8, shared))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D,G,ps,seed", [(64, 8, 32, 0), (128, 5, 64, 1), (128, 16, 16, 2), (64, 1, 128, 3)])
def test_pieces_of_every_kind_in_a_row(dtype, D, G, ps, seed):
    """Prefixes with fewer and more than 128 queries, own tokens of none, one and several tiles, one after the other in
    every block's range."""
    rng = torch.Generator().manual_seed(seed)
    rows, leads, shared = [], [], []
    while len(rows) < 260:
        first, members = len(rows), int(torch.randint(1, 40, (1,), generator=rng))
        prompt = int(torch.randint(1, 1200, (1,), generator=rng))
        for _ in range(members):
            own = int(torch.randint(0, 700, (1,), generator=rng)) if torch.rand(1, generator=rng) < 0.6 else 0
            rows.append([prompt + own])
            leads.append(first)
            shared.append([prompt // ps])
    check(*build(rows, leads, 1, G, D, ps, DT[dtype], seed, shared))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("members,G,ps", [(24, 8, 16), (70, 4, 64), (3, 5, 32)])
def test_members_that_share_less(dtype, members, G, ps):
    """Every member has its own length in common with the lead."""
    rng = torch.Generator().manual_seed(members)
    prompt = 6000
    pages = prompt // ps
    cut = [[int(torch.randint(0, pages + 1, (1,), generator=rng)), pages if n % 3 else n % 2 * pages // 2] for n in range(members)]
    rows = [[prompt + n * 7, prompt + n] for n in range(members)]
    check(*build(rows, [1] * members, 2, G, 64, ps, DT[dtype], members, cut))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_infinities_stay_with_their_owner(dtype):
    """An infinite value, or a key of -inf, in the tokens that one sequence has for itself."""
    rows, leads, shared = family(5, 600, lambda n, h: 50, 1, 64)
    shared[2] = [3]                                       # shares only the first 192 tokens
    q, cache, lead = build(rows, leads, 1, 4, 64, 64, DT[dtype], 6, shared)
    want = kvp.kvp_paged_prefix_decode_attn(q, cache, lead)
    cache.v_pool[cache.table[2, 7].long(), 5] = math.inf
    cache.k_pool[cache.table[4, 10].long(), 60:] = -math.inf   # (behind the end of the row, 650: no token)
    got = kvp.kvp_paged_prefix_decode_attn(q, cache, lead)
    for n in range(5):
        assert torch.equal(got[n], want[n]) == (n != 2)
    assert not torch.isfinite(got[2]).any()               # infinite, or NaN where a part of a weight is 0 or negative


def test_matches_paged_decode_in_a_run():
    """Prompt, fork, a few steps of norms, rotation, append and attention, an eviction of one sequence, a cut; and the
    same step captured once and replayed while the cache grows."""
    N, h_kv, G, D, ps = 6, 2, 4, 128, 32
    gen = torch.Generator("cuda").manual_seed(0)
    dt = torch.bfloat16
    R, heads = N * h_kv, h_kv * (G + 2)
    cache = kvp.PagedCache.empty(R, 40, 300, ps, D, dt)
    rope = kvp.Rope(D, theta=1e6)
    w = torch.rand(D, device="cuda", generator=gen) + 0.5
    counts = torch.zeros(R, dtype=torch.int32, device="cuda")
    counts[:h_kv] = 700
    prompt = torch.randn(N, 700, heads, D, device="cuda", generator=gen).to(dt).transpose(1, 2)
    q, k = kvp.kvp_qk_norm_rope(prompt[:, :h_kv * G], prompt[:, h_kv * G:h_kv * (G + 1)], w, w, rope=rope)
    kvp.kvp_paged_append(cache, k, prompt[:, h_kv * (G + 1):], counts=counts)
    src = torch.full((N, h_kv), -1, dtype=torch.int32, device="cuda")
    src[1:] = torch.arange(h_kv, device="cuda", dtype=torch.int32)
    kvp.kvp_paged_fork(cache, src.view(-1))
    lead = torch.zeros(N, dtype=torch.int32, device="cuda")
    qkv = torch.empty(N, 1, heads, D, dtype=dt, device="cuda")

    def step():
        x = qkv.transpose(1, 2)
        pos = cache.lens.view(N, h_kv)[:, :1].contiguous()
        q, k = kvp.kvp_qk_norm_rope(x[:, :h_kv * G], x[:, h_kv * G:h_kv * (G + 1)], w, w, rope=rope, positions=pos)
        kvp.kvp_paged_append(cache, k, x[:, h_kv * (G + 1):])
        return q[:, :, 0], kvp.kvp_paged_prefix_decode_attn(q[:, :, 0], cache, lead, return_lse=True)

    def compare(q, got):
        want, want_lse, tol, tol_lse = reference(q, cache)
        assert bool(((got[0].double() - want).abs() <= tol).all()) and bool(((got[1].double() - want_lse).abs() <= tol_lse).all())
        per_row, lse = kvp.kvp_paged_decode_attn(q, cache, return_lse=True)
        assert bool(((per_row.double() - got[0].double()).abs() <= 2 * tol).all())

    for _ in range(3):
        qkv.normal_(generator=gen)
        compare(*step())
    idx = torch.arange(0, 400, device="cuda", dtype=torch.int32).repeat(R, 1) + 7
    keep = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    keep[2 * h_kv:3 * h_kv] = 400                         # sequence 2 drops its first seven tokens and its last
    kvp.kvp_paged_compact(cache, idx, keep)
    cut = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    cut[4 * h_kv:5 * h_kv] = 100
    kvp.kvp_paged_free(cache, cut)
    compare(*step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, got = step()
    for _ in range(70):
        qkv.normal_(generator=gen)
        graph.replay()
    compare(q, got)
    cut.fill_(-1)
    cut[:h_kv] = 0                                        # the lead leaves: nobody shares with an empty row
    kvp.kvp_paged_free(cache, cut)
    qkv.normal_(generator=gen)
    graph.replay()
    compare(q, got)
    kvp.kvp_check_device_status()


def test_two_calls_at_once():
    rows, leads, shared = family(8, 3000, lambda n, h: n * 20, 2, 64)
    q, cache, lead = build(rows, leads, 2, 4, 128, 64, torch.bfloat16, 5, shared)
    want = kvp.kvp_paged_prefix_decode_attn(q, cache, lead)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            got.append(kvp.kvp_paged_prefix_decode_attn(q, cache, lead, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("dtype", list(DT))
def test_the_same_again(dtype):
    """Results to the last bit, whatever the calls between them leave behind."""
    rows, leads, shared = family(24, 900, lambda n, h: n * 37, 8, 64)
    q, cache, lead = build(rows, leads, 8, 4, 128, 64, DT[dtype], 6, shared)
    other, far = q.flip(0) * 30, torch.full_like(lead, -1)
    want = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True)
    alone = kvp.kvp_paged_prefix_decode_attn(q, cache, far, return_lse=True)
    for _ in range(20):
        kvp.kvp_paged_prefix_decode_attn(other, cache, far)
        got = kvp.kvp_paged_prefix_decode_attn(q, cache, lead, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        kvp.kvp_paged_prefix_decode_attn(other, cache, lead)
        got = kvp.kvp_paged_prefix_decode_attn(q, cache, far, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, alone))


def test_wrong_leads_cost_time_only():
    rows, leads, shared = family(4, 600, lambda n, h: 20 * n, 1, 64)
    q, cache, lead = build(rows, leads, 1, 4, 64, 64, torch.float16, 6, shared)
    for other in ([1, 2, 3, 0], [1, 1, 1, 1], [2, 0, 2, 0], [-5, 0, 1, 2], [3, 3, 3, 3]):
        lead.copy_(torch.tensor(other, dtype=torch.int32))
        check(q, cache, lead)
    lead.copy_(torch.tensor([0, 0, 4, 0], dtype=torch.int32))
    out = kvp.kvp_paged_prefix_decode_attn(q, cache, lead)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_check_device_status()
    want, _, tol, _ = reference(q, cache)
    assert bool(((out.double() - want).abs() <= tol).all())


def test_refusals():
    rows, leads, shared = family(4, 100, lambda n, h: 3, 1, 64)
    q, cache, lead = build(rows, leads, 1, 4, 64, 64, torch.float16, 6, shared)
    call = kvp.kvp_paged_prefix_decode_attn
    for error, f in [(TypeError, lambda: call(q, None, lead)), (TypeError, lambda: call(None, cache, lead)),
                     (TypeError, lambda: call(q, cache, [0] * 4)), (ValueError, lambda: call(q, cache, lead.long())),
                     (ValueError, lambda: call(q, cache, lead[:3])), (ValueError, lambda: call(q, cache, lead.cpu())),
                     (ValueError, lambda: call(q.float(), cache, lead)), (ValueError, lambda: call(q[:3], cache, lead[:3])),
                     (ValueError, lambda: call(q, cache, lead, out=torch.empty(4, 4, 64, device="cuda"))),
                     (ValueError, lambda: call(q, cache, lead, lse=torch.empty(4, 3, device="cuda"))),
                     (kvp.KvpError, lambda: call(q, cache, lead, sm_scale=math.inf)),
                     (kvp.KvpError, lambda: call(q, cache, lead, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))]:
        with pytest.raises(error):
            f()
    torch.cuda.synchronize()
