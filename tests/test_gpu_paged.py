"""GPU parity of the paged cache: the books and the moved tokens are bit-exact against the oracle, decode
attention is within a bound made of its own roundings.

Decode's bound, per output, from the fp64 oracle's A = sum_t p_t |v_t| (each probability p_t is off by a
relative e at most, so the output by e * A):
* a logit is a sum of D fp32 products, each step off by at most 2^-23 (products of 16-bit values are exact;
  the tensor cores may truncate) of scale * sum_i |q_i k_i|, plus its scaling: d = (D + 4) 2^-23 * that sum;
  a softmax weight and the normaliser share it twice: 2 d;
* exp2 is off by 2^-22, the split of p into 16-bit parts by 2^-23 or less;
* every state sums n / 16 + 64 terms one after the other at most, in fp32: that many 2^-23, for the outputs and
  for the normaliser;
* the output's own rounding, half a step of its type.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import paged

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BITS = {torch.float32: torch.int32, torch.bfloat16: torch.int16, torch.float16: torch.int16}


@pytest.fixture(scope="module")
def kvp():
    import learned_kv_cache_gb300 as m
    m.load()
    return m


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def to_gpu(kvp, o, dtype, scores=True, positions=True):
    """The oracle's cache (its tokens' bits) on the GPU."""
    pools = [torch.from_numpy(o[x]).view(dtype).cuda() for x in ("k", "v")]
    return kvp.PagedCache(pools[0], pools[1], i32(o["table"]), i32(o["lens"]), i32(o["refs"]),
                          torch.from_numpy(paged.free_mask(o)).cuda(),
                          torch.from_numpy(o["score"]).float().cuda() if scores else None,
                          i32(o["pos"]) if positions else None)


def check_same(c, o, what=""):
    ps, R = c.page_size, c.n_rows
    torch.cuda.synchronize()
    assert c.lens.cpu().tolist() == o["lens"].tolist(), what
    assert c.refs.cpu().tolist() == o["refs"].tolist(), what
    assert c.free_mask.cpu().tolist() == paged.free_mask(o).tolist(), what
    assert (c.table.cpu().numpy() == o["table"]).all(), what
    for name, pool in (("k", c.k_pool), ("v", c.v_pool)):
        assert (pool.cpu().view(BITS[c.dtype]).numpy() == o[name]).all(), (what, name)
    if c.pos is not None:
        for r in range(R):
            n = int(o["lens"][r])
            assert (c.pos[r, :n].cpu().numpy() == o["pos"][r, :n]).all(), what
            assert (c.score[r, :n].cpu().numpy() == o["score"][r, :n].astype(np.float32)).all(), what


@pytest.mark.parametrize("dtype,D,ps,seed", [("bf16", 128, 16, 0), ("f16", 64, 32, 1), ("f32", 128, 16, 2),
                                             ("f32", 64, 64, 3), ("bf16", 64, 16, 4), ("f16", 128, 64, 5)])
def test_random_streams_match_the_oracle(kvp, dtype, D, ps, seed):
    """Append, fork (shared and copied), compact and free in any order, until pages run out and back: every
    table entry, count, bit, token, score and position equals the oracle's; rows that find no pages are left
    alone and raise the device status."""
    rng = np.random.default_rng(seed)
    R, mp = 7, 5
    n_pages = 37 if seed % 2 else 26
    np_dt = np.int32 if dtype == "f32" else np.int16
    o = paged.empty_cache(R, mp, n_pages, ps, D, np_dt, scores=True, positions=True)
    c = kvp.PagedCache.empty(R, mp, n_pages, ps, D, DT[dtype], scores=True, positions=True)
    for t in (c.k_pool, c.v_pool):
        t.view(BITS[c.dtype]).zero_()
    check_same(c, o, "empty")
    for step in range(60):
        op = ("append", "append", "fork", "compact", "free")[rng.integers(5)]
        if op == "append":
            n_new = int(rng.choice([1, 1, 5, 2 * ps + 3]))
            new = rng.integers(0, 1 << 14, (2, R, n_new, D)).astype(np_dt)
            cnt = [int(min(rng.integers(0, n_new + 1), mp * ps - o["lens"][r])) for r in range(R)]
            at = rng.integers(0, 1000, R) if step % 2 else None
            k, v = (torch.from_numpy(x).view(DT[dtype]).cuda() for x in new)
            bad = paged.append(o, new[0], new[1], cnt, at)
            kvp.kvp_paged_append(c, k, v, counts=i32(cnt), new_pos=None if at is None else i32(at))
        elif op == "fork":
            src = [-1] * R
            for r in range(R):
                s = int(rng.integers(R))
                if o["lens"][r] == 0 and s != r and src[s] < 0 and all(x != r for x in src):
                    src[r] = s
            copy = bool(rng.integers(2))
            bad = paged.fork(o, src, copy)
            kvp.kvp_paged_fork(c, i32(src), copy=copy)
        elif op == "compact":
            b_max = mp * ps if step % 2 else mp * ps + 9
            idx, cnt = np.full((R, b_max), -1), []
            for r in range(R):
                n = int(o["lens"][r])
                kept = sorted(rng.choice(n, int(rng.integers(0, n + 1)), replace=False).tolist()) if n else []
                if n and rng.integers(2):                       # a prefix that stays where it is
                    m = int(rng.integers(0, n + 1))
                    kept = sorted(set(range(m)) | {j for j in kept if j >= m})
                idx[r, :len(kept)] = kept
                cnt.append(len(kept) if rng.integers(4) else -1)
            bad = paged.compact(o, idx, cnt)
            kvp.kvp_paged_compact(c, i32(idx), i32(cnt))
        else:
            keep = [int(rng.integers(-1, n + 1)) for n in o["lens"]]
            bad = []
            paged.free(o, keep)
            kvp.kvp_paged_free(c, i32(keep))
        if bad:
            with pytest.raises(kvp.KvpError):
                kvp.kvp_check_device_status()
        else:
            kvp.kvp_check_device_status()
        # give the scores something to carry
        add = rng.integers(0, 9, o["score"].shape).astype(np.float64)
        o["score"] += add
        c.score += torch.from_numpy(add).float().cuda()
        check_same(c, o, f"step {step}: {op}")
    kvp.kvp_paged_free(c)
    paged.free(o)
    check_same(c, o, "freed")


def test_rows_that_find_no_pages_stay_as_they_were(kvp):
    """Append, copy and compact on a pool that runs out in the middle of the rows."""
    def pair():
        o = paged.empty_cache(6, 4, 8, 16, 64, np.int16, scores=True, positions=True)
        new = np.arange(2 * 6 * 40 * 64).reshape(2, 6, 40, 64).astype(np.int16) & 0x3fff
        assert paged.append(o, new[0], new[1], [40, 33, 0, 0, 0, 0]) == []
        assert paged.fork(o, [-1, -1, 0, -1, -1, -1]) == []
        return o, to_gpu(kvp, o, torch.float16), new

    def gpu(t):
        return torch.from_numpy(t).view(torch.float16).cuda()

    o, c, new = pair()                      # two pages are free
    assert paged.append(o, new[0], new[1], [1, 8, 1, 1, 17, 0]) == [3, 4]
    raises_status(kvp, lambda: kvp.kvp_paged_append(c, gpu(new[0]), gpu(new[1]), counts=i32([1, 8, 1, 1, 17, 0])))
    check_same(c, o, "append")
    o, c, new = pair()
    assert paged.fork(o, [-1, -1, -1, 1, -1, -1], True) == [3]
    raises_status(kvp, lambda: kvp.kvp_paged_fork(c, i32([-1, -1, -1, 1, -1, -1]), copy=True))
    check_same(c, o, "copy")
    o, c, new = pair()
    idx = np.tile(np.arange(1, 40), (6, 1))
    assert paged.compact(o, idx, [20, 10, 39, -1, 0, 0]) == [2]
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32(idx), i32([20, 10, 39, -1, 0, 0])))
    check_same(c, o, "compact")


def test_many_rows_and_pages(kvp):
    """More rows than the plan has threads, more pages than it looks at in one step: the i-th page that is
    needed is the i-th lowest free one."""
    R, ps, n_pages, D = 2600, 16, 150001, 64
    rng = np.random.default_rng(7)
    c = kvp.PagedCache.empty(R, 60, n_pages, ps, D, torch.float16)
    refs = torch.from_numpy((rng.random(n_pages) < 0.3).astype(np.int32))      # pages other rows hold
    refs[:131200] = 1
    refs[::5000] = 0
    c.refs.copy_(refs)
    c.free_mask.copy_(torch.from_numpy(paged.free_mask({"refs": refs.numpy()})))
    free = np.nonzero(refs.numpy() == 0)[0]
    lens = np.zeros(R, np.int64)
    table = np.full((R, 60), -1)
    at = 0
    for n_new in (40, 1, 33):
        cnt = rng.integers(0, n_new + 1, R)
        new = torch.randn(2, R, n_new, D, device="cuda").half()
        kvp.kvp_paged_append(c, new[0], new[1], counts=i32(cnt))
        kvp.kvp_check_device_status()
        for r in range(R):
            for j in range(-(-lens[r] // ps), -(-(lens[r] + cnt[r]) // ps)):
                table[r, j] = free[at]
                at += 1
        held = c.table.long()
        t = torch.from_numpy(lens).cuda()[:, None] + torch.arange(n_new, device="cuda")
        live = torch.arange(n_new, device="cuda") < i32(cnt)[:, None]
        page = held.gather(1, (t // ps).clamp(max=59))
        for pool, x in ((c.k_pool, new[0]), (c.v_pool, new[1])):
            assert torch.equal(pool[page.clamp(min=0), t % ps][live], x[live])
        lens += cnt
        assert (c.table.cpu().numpy() == table).all() and (c.lens.cpu().numpy() == lens).all()
    src = np.full(R, -1)
    kvp.kvp_paged_free(c, i32(np.where(np.arange(R) % 3, -1, 0)))
    src[::3] = np.arange(R)[1::3][:len(src[::3])]
    kvp.kvp_paged_fork(c, i32(src), copy=True)
    kvp.kvp_check_device_status()
    got, n = c.table.cpu().numpy(), lens.copy()
    n[::3] = lens[src[::3]]
    assert (c.lens.cpu().numpy() == n).all()
    rows = rows_of(c)
    for r in range(0, R, 3):
        assert torch.equal(rows[0][r], rows[0][src[r]]) and torch.equal(rows[1][r], rows[1][src[r]])
        assert not set(got[r, :-(-n[r] // ps)]) & set(got[src[r], :-(-n[r] // ps)])
    used = np.concatenate([got[r, :-(-n[r] // ps)] for r in range(R)])
    assert len(set(used)) == len(used)
    own = refs.numpy().copy()
    own[used] += 1
    assert (c.refs.cpu().numpy() == own).all()
    assert (c.free_mask.cpu().numpy() == paged.free_mask({"refs": own})).all()


@pytest.mark.parametrize("dtype,D,R", [("f16", 128, 5), ("f32", 128, 3), ("f32", 64, 40), ("bf16", 64, 9), ("f16", 128, 30), ("bf16", 128, 8)])
def test_compact_long_rows(kvp, dtype, D, R):
    """Rows of many chunks, kept in long runs, single tokens and none; half of them share pages with others."""
    rng = np.random.default_rng(D + R)
    ps, T = 32, 2500
    c = kvp.PagedCache.empty(2 * R, 81, R * 81 + 2 * R * 81, ps, D, DT[dtype], scores=True, positions=True)
    new = torch.randn(2, 2 * R, T, D, device="cuda").to(DT[dtype])
    kvp.kvp_paged_append(c, new[0], new[1], counts=i32([T - 7 * r for r in range(R)] + [0] * R))
    kvp.kvp_paged_fork(c, i32([-1] * R + [r if r % 2 else -1 for r in range(R)]))
    c.score.copy_(torch.rand(c.score.shape, device="cuda"))
    score, lens = c.score.clone(), c.lens.tolist()
    idx, cnt = np.full((2 * R, 2000), -1), []
    for r in range(2 * R):
        n = min(lens[r], 2000)
        share = (0.02, 0.5, 0.97, 1.0, 0.3)[r % 5]
        kept = np.nonzero(rng.random(lens[r]) < share)[0][:2000] if lens[r] else np.zeros(0, int)
        if r % 4 == 1:
            kept = np.concatenate([np.arange(n // 3), kept[kept >= n // 3]])[:2000]
        if r % 7 == 6:
            kept = kept[:0]
        idx[r, :len(kept)] = kept
        cnt.append(len(kept))
    kvp.kvp_paged_compact(c, i32(idx), i32(cnt))
    kvp.kvp_check_device_status()
    rows = rows_of(c)
    assert c.lens.tolist() == cnt
    held = torch.zeros(c.n_pages, dtype=torch.int64)
    for r in range(2 * R):
        kept = torch.from_numpy(idx[r, :cnt[r]])
        s = r if r < R else r - R
        assert torch.equal(rows[0][r], new[0, s].cpu()[kept]), r
        assert torch.equal(rows[1][r], new[1, s].cpu()[kept]), r
        assert torch.equal(c.score[r, :cnt[r]], score[r][kept.cuda()])
        if r < R:
            assert torch.equal(c.pos[r, :cnt[r]].cpu(), kept.int())
        pages = -(-cnt[r] // ps)
        held[c.table[r, :pages].cpu().long()] += 1
        assert (c.table[r, pages:] == -1).all()
    assert torch.equal(held.int(), c.refs.cpu())
    assert torch.equal(c.free_mask.cpu(), torch.from_numpy(paged.free_mask({"refs": held.numpy()})))


def filled(kvp, lens, ps, D, dtype, seed, spare=3, scores=False, stale=float("nan"), interleaved=False, key_scale=1.0):
    """A cache whose rows' pages lie in any order; slots behind the rows' ends hold ``stale``."""
    gen = torch.Generator().manual_seed(seed)
    lens = torch.as_tensor(lens)
    R = lens.numel()
    pages = (lens + ps - 1) // ps
    n_pages, mp = int(pages.sum()) + spare, int(pages.max()) + 2
    kv = torch.full((n_pages, 2, ps, D), stale, dtype=DT[dtype])
    table = torch.full((R, mp), -7, dtype=torch.int32)        # what stands behind a row's pages is not read
    place = torch.randperm(n_pages, generator=gen)
    at = 0
    for r in range(R):
        for j in range(int(pages[r])):
            p = int(place[at])
            at += 1
            table[r, j] = p
            n = min(ps, int(lens[r]) - j * ps)
            kv[p, 0, :n] = (torch.randn(n, D, generator=gen) * key_scale).to(DT[dtype])
            kv[p, 1, :n] = torch.randn(n, D, generator=gen).to(DT[dtype])
    refs = torch.zeros(n_pages, dtype=torch.int32)
    refs[place[:at]] = 1
    words = paged.free_mask({"refs": refs.numpy()})
    kv = kv.cuda()
    k, v = (kv[:, 0], kv[:, 1]) if interleaved else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
    score = torch.rand(R, mp * ps, generator=gen).cuda() if scores else None
    return kvp.PagedCache(k, v, table.cuda(), lens.to(torch.int32).cuda(), refs.cuda(), torch.from_numpy(words).cuda(),
                          score)


def rows_of(c):
    """Every row's K and V on the host, in order."""
    out = ([], [])
    table, k, v = c.table.cpu(), c.k_pool.cpu(), c.v_pool.cpu()
    for r, n in enumerate(c.lens.cpu().tolist()):
        held = table[r, : -(-n // c.page_size)].long()
        for x, pool in zip(out, (k, v)):
            x.append(pool[held].reshape(-1, c.head_dim)[:n])
    return out


def check_decode(kvp, c, q, out_dtype=None, sm_scale=None, **kw):
    D = c.head_dim
    scale = D ** -0.5 if sm_scale is None else sm_scale
    before = None if c.score is None else c.score.clone()
    out, lse = kvp.kvp_paged_decode_attn(q, c, sm_scale=sm_scale, out_dtype=out_dtype, return_lse=True,
                                         add_scores=c.score is not None, **kw)
    torch.cuda.synchronize()
    kvp.kvp_check_device_status()
    k, v = rows_of(c)
    ref, ref_lse, mass, mag = paged.paged_decode_attn(q, k, v, scale)
    L, Hq, _ = q.shape
    G = L * Hq // c.n_rows
    q64 = np.abs(q.double().cpu().numpy()).reshape(c.n_rows, G, D)
    eps = np.zeros((c.n_rows, G))
    logit = np.zeros((c.n_rows, G))
    for r in range(c.n_rows):
        n = k[r].shape[0]
        if n:
            d = (D + 4) * 2.0 ** -23 * scale * (np.abs(k[r].double().numpy()) @ q64[r].T).max(0)
            logit[r] = d
            eps[r] = 2 * d + 2.0 ** -21 + 2 * (n / 16 + 64) * 2.0 ** -23
    eps, logit = eps.reshape(L, Hq), logit.reshape(L, Hq)
    step = torch.finfo(out.dtype).eps / 2
    tol = eps[:, :, None] * mag * (1 + step) + step * np.abs(ref) + 1e-30
    if out.dtype == torch.float16:
        tol += 2.0 ** -25                                       # half a step of the subnormal range
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()
    got = lse.double().cpu().numpy()
    dead = np.isneginf(ref_lse)
    assert (np.isneginf(got) == dead).all()
    tol_l = eps + logit + 2.0 ** -22 * (np.abs(np.where(dead, 0, ref_lse)) + 1)
    assert (np.abs(np.where(dead, 0, got) - np.where(dead, 0, ref_lse)) <= tol_l).all()
    if before is not None:
        got, b = c.score.double().cpu().numpy(), before.double().cpu().numpy()
        for r, m in enumerate(mass):
            n = m.size
            e = (eps.reshape(c.n_rows, G) + logit.reshape(c.n_rows, G)).max(1)[r] + 2.0 ** -20
            assert (np.abs(got[r, :n] - b[r, :n] - m) <= e * m + 2.0 ** -23 * (b[r, :n] + m)).all(), r
            assert (got[r, n:] == b[r, n:]).all(), r            # slots behind the row stay
    return out, lse


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1, 0, 0, 700, 2]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,G,ps", [(128, 1, 16), (128, 4, 64), (64, 2, 32), (128, 6, 128), (64, 8, 16), (128, 5, 32),
                                    (128, 12, 64), (64, 16, 256), (128, 16, 16), (64, 9, 64), (128, 3, 1024)])
def test_decode_shapes(kvp, dtype, D, G, ps):
    """Lengths at every edge of a warp's keys, a tile and a page; empty rows; NaN behind the rows' ends."""
    c = filled(kvp, EDGES, ps, D, dtype, seed=D + G + ps, scores=G % 2 == 0)
    gen = torch.Generator().manual_seed(G)
    q = torch.randn(len(EDGES) // 2, 2 * G, D, generator=gen).to(DT[dtype]).cuda()
    check_decode(kvp, c, q)
    if dtype != "f32":
        check_decode(kvp, c, q, out_dtype=DT[dtype])


@pytest.mark.parametrize("dtype,lens", [
    ("bf16", [20000]),                                   # one row over many CTAs
    ("f16", [0, 0, 0, 5003, 0, 9001, 64, 0]),            # a few long rows between empty ones
    ("bf16", [7] * 999 + [3000]),                        # more rows than threads and CTAs
    ("f32", [6007, 1, 300, 0]),
    ("f32", [30000]),
    ("f32", [3] * 700 + [900]),
    ("f16", [0] * 40),                                   # nothing at all
    ("bf16", [64 * 4 * 304 // 8] * 8),                   # CTA borders on row borders
])
def test_decode_splits(kvp, dtype, lens):
    c = filled(kvp, lens, 64, 128, dtype, seed=len(lens), scores=True)
    G = 4
    q = torch.randn(1, len(lens) * G, 128, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    check_decode(kvp, c, q)
    check_decode(kvp, c, q, sm_scale=0.31)


def capped(c, pages):
    """The same rows with a table cut to `pages` columns."""
    t = c.table[:, :pages].contiguous()
    score = None if c.score is None else c.score[:, :pages * c.page_size].contiguous()
    return type(c)(c.k_pool, c.v_pool, t, c.lens, c.refs, c.free_mask, score, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,G,lens", [
    (128, 1, [20000]), (64, 4, [5003, 0, 9001, 64]), (128, 16, [700, 129]), (64, 16, [4100]),
    (128, 5, [0, 0, 33000, 1, 0, 65]), (128, 8, [1500 + 64 * i for i in range(18)]), (64, 3, [900 + i for i in range(19)]),
])
def test_decode_of_few_rows(kvp, dtype, D, G, lens):
    """Rows that many CTAs share, without scores: from one part to as many as there are CTAs."""
    c = filled(kvp, lens, 64, D, dtype, seed=len(lens) + G)
    q = torch.randn(1, len(lens) * G, D, generator=torch.Generator().manual_seed(G)).to(DT[dtype]).cuda()
    check_decode(kvp, c, q)
    if dtype != "f32":
        check_decode(kvp, c, q, out_dtype=DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,G,ps,cap,R", [(128, 6, 64, 192, 1), (64, 2, 16, 192, 56), (128, 1, 64, 576, 303), (128, 4, 32, 192, 304),
                                          (64, 16, 64, 576, 305), (128, 8, 16, 80, 1216), (64, 1, 64, 64, 1217),
                                          (128, 12, 128, 512, 700)])
def test_decode_of_short_rows(kvp, dtype, D, G, ps, cap, R):
    """Tables so narrow that rows are not cut (and, of fp32, some that are): one row or several per CTA,
    empty rows first, last and in runs, full ones."""
    gen = torch.Generator().manual_seed(R)
    lens = torch.randint(0, cap + 1, (R,), generator=gen)
    lens[torch.rand(R, generator=gen) < 0.3] = 0
    lens[R // 3:R // 3 + 9] = 0
    lens[R // 2], lens[-1] = cap, 0 if R > 1 else cap
    q = torch.randn(1, R * G, D, generator=gen).to(DT[dtype]).cuda()
    for scores in (False, True):
        check_decode(kvp, capped(filled(kvp, lens.tolist(), ps, D, dtype, seed=R, scores=scores), cap // ps), q)


def test_decode_extreme_values(kvp):
    """One-hot softmax at large logits, equal keys (the mean of the values), stale infinities."""
    c = filled(kvp, [200, 90, 64, 1], 32, 128, "bf16", seed=3, stale=float("inf"), key_scale=30.0)
    q = torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    check_decode(kvp, c, q, sm_scale=1.0)
    c.k_pool.copy_(c.k_pool[:1, :1].nan_to_num(0, 0, 0).expand_as(c.k_pool))
    out, _ = check_decode(kvp, c, q)
    v = rows_of(c)[1]
    assert torch.allclose(out[0, 0].cpu().double(), v[0].double().mean(0), atol=1e-4)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_decode_nan_and_inf_in_live_tokens(kvp, dtype):
    """A NaN key makes its row NaN and no other; keys of -inf weigh nothing; a row of them alone gives 0."""
    c = filled(kvp, [100, 100, 70, 3], 16, 64, dtype, seed=5, scores=True)
    q = torch.ones(1, 4, 64, dtype=DT[dtype], device="cuda")
    t = c.table.cpu()
    c.k_pool[t[0, 2], 5] = float("nan")
    c.k_pool[t[1, 0], 3] = float("-inf")
    for j in range(3):
        c.k_pool[t[3, 0], j] = float("-inf")
    out, lse = kvp.kvp_paged_decode_attn(q, c, return_lse=True, add_scores=True)
    out = out.cpu()
    assert out[0, 0].isnan().all() and lse[0, 0].isnan()
    assert out[0, 1:].isfinite().all() and lse[0, 1:3].isfinite().all()
    assert (out[0, 3] == 0).all() and lse[0, 3] == float("-inf")
    k, v = rows_of(c)
    p = torch.softmax(k[1].double().sum(1) / 8, 0)
    assert (out[0, 1].double() - p @ v[1].double()).abs().max() < 1e-4
    assert c.score[1:].isfinite().all()


def test_strided_pools_and_queries(kvp):
    """K and V interleaved in one buffer; queries and new tokens read out of a fused QKV projection."""
    D, Hq, Hkv, B, ps = 128, 8, 2, 3, 32
    c = filled(kvp, [40, 0, 33, 64, 5, 90], ps, D, "bf16", seed=8, interleaved=True)
    assert not c.k_pool.is_contiguous()
    qkv = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    q = qkv[:, :Hq]
    check_decode(kvp, c, q)
    n = c.lens.cpu()
    held = [x.clone() for x in rows_of(c)[0]]
    kvp.kvp_paged_append(c, qkv[:, Hq:Hq + Hkv, None], qkv[:, Hq + Hkv:, None])
    kvp.kvp_check_device_status()
    assert (c.lens.cpu() == n + 1).all()
    rows = rows_of(c)
    for r in range(B * Hkv):
        assert torch.equal(rows[0][r][:-1], held[r]) and torch.equal(rows[0][r][-1], qkv[r // Hkv, Hq + r % Hkv].cpu())
        assert torch.equal(rows[1][r][-1], qkv[r // Hkv, Hq + Hkv + r % Hkv].cpu())
    check_decode(kvp, c, q)


@pytest.mark.parametrize("dtype,D,R,n_new,ps", [("f16", 128, 512, 1, 16), ("f32", 64, 200, 5, 16), ("bf16", 64, 1, 60, 32),
                                                ("f32", 128, 300, 2, 64), ("bf16", 128, 513, 1, 16)])
def test_appends_of_a_step(kvp, dtype, D, R, n_new, ps):
    """Small appends (one launch, no workspace) and the first that are not: pages from all over the mask, every
    second row with a tail that it shares."""
    rng = np.random.default_rng(R)
    np_dt = np.int32 if dtype == "f32" else np.int16
    n_pages = 70000
    o = paged.empty_cache(2 * R, 6, n_pages, ps, D, np_dt, scores=True, positions=True) if R < 300 else None
    if o is None:
        R //= 2
        o = paged.empty_cache(2 * R, 6, n_pages, ps, D, np_dt, scores=True, positions=True)
    c = to_gpu(kvp, o, DT[dtype])
    first = rng.integers(0, 1 << 14, (2, 2 * R, 40, D)).astype(np_dt)
    cnt = [int(x) if r < R else 0 for r, x in enumerate(rng.integers(0, 41, 2 * R))]
    paged.append(o, first[0], first[1], cnt)
    kvp.kvp_paged_append(c, *(torch.from_numpy(x).view(DT[dtype]).cuda() for x in first), counts=i32(cnt))
    src = [-1] * R + [r if r % 2 else -1 for r in range(R)]
    paged.fork(o, src)
    kvp.kvp_paged_fork(c, i32(src))
    for step in range(3):
        new = rng.integers(0, 1 << 14, (2, 2 * R, n_new, D)).astype(np_dt)
        cnt = rng.integers(0, min(n_new, 6 * ps // 4) + 1, 2 * R)
        cnt = np.minimum(cnt, 6 * ps - o["lens"])
        assert paged.append(o, new[0], new[1], cnt) == []
        kvp.kvp_paged_append(c, *(torch.from_numpy(x).view(DT[dtype]).cuda() for x in new), counts=i32(cnt))
        kvp.kvp_check_device_status()
        torch.cuda.synchronize()
        assert c.lens.tolist() == o["lens"].tolist() and c.refs.tolist() == o["refs"].tolist()
        assert (c.table.cpu().numpy() == o["table"]).all()
        assert (c.free_mask.cpu().numpy() == paged.free_mask(o)).all()
        used = np.nonzero(o["refs"])[0]
        for name, pool in (("k", c.k_pool), ("v", c.v_pool)):
            got = pool[torch.from_numpy(used).cuda()].cpu().view(BITS[c.dtype]).numpy()
            assert (got == o[name][used]).all()
        for r in range(2 * R):
            n = int(o["lens"][r])
            assert (c.pos[r, :n].cpu().numpy() == o["pos"][r, :n]).all()


def test_layers_share_one_pool(kvp):
    """rows(): the calls on one layer's rows leave the other layers' alone."""
    c = kvp.PagedCache.empty(12, 4, 40, 16, 64, torch.float16)
    new = torch.randn(2, 4, 20, 64, device="cuda").half()
    for layer in (1, 0, 2):
        kvp.kvp_paged_append(c.rows(4 * layer, 4 * layer + 4), new[0] + layer, new[1] + layer)
    kvp.kvp_check_device_status()
    assert c.lens.tolist() == [20] * 12
    assert c.table[4:8, :2].flatten().tolist() == list(range(8))
    assert torch.equal(torch.stack(rows_of(c)[0]), torch.cat([new[0] + i for i in range(3)]).cpu())
    kvp.kvp_paged_free(c.rows(4, 8))
    assert c.lens.tolist() == [20] * 4 + [0] * 4 + [20] * 4 and int(c.refs.sum()) == 16


def test_prune_and_decode_on_pages(kvp):
    """Prefill, decode with accumulated scores, eviction to head-wise budgets, a fork, more decode steps: the
    pages' path against the dense calls on the same tokens, and against the oracle."""
    L, Hkv, G, D, ps, T = 3, 2, 3, 128, 32, 300
    R, Hq = L * Hkv, Hkv * G
    gen = torch.Generator(device="cuda").manual_seed(4)
    k, v = torch.randn(2, R, T, D, generator=gen, device="cuda").to(torch.float16)
    q = torch.randn(5, L, Hq, D, generator=gen, device="cuda").to(torch.float16)
    c = kvp.PagedCache.empty(2 * R, 12, 160, ps, D, torch.float16, scores=True, positions=True)
    first = c.rows(0, R)
    kvp.kvp_paged_append(first, k, v)
    for i in range(2):
        kvp.kvp_paged_decode_attn(q[i], first, add_scores=True)
    mass = torch.zeros(R, T, device="cuda")
    full = torch.full((R,), T, dtype=torch.int32, device="cuda")
    for i in range(2):
        kvp.kvp_decode_attn(q[i], k, v, full, key_mass=mass, accumulate=True)
    assert (c.score[:R, :T] - mass).abs().max() < 2e-3
    budgets = torch.tensor([40, 64, 100, 33, 300, 250], dtype=torch.int32, device="cuda")
    idx, count = kvp.kvp_select_topk(c.score[:R], budgets, 4, 16, 300, T=T)
    kvp.kvp_paged_compact(first, idx, count)
    kvp.kvp_check_device_status()
    kc, vc = kvp.kvp_compact_kv(k, v, idx, count)
    assert int((c.refs > 0).sum()) == sum(-(-int(n) // ps) for n in count.tolist())
    for r in range(R):
        n = int(count[r])
        assert torch.equal(c.pos[r, :n], idx[r, :n])
        assert torch.equal(rows_of(c)[0][r], kc[r, :n].cpu()) and torch.equal(rows_of(c)[1][r], vc[r, :n].cpu())
    src = torch.tensor([-1] * R + list(range(R)), dtype=torch.int32, device="cuda")
    kvp.kvp_paged_fork(c, src)
    new = torch.randn(2, 2 * R, 1, D, generator=gen, device="cuda").to(torch.float16)
    at = torch.full((2 * R,), T, dtype=torch.int32, device="cuda")
    kvp.kvp_paged_append(c, new[0], new[1], new_pos=at)
    kvp.kvp_check_device_status()
    q2 = torch.cat([q[2], q[3]])
    check_decode(kvp, c, q2)
    dense = kvp.kvp_decode_attn(q[2], torch.cat([kc, kc[:, :1]], 1).scatter(1, count.long()[:, None, None].expand(-1, 1, D), new[0][:R]),
                                torch.cat([vc, vc[:, :1]], 1).scatter(1, count.long()[:, None, None].expand(-1, 1, D), new[1][:R]),
                                count + 1)
    paged_out = kvp.kvp_paged_decode_attn(q2, c)
    assert (paged_out[:L] - dense).abs().max() < 2e-3
    assert torch.equal(c.pos[torch.arange(2 * R), (c.lens - 1).long()], at)
    kvp.kvp_paged_free(c)
    assert int(c.refs.sum()) == 0 and c.lens.tolist() == [0] * (2 * R)


def test_a_captured_step_serves_a_growing_cache(kvp):
    """One captured append + decode, replayed while the rows grow over page and tile borders."""
    R, G, D, ps = 4, 4, 64, 16
    c = kvp.PagedCache.empty(R, 20, 90, ps, D, torch.bfloat16, scores=True)
    new = torch.zeros(2, R, 1, D, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(2, 2 * G, D, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros(2, 2 * G, D, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kvp.kvp_paged_append(c, new[0], new[1])
        kvp.kvp_paged_decode_attn(q, c, out=out, add_scores=True)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvp.kvp_paged_append(c, new[0], new[1])
        kvp.kvp_paged_decode_attn(q, c, out=out, add_scores=True)
    kvp.kvp_paged_free(c)
    c.score.zero_()
    for step in range(200):
        new.normal_()
        q.normal_()
        g.replay()
        if step % 23 == 0 or step == 199:
            torch.cuda.synchronize()
            kvp.kvp_check_device_status()
            assert c.lens.tolist() == [step + 1] * R
            ref = paged.paged_decode_attn(q, *rows_of(c), D ** -0.5)[0]
            assert np.abs(out.double().cpu().numpy() - ref).max() < 2e-3
    assert abs(float(c.score.double().sum()) - 200 * R * G) < 1e-2


def test_two_decodes_at_once(kvp):
    """Calls on two streams have workspaces of their own; a stream given by the caller is used throughout."""
    c = filled(kvp, [9000, 70, 4000, 1], 64, 128, "bf16", seed=11)
    qs = [torch.randn(1, 16, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [kvp.kvp_paged_decode_attn(q, c) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i in range(2):
            got[i].append(kvp.kvp_paged_decode_attn(qs[i], c, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_results_do_not_depend_on_what_ran_before(kvp):
    c = filled(kvp, [3000, 17, 640, 5000], 32, 128, "f16", seed=12)
    q = torch.randn(2, 8, 128, device="cuda").half()
    ws = torch.full((1 << 24,), 0xAB, dtype=torch.uint8, device="cuda")
    a = kvp.kvp_paged_decode_attn(q, c, workspace=ws)
    b = kvp.kvp_paged_decode_attn(q, c, workspace=ws.fill_(0xFF))
    assert torch.equal(a, b)


def raises_status(kvp, fn):
    fn()
    with pytest.raises(kvp.KvpError):
        kvp.kvp_check_device_status()
    kvp.kvp_check_device_status()                               # read once


def test_what_only_the_device_sees(kvp):
    """Lengths, pages, counts and indices out of range raise the status and touch nothing they should not."""
    c = filled(kvp, [40, 40, 20, 0], 16, 64, "bf16", seed=13, spare=8)
    q = torch.randn(1, 8, 64, device="cuda").to(torch.bfloat16)
    books = [t.clone() for t in (c.table, c.lens, c.refs, c.free_mask)]

    def reset():
        for t, b in zip((c.table, c.lens, c.refs, c.free_mask), books):
            t.copy_(b)

    c.lens[1] = 10 ** 6
    raises_status(kvp, lambda: kvp.kvp_paged_free(c, i32([-1, 0, -1, -1])))
    raises_status(kvp, lambda: kvp.kvp_paged_append(c, q.view(4, 2, 64)[:, :1].contiguous(), q.view(4, 2, 64)[:, :1].contiguous()))
    assert c.lens.tolist() == [41, 10 ** 6, 21, 1]
    reset()
    for page in (-5, c.n_pages, 2 ** 31 - 1):
        c.table[1, 1] = page
        raises_status(kvp, lambda: kvp.kvp_paged_decode_attn(q, c))
        raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32([[0, 17]] * 4), i32([-1, 2, -1, -1])))
        reset()
    c.lens[2] = -3
    raises_status(kvp, lambda: kvp.kvp_paged_decode_attn(q, c))
    reset()
    z = torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda")
    raises_status(kvp, lambda: kvp.kvp_paged_append(c, z, z, counts=i32([0, 4, -1, 0])))
    raises_status(kvp, lambda: kvp.kvp_paged_free(c, i32([41, -1, -1, -1])))
    for src in ([-1, 0, -1, -1], [-1, -1, -1, 3], [-1, -1, -1, 4], [3, -1, -1, 0]):
        raises_status(kvp, lambda: kvp.kvp_paged_fork(c, i32(src)))
        raises_status(kvp, lambda: kvp.kvp_paged_fork(c, i32(src), copy=True))
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32([[0]] * 4), i32([2, -1, -1, -1])))
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32([[0, 1]] * 4), i32([-1, -1, -1, 1])))
    for t, b in zip((c.table, c.lens, c.refs, c.free_mask), books):
        assert torch.equal(t, b)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
def test_pages_out_of_range_spoil_their_row_only(kvp, dtype, G):
    c = filled(kvp, [400, 700, 90, 33], 16, 128, dtype, seed=G, spare=3)
    q = torch.randn(1, 4 * G, 128, generator=torch.Generator().manual_seed(G)).to(DT[dtype]).cuda()
    out = kvp.kvp_paged_decode_attn(q, c)
    for page in (-1, c.n_pages, -2 ** 31, 2 ** 31 - 1):
        c.table[1, 17] = page
        got = []
        raises_status(kvp, lambda: got.append(kvp.kvp_paged_decode_attn(q, c)))
        keep = [h for h in range(4 * G) if h // G != 1]
        assert torch.equal(got[0][0, keep], out[0, keep]) and got[0].isfinite().all()


def test_bits_behind_the_last_page_are_no_pages(kvp):
    c = kvp.PagedCache.empty(1, 3, 2, 16, 64, torch.float16)
    c.free_mask.fill_(-1)
    z = torch.ones(1, 40, 64, device="cuda").half()
    raises_status(kvp, lambda: kvp.kvp_paged_append(c, z, z))                # three pages of two
    kvp.kvp_paged_append(c, z[:, :32], z[:, :32])
    kvp.kvp_check_device_status()
    assert c.lens.tolist() == [32] and c.table[0, :2].tolist() == [0, 1]


def test_unordered_indices_do_not_reach_shared_pages(kvp):
    """Indices that are not ascending raise the status; another row on the same pages keeps its tokens."""
    c = kvp.PagedCache.empty(2, 4, 12, 16, 64, torch.float16)
    new = torch.randn(2, 2, 40, 64, device="cuda").half()
    kvp.kvp_paged_append(c, new[0], new[1], counts=i32([40, 0]))
    kvp.kvp_paged_fork(c, i32([-1, 0]))
    idx = list(range(16))
    idx[3], idx[4] = 9, 9
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32([idx, idx]), i32([-1, 16])))
    assert torch.equal(rows_of(c)[0][0], new[0, 0].cpu()) and torch.equal(rows_of(c)[1][0], new[1, 0].cpu())


def test_python_refusals(kvp):
    c = kvp.PagedCache.empty(4, 3, 9, 16, 64, torch.float16)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.float16)
    for bad in (q.float(), q[:, :, :32], q.cpu(), q[0], q.expand(2, 4, 64).transpose(0, 1), q[:1].expand(2, 4, 64),
                torch.zeros(3, 4, 64, device="cuda", dtype=torch.float16), q[:0]):
        with pytest.raises((ValueError, TypeError)):
            kvp.kvp_paged_decode_attn(bad, c)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_paged_decode_attn(q, c, add_scores=True)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_paged_decode_attn(q, c, out_dtype=torch.bfloat16)
    z = torch.zeros(4, 2, 64, device="cuda", dtype=torch.float16)
    for bad in (z.float(), z[:3], z.cpu(), z[..., :32], z.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            kvp.kvp_paged_append(c, bad, z)
        with pytest.raises((ValueError, TypeError)):
            kvp.kvp_paged_append(c, z, bad)
    with pytest.raises(ValueError):
        kvp.kvp_paged_append(c, z, z, counts=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        kvp.kvp_paged_fork(c, i32([0]))
    with pytest.raises(ValueError):
        kvp.kvp_paged_compact(c, i32([0, 1, 2, 3]), i32([1, 1, 1, 1]))
    with pytest.raises(ValueError):
        kvp.kvp_paged_free(c, i32([1]))
    with pytest.raises(ValueError):
        c.rows(2, 2)
    with pytest.raises(ValueError):
        kvp.PagedCache(c.k_pool, c.v_pool.float(), c.table, c.lens, c.refs, c.free_mask)
    with pytest.raises(ValueError):
        kvp.PagedCache(c.k_pool, c.v_pool, c.table, c.lens, c.refs, c.free_mask[:0])
    with pytest.raises(TypeError):
        kvp.kvp_paged_init(None)


def test_offsets_past_32_bits(kvp):
    """Pools of more than 2^31 elements and per-slot arrays of more than 2^31 entries, used at their far ends."""
    D, ps, n_pages = 128, 128, 140000                           # 2.3e9 elements a pool
    c = kvp.PagedCache.empty(8, 6, n_pages, ps, D, torch.float16)
    refs = np.ones(n_pages, np.int32)
    refs[-40:] = 0
    c.refs.copy_(torch.from_numpy(refs))
    words = np.zeros((n_pages + 31) // 32, np.uint32)
    for p in range(n_pages - 40, n_pages):
        words[p // 32] |= np.uint32(1 << (p % 32))
    c.free_mask.copy_(torch.from_numpy(words.view(np.int32)))
    new = torch.randn(2, 8, 600, D, device="cuda").half()
    lens = [600, 300, 1, 129, 0, 0, 0, 0]
    kvp.kvp_paged_append(c, new[0], new[1], counts=i32(lens))
    kvp.kvp_paged_fork(c, i32([-1, -1, -1, -1, 0, -1, -1, -1]), copy=True)
    kvp.kvp_paged_fork(c, i32([-1, -1, -1, -1, -1, 1, -1, -1]))
    idx = np.tile(np.arange(0, 1200, 2), (8, 1))
    kvp.kvp_paged_compact(c, i32(idx), i32([-1, 150, -1, -1, 300, -1, -1, -1]))
    kvp.kvp_check_device_status()
    assert int(c.table[0, 0]) == n_pages - 40
    rows = rows_of(c)
    for x in range(2):
        assert torch.equal(rows[x][0], new[x, 0].cpu()) and torch.equal(rows[x][5], new[x, 1, :300].cpu())
        assert torch.equal(rows[x][1], new[x, 1, :300:2].cpu()) and torch.equal(rows[x][4], new[x, 0, ::2].cpu())
    check_decode(kvp, c, torch.randn(2, 16, D, device="cuda").half())
    del c, new

    c = kvp.PagedCache.empty(3, 1 << 20, 64, 1024, 64, torch.bfloat16, positions=True)   # 3 * 2^30 slots
    new = torch.randn(3, 1500, 64, device="cuda").to(torch.bfloat16)
    kvp.kvp_paged_append(c, new, new, counts=i32([1500, 0, 1500]), new_pos=i32([7, 0, 10 ** 6]))
    kvp.kvp_paged_compact(c, i32(np.tile(np.arange(500, 1500), (3, 1))), i32([-1, -1, 1000]))
    kvp.kvp_paged_fork(c, i32([-1, 2, -1]))
    kvp.kvp_check_device_status()
    assert c.pos[0, :1500].tolist() == list(range(7, 1507))
    for r in (1, 2):
        assert c.pos[r, :1000].tolist() == list(range(10 ** 6 + 500, 10 ** 6 + 1500))
        assert torch.equal(rows_of(c)[0][r], new[2, 500:].cpu())
    check_decode(kvp, c, torch.randn(1, 3, 64, device="cuda").to(torch.bfloat16))


def test_captured_evictions(kvp):
    """Two graphs on one cache (append + decode, compact + free), each with its own temporaries, replayed in turn."""
    R, D, ps, cap = 4, 64, 16, 64
    c = kvp.PagedCache.empty(R, 8, 40, ps, D, torch.float16, scores=True, positions=True)
    new = torch.zeros(2, R, 1, D, device="cuda").half()
    q = torch.zeros(2, 4, D, device="cuda").half()
    at = torch.zeros(R, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 4, D, device="cuda")
    budgets = torch.full((R,), 40, dtype=torch.int32, device="cuda")

    def step():
        kvp.kvp_paged_append(c, new[0], new[1], new_pos=at)
        kvp.kvp_paged_decode_attn(q, c, out=out, add_scores=True)

    def evict():
        idx, count = kvp.kvp_select_topk(c.score, budgets, 2, 8, 40, T=cap)
        kvp.kvp_paged_compact(c, idx, count)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(cap):
            step()
        evict()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    kvp.kvp_check_device_status()
    graphs = []
    for fn in (step, evict):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        graphs.append(g)
    kvp.kvp_paged_free(c)
    c.score.zero_()
    seen = [[] for _ in range(R)]                               # (position, key) of the tokens a row holds
    for t in range(200):
        new.normal_()
        q.normal_()
        at.fill_(t)
        graphs[0].replay()
        for r in range(R):
            seen[r].append((t, new[0, r, 0].cpu()))
        if len(seen[0]) == cap:
            torch.cuda.synchronize()
            kept, _ = oracle.select_topk(c.score[:, :cap].cpu().numpy(), [40] * R, 2, 8, b_max=40)
            graphs[1].replay()
            seen = [[x[j] for j in kept[r]] for r, x in enumerate(seen)]
            torch.cuda.synchronize()
            kvp.kvp_check_device_status()
            for r in range(R):
                assert c.pos[r, :40].tolist() == [p for p, _ in seen[r]]
                assert torch.equal(rows_of(c)[0][r], torch.stack([k for _, k in seen[r]]))
            assert int(c.refs.sum()) == R * 3
    assert c.lens.tolist() == [len(seen[0])] * R
