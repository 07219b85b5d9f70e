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


def books_of(c):
    """Everything of a cache, the pools by their bits (slots that nobody has written may hold NaN)."""
    return [t.clone() for t in (c.table, c.lens, c.refs, c.free_mask, c.k_pool.view(torch.int16), c.v_pool.view(torch.int16),
                                c.score, c.pos)]


def grown(kvp, dtype, D, ps, lens, shared, spare, seed):  # noqa: F811
    """Rows of these lengths and as many after them, which share the pages of those that `shared` names."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, mp = len(lens), -(-max(lens) // ps) + 1
    c = kvp.PagedCache.empty(2 * R, mp, sum(-(-n // ps) for n in lens) + spare, ps, D, DT[dtype], scores=True, positions=True)
    new = torch.randn(2, 2 * R, max(lens), D, generator=gen, device="cuda").to(DT[dtype])
    kvp.kvp_paged_append(c, new[0], new[1], counts=i32(list(lens) + [0] * R))
    kvp.kvp_paged_fork(c, i32([-1] * R + [r if r in shared else -1 for r in range(R)]))
    c.score.copy_(torch.rand(c.score.shape, generator=gen, device="cuda"))
    kvp.kvp_check_device_status()
    return c


BAD = {"past the end": lambda x, n: x[:-1] + [n], "far past": lambda x, n: x[:-1] + [2 ** 31 - 1], "negative": lambda x, n: [-1] + x[1:],
       "lowest": lambda x, n: [-2 ** 31] + x[1:], "twice": lambda x, n: x[:-1] + [x[-2]], "twice, inside": lambda x, n: x[:7] + [x[6]] + x[8:],
       "swapped": lambda x, n: x[:5] + [x[6], x[5]] + x[7:], "swapped, across pages": lambda x, n: x[:31] + [x[32], x[31]] + x[33:],
       "descending": lambda x, n: x[::-1], "far inside": lambda x, n: x[:len(x) // 2] + [n + 3] + x[len(x) // 2 + 1:]}


@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("dtype,D,ps,R", [("f16", 128, 32, 5), ("f32", 64, 16, 3), ("bf16", 64, 32, 40)])
def test_rows_with_bad_indices_are_left_alone(kvp, what, dtype, D, ps, R):  # noqa: F811
    """Compaction: indices that are not ascending or not the row's raise the status, and the row keeps its tokens, pages,
    scores and positions; the other rows are compacted as the oracle does it, on the same pages as if that row had not been
    asked for."""
    lens = [700 + 37 * r for r in range(R)]
    c = grown(kvp, dtype, D, ps, lens, set(range(0, R, 2)), R * 30, seed=R)
    rng = np.random.default_rng(R)
    idx, cnt = np.full((2 * R, 650), -1, np.int64), np.full(2 * R, -1)
    wrong = {0, R - 1, R if R % 2 else 1}                       # the last of them is a fork of row 0, or private
    for r in range(2 * R):
        n = int(c.lens[r])
        if n:
            kept = np.sort(rng.choice(n, int(rng.integers(60, 600)), replace=False)).tolist()
            if r in wrong:
                kept = BAD[what](kept, n)
            idx[r, :len(kept)], cnt[r] = kept, len(kept)
    np_dt = np.int32 if dtype == "f32" else np.int16
    o = {"k": c.k_pool.cpu().view(torch.int32 if dtype == "f32" else torch.int16).numpy().astype(np_dt),
         "v": c.v_pool.cpu().view(torch.int32 if dtype == "f32" else torch.int16).numpy().astype(np_dt),
         "table": c.table.cpu().numpy().astype(np.int64), "lens": c.lens.cpu().numpy().astype(np.int64),
         "refs": c.refs.cpu().numpy().astype(np.int64), "score": c.score.cpu().double().numpy(),
         "pos": c.pos.cpu().numpy().astype(np.int64)}
    before = books_of(c)
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32(idx), i32(cnt)))
    assert paged.compact(o, idx, [-1 if r in wrong else int(cnt[r]) for r in range(2 * R)]) == []
    for r in wrong:
        assert torch.equal(c.table[r], before[0][r]) and int(c.lens[r]) == int(before[1][r])
        assert torch.equal(c.score[r], before[6][r]) and torch.equal(c.pos[r], before[7][r])
    assert c.lens.tolist() == o["lens"].tolist() and c.refs.tolist() == o["refs"].tolist()
    assert (c.table.cpu().numpy() == o["table"]).all() and (c.free_mask.cpu().numpy() == paged.free_mask(o)).all()
    bits = torch.int32 if dtype == "f32" else torch.int16
    for name, pool in (("k", c.k_pool), ("v", c.v_pool)):
        for r in range(2 * R):
            held = c.table[r, : -(-int(c.lens[r]) // ps)].long()
            n = int(c.lens[r])
            got = pool[held].cpu().view(bits).numpy().reshape(-1, D)[:n]
            assert (got == paged.row_tokens(o, name, r).reshape(-1, D)).all(), r
    for r in range(2 * R):
        n = int(c.lens[r])
        assert (c.pos[r, :n].cpu().numpy() == o["pos"][r, :n]).all()
        assert (c.score[r, :n].cpu().double().numpy() == o["score"][r, :n]).all()


@pytest.mark.parametrize("page", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("where", [0, 11, 20])
def test_rows_with_bad_pages_are_not_compacted(kvp, page, where):  # noqa: F811
    """A page id out of range, kept or not, leaves the row as it is."""
    c = grown(kvp, "f16", 64, 32, [700, 690], set(), 3, seed=1)
    good = int(c.table[0, where])
    c.table[0, where] = page
    before = books_of(c)
    idx = [list(range(1, 700, 3)), list(range(0, 690, 3))]
    raises_status(kvp, lambda: kvp.kvp_paged_compact(c, i32([x[:230] for x in idx] * 2), i32([230, -1, -1, -1])))
    for t, b in zip(books_of(c), before):
        assert torch.equal(t, b)
    c.table[0, where] = good
    kvp.kvp_paged_compact(c, i32([x[:230] for x in idx] * 2), i32([230, 230, -1, -1]))
    kvp.kvp_check_device_status()
    assert c.pos[0, :230].tolist() == idx[0][:230] and c.pos[1, :230].tolist() == idx[1][:230]


def test_a_selection_for_the_longest_row_does_not_cut_the_others(kvp):  # noqa: F811
    """kvp_select_topk keeps the newest of T tokens in every row: behind the end of a shorter one.  No token is lost."""
    lens = [700, 200, 690, 31]
    c = grown(kvp, "bf16", 128, 32, lens, set(), 3, seed=2)
    first = c.rows(0, 4)
    budgets = torch.full((4,), 150, dtype=torch.int32, device="cuda")
    idx, count = kvp.kvp_select_topk(first.score, budgets, 4, 16, 150, T=700)
    rows, table, score = rows_of(first), first.table.clone(), first.score.clone()
    raises_status(kvp, lambda: kvp.kvp_paged_compact(first, idx, count))
    assert first.lens.tolist() == [150, 200, 690, 31]
    for r in (1, 2, 3):
        assert torch.equal(first.table[r], table[r]) and torch.equal(first.score[r], score[r])
        assert all(torch.equal(x[r], y[r]) for x, y in zip(rows_of(first), rows))


def select_ragged(kvp, c, budgets, n_sink, n_recent, T):  # noqa: F811
    """Kept tokens of rows of any length: every row's first n_sink and newest n_recent, and the best of the rest."""
    col, n = torch.arange(T, device="cuda"), c.lens[:, None]
    score = torch.where((col < n_sink) | (col >= n - n_recent), float("inf"), c.score[:, :T])
    score = torch.where(col < n, score, float("nan"))           # NaN ranks last
    return kvp.kvp_select_topk(score, torch.minimum(budgets, c.lens), 0, 0, int(budgets.max()), T=T)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_a_ragged_cache_is_evicted_again_and_again(kvp, dtype):  # noqa: F811
    """Prefill of ragged prompts, decode steps with scores, evictions to head-wise budgets, a fork of every row in between."""
    import oracle
    D, ps, n_sink, n_recent, T = 64, 16, 4, 8, 448
    lens, budgets = [300, 20, 150, 4, 0, 256], [40, 64, 100, 12, 30, 200]
    R = len(lens)
    gen = torch.Generator(device="cuda").manual_seed(3)
    c = kvp.PagedCache.empty(2 * R, T // ps, 160, ps, D, DT[dtype], scores=True, positions=True)
    first = c.rows(0, R)
    new = torch.randn(2, R, 300, D, generator=gen, device="cuda").to(DT[dtype])
    kvp.kvp_paged_append(first, new[0], new[1], counts=i32(lens))
    seen = [[(j, new[0, r, j].cpu()) for j in range(n)] for r, n in enumerate(lens)]      # position, key
    at = i32(lens)
    for turn in range(4):
        for _ in range(3 + 20 * turn):
            step = torch.randn(2, R, 1, D, generator=gen, device="cuda").to(DT[dtype])
            kvp.kvp_paged_append(first, step[0], step[1], new_pos=at)
            for r in range(R):
                seen[r].append((int(at[r]), step[0, r, 0].cpu()))
            at += 1
            q = torch.randn(2, R, D, generator=gen, device="cuda").to(DT[dtype])
            kvp.kvp_paged_decode_attn(q, first, add_scores=True)
        kvp.kvp_check_device_status()
        score = first.score.cpu().numpy()
        idx, count = select_ragged(kvp, first, i32(budgets), n_sink, n_recent, T)
        if turn == 2:                                           # the pages of an evicted row may be somebody else's
            kvp.kvp_paged_fork(c, i32([-1] * R + list(range(R))))
            forked = [x[:R] for x in rows_of(first)]
        kvp.kvp_paged_compact(first, idx, count)
        kvp.kvp_check_device_status()
        kept = [oracle.select_row(score[r, :len(x)], budgets[r], n_sink, n_recent) for r, x in enumerate(seen)]
        seen = [[x[j] for j in k] for x, k in zip(seen, kept)]
        assert first.lens.tolist() == [len(x) for x in seen]
        rows = rows_of(first)[0]
        for r in range(R):
            assert first.pos[r, :len(seen[r])].tolist() == [p for p, _ in seen[r]], (turn, r)
            assert torch.equal(rows[r], torch.stack([k for _, k in seen[r]]))
        if turn == 2:
            back = rows_of(c.rows(R, 2 * R))
            assert all(torch.equal(a, b) for x, y in zip(back, forked) for a, b in zip(x, y))
            kvp.kvp_paged_free(c.rows(R, 2 * R))
    kvp.kvp_paged_free(c)
    assert int(c.refs.sum()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 8])
def test_a_scale_of_zero_gives_the_mean(kvp, dtype, G):  # noqa: F811
    """Dot products up to 2^126, of either sign, weigh the same: out is off by the sums of 40 values and a division, 2^-23
    each of the mean magnitude (and exp2(0) and the weights are exact)."""
    c = filled(kvp, [40, 3], 16, 64, dtype, seed=G)
    c.k_pool.copy_(torch.randn(c.k_pool.shape, generator=torch.Generator().manual_seed(1)) * 2.0 ** 120)
    q = torch.randn(1, 2 * G, 64, generator=torch.Generator().manual_seed(2)).to(DT[dtype]).cuda()
    out, lse = kvp.kvp_paged_decode_attn(q, c, sm_scale=0.0, return_lse=True)
    kvp.kvp_check_device_status()
    _, v = rows_of(c)
    for r, n in enumerate((40, 3)):
        got, want = out[0, r * G:(r + 1) * G].double().cpu(), v[r].double()
        assert ((got - want.mean(0)).abs() <= 44 * 2.0 ** -23 * want.abs().mean(0)).all()
        assert (lse[0, r * G:(r + 1) * G].double().cpu() - np.log(n)).abs().max() <= 2.0 ** -20
