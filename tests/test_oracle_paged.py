"""Pins of the paged cache's oracle: books that always add up, rows that read back what was written,
attention that equals the dense oracle's, and hand-worked page choices."""
import numpy as np
import pytest

import oracle
from oracle import paged


def check_books(c):
    ps = c["k"].shape[1]
    held = np.zeros(c["refs"].shape[0], np.int64)
    for r, n in enumerate(c["lens"]):
        for j in range(-(-int(n) // ps)):
            held[c["table"][r, j]] += 1
    assert (held == c["refs"]).all()


def test_pages_are_taken_lowest_first():
    c = paged.empty_cache(3, 4, 8, 16, 4)
    new = np.arange(3 * 40 * 4).reshape(3, 40, 4).astype(np.int16)
    assert paged.append(c, new, new, [40, 16, 1]) == []
    assert c["table"][0, :3].tolist() == [0, 1, 2] and c["table"][1, 0] == 3 and c["table"][2, 0] == 4
    paged.free(c, [-1, 0, -1])
    assert c["refs"].tolist() == [1, 1, 1, 0, 1, 0, 0, 0]
    assert paged.free_mask(c).tolist() == [0b11101000]
    assert paged.append(c, new, new, [10, 0, 20]) == []       # row 0: one page (3); row 2: one page (5)
    assert c["table"][0, 3] == 3 and c["table"][2, 1] == 5
    check_books(c)


def test_rows_past_the_free_pages_are_left_alone():
    c = paged.empty_cache(3, 4, 3, 16, 4)
    new = np.ones((3, 33, 4), np.int16)
    assert paged.append(c, new, new, [16, 33, 1]) == [1, 2]   # 1 + 3 pages are more than 3
    assert c["lens"].tolist() == [16, 0, 0]
    check_books(c)


def test_shared_tail_is_copied_before_it_is_written():
    c = paged.empty_cache(2, 4, 6, 16, 2)
    new = np.arange(2 * 20 * 2).reshape(2, 20, 2).astype(np.int16)
    paged.append(c, new, new, [20, 0])
    paged.fork(c, [-1, 0])
    assert (c["table"][1, :2] == c["table"][0, :2]).all() and c["refs"][:2].tolist() == [2, 2]
    paged.append(c, new + 100, new + 100, [0, 1])
    assert c["table"][1, 0] == 0 and c["table"][1, 1] == 2 and c["refs"][:3].tolist() == [2, 1, 1]
    assert (paged.row_tokens(c, "k", 0) == new[0, :20]).all()
    assert (paged.row_tokens(c, "k", 1)[:20] == new[0, :20]).all()
    assert (paged.row_tokens(c, "k", 1)[20] == new[1, 0] + 100).all()
    check_books(c)


@pytest.mark.parametrize("seed", range(8))
def test_random_streams_against_plain_lists(seed):
    """Rows kept as plain lists of tokens beside the pages: append, fork, compact, free in any order."""
    rng = np.random.default_rng(seed)
    R, ps, mp = 5, 16, 6
    c = paged.empty_cache(R, mp, 24, ps, 2, scores=True, positions=True)
    rows = [[] for _ in range(R)]
    for step in range(40):
        op = rng.integers(4)
        if op == 0:
            new = rng.integers(-999, 999, (R, 30, 2)).astype(np.int16)
            cnt = [int(min(rng.integers(0, 31), mp * ps - len(rows[r]))) for r in range(R)]
            bad = paged.append(c, new, new + 1, cnt)
            for r in range(R):
                if r not in bad:
                    rows[r] += [new[r, i].tolist() for i in range(cnt[r])]
        elif op == 1:
            src = [-1] * R
            for r in range(R):
                s = int(rng.integers(R))
                if not rows[r] and s != r and src[s] < 0 and all(x != r for x in src):
                    src[r] = s
            bad = paged.fork(c, src, copy=bool(rng.integers(2)))
            for r in range(R):
                if src[r] >= 0 and r not in bad:
                    rows[r] = list(rows[src[r]])
        elif op == 2:
            kept = [sorted(rng.choice(len(x), int(rng.integers(0, len(x) + 1)), replace=False).tolist()) if x else []
                    for x in rows]
            cnt = [len(x) if rng.integers(4) else -1 for x in kept]
            idx = np.full((R, mp * ps), -1)
            for r in range(R):
                idx[r, :len(kept[r])] = kept[r]
            bad = paged.compact(c, idx, cnt)
            for r in range(R):
                if cnt[r] >= 0 and r not in bad:
                    rows[r] = [rows[r][j] for j in kept[r]]
        else:
            keep = [int(rng.integers(-1, len(x) + 1)) for x in rows]
            paged.free(c, keep)
            rows = [x if k < 0 else x[:k] for x, k in zip(rows, keep)]
        check_books(c)
        for r in range(R):
            assert c["lens"][r] == len(rows[r])
            assert paged.row_tokens(c, "k", r).tolist() == rows[r]
            assert paged.row_tokens(c, "v", r).tolist() == [[a + 1 for a in t] for t in rows[r]]


def test_decode_equals_the_dense_oracle():
    rng = np.random.default_rng(0)
    L, Hkv, G, D, T = 2, 2, 3, 8, 21
    k, v = rng.standard_normal((2, L * Hkv, T, D))
    q = rng.standard_normal((L, Hkv * G, D))
    lens = [21, 0, 5, 1]
    want, mass = oracle.decode_attn(q, k, v, lens, 0.3)
    out, lse, got, mag = paged.paged_decode_attn(q, [k[r, :n] for r, n in enumerate(lens)],
                                                 [v[r, :n] for r, n in enumerate(lens)], 0.3)
    assert np.abs(out - want).max() < 1e-13
    assert (mag >= np.abs(out) - 1e-15).all()
    for r, n in enumerate(lens):
        assert np.abs(mass[r, :n] - got[r]).max(initial=0) < 1e-14
    assert np.isneginf(lse[0, 3:]).all() and np.isfinite(lse[0, :3]).all()
    s = (k[0] @ q[0, 0]) * 0.3
    assert abs(lse[0, 0] - np.log(np.exp(s).sum())) < 1e-12
