"""Plain oracle of the paged cache: one Python loop per token and page.

LKV, "LKV-H" (every KV head keeps its own budget) and How much KV cache can you prune,
"Conclusion" (copying the kept entries into a new tensor does not free the old one): a row's
tokens stand in pages of one pool, named by the row's part of a table; pages that several rows
hold are counted.

The cache is a dict of numpy arrays: "k", "v" [n_pages, page_size, D] (any dtype: tokens are only
moved), "table" [R, max_pages], "lens" [R], "refs" [n_pages], and optionally "score", "pos"
[R, max_pages * page_size].  Free pages are those with refs 0; :func:`free_mask` gives their bits.
Pages are taken lowest first, for the rows in order; a row that finds too few is left as it was,
and so is every later row that needs a page (the pages are dealt out before any row is served).
"""
from __future__ import annotations

import numpy as np

from .attention_mass import _as_f64


def empty_cache(n_rows, max_pages, n_pages, page_size, head_dim, dtype=np.int16, scores=False, positions=False):
    c = {"k": np.zeros((n_pages, page_size, head_dim), dtype), "v": np.zeros((n_pages, page_size, head_dim), dtype),
         "table": np.full((n_rows, max_pages), -1, np.int64), "lens": np.zeros(n_rows, np.int64),
         "refs": np.zeros(n_pages, np.int64)}
    if scores:
        c["score"] = np.zeros((n_rows, max_pages * page_size))
    if positions:
        c["pos"] = np.zeros((n_rows, max_pages * page_size), np.int64)
    return c


def free_mask(c):
    """The free pages as 32-bit words (int32): bit p % 32 of word p // 32."""
    n = c["refs"].shape[0]
    words = np.zeros((n + 31) // 32, np.uint32)
    for p in range(n):
        if c["refs"][p] == 0:
            words[p // 32] |= np.uint32(1 << (p % 32))
    return words.view(np.int32)


def _pages(n, c):
    return -(-int(n) // c["k"].shape[1])


def _deal(c, needs):
    """Pages for every row's need, or None for a row that is not served."""
    free = [p for p in range(c["refs"].shape[0]) if c["refs"][p] == 0]
    at, out = 0, []
    for need in needs:
        out.append(free[at:at + need] if at + need <= len(free) else (None if need else []))
        at += need
    return out


def _release(c, p):
    assert c["refs"][p] > 0
    c["refs"][p] -= 1


def append(c, new_k, new_v, counts, new_pos=None):
    """new_k, new_v [R, n_new, D].  Returns the rows that found no pages."""
    ps, R = c["k"].shape[1], c["lens"].shape[0]
    shared = [int(counts[r]) > 0 and c["lens"][r] % ps > 0 and
              c["refs"][c["table"][r, c["lens"][r] // ps]] > 1 for r in range(R)]
    firsts = [int(c["lens"][r]) // ps if shared[r] else _pages(c["lens"][r], c) for r in range(R)]
    dealt = _deal(c, [(_pages(c["lens"][r] + counts[r], c) - firsts[r]) if counts[r] else 0 for r in range(R)])
    old = c["table"].copy()
    failed = []
    for r in range(R):
        n, cnt = int(c["lens"][r]), int(counts[r])
        if dealt[r] is None:
            failed.append(r)
            continue
        for j, p in enumerate(dealt[r]):
            c["table"][r, firsts[r] + j] = p
            c["refs"][p] = 1
        if shared[r]:
            p, q = int(old[r, n // ps]), int(c["table"][r, n // ps])
            for o in range(n % ps):
                c["k"][q, o], c["v"][q, o] = c["k"][p, o], c["v"][p, o]
            _release(c, p)
        for i in range(cnt):
            p, o = int(c["table"][r, (n + i) // ps]), (n + i) % ps
            c["k"][p, o], c["v"][p, o] = new_k[r, i], new_v[r, i]
            if "score" in c:
                c["score"][r, n + i] = 0.0
            if "pos" in c:
                c["pos"][r, n + i] = n + i if new_pos is None else int(new_pos[r]) + i
        c["lens"][r] = n + cnt
    return failed


def fork(c, src, copy=False):
    ps, R = c["k"].shape[1], c["lens"].shape[0]
    dealt = _deal(c, [_pages(c["lens"][s], c) if s >= 0 and copy else 0 for s in src])
    failed = []
    for r in range(R):
        s = int(src[r])
        if s < 0:
            continue
        assert s != r and src[s] < 0 and c["lens"][r] == 0
        n = int(c["lens"][s])
        if dealt[r] is None:
            failed.append(r)
            continue
        for j in range(_pages(n, c)):
            p = int(c["table"][s, j])
            if copy:
                q = dealt[r][j]
                for o in range(min(ps, n - j * ps)):
                    c["k"][q, o], c["v"][q, o] = c["k"][p, o], c["v"][p, o]
                p = q
            c["table"][r, j] = p
            c["refs"][p] += 1
        for name in ("score", "pos"):
            if name in c:
                c[name][r, :n] = c[name][s, :n]
        c["lens"][r] = n
    return failed


def compact(c, idx, count):
    """idx [R, b_max], count [R] (negative: the row stays).  Returns the rows that found no pages."""
    ps, R = c["k"].shape[1], c["lens"].shape[0]
    fresh = []
    for r in range(R):
        cnt = int(count[r])
        changed = [any(idx[r, m] != m for m in range(j * ps, min((j + 1) * ps, cnt))) for j in range(_pages(max(cnt, 0), c))]
        fresh.append([j for j, ch in enumerate(changed) if ch and c["refs"][c["table"][r, j]] > 1])
    dealt = _deal(c, [len(f) for f in fresh])
    failed = []
    for r in range(R):
        cnt, n = int(count[r]), int(c["lens"][r])
        if cnt < 0:
            continue
        if dealt[r] is None:
            failed.append(r)
            continue
        kept = [int(j) for j in idx[r, :cnt]]
        assert kept == sorted(set(kept)) and all(0 <= j < n for j in kept)
        tokens = [(c["k"][c["table"][r, j // ps], j % ps].copy(), c["v"][c["table"][r, j // ps], j % ps].copy())
                  for j in kept]
        for j, p in zip(fresh[r], dealt[r]):
            _release(c, int(c["table"][r, j]))
            c["table"][r, j] = p
            c["refs"][p] = 1
        for j in range(_pages(cnt, c), _pages(n, c)):
            _release(c, int(c["table"][r, j]))
            c["table"][r, j] = -1
        for m, (k, v) in enumerate(tokens):
            if kept[m] != m or m // ps in fresh[r]:
                c["k"][c["table"][r, m // ps], m % ps] = k
                c["v"][c["table"][r, m // ps], m % ps] = v
        for name in ("score", "pos"):
            if name in c:
                c[name][r, :cnt] = c[name][r, kept]
        c["lens"][r] = cnt
    return failed


def free(c, keep=None):
    for r in range(c["lens"].shape[0]):
        kept = 0 if keep is None else int(keep[r])
        if kept < 0:
            continue
        for j in range(_pages(kept, c), _pages(c["lens"][r], c)):
            _release(c, int(c["table"][r, j]))
            c["table"][r, j] = -1
        c["lens"][r] = kept


def row_tokens(c, name, r):
    """Row r's tokens of pool ``name`` in order, [lens[r], D]."""
    ps = c["k"].shape[1]
    return np.stack([c[name][c["table"][r, t // ps], t % ps] for t in range(int(c["lens"][r]))]) \
        if c["lens"][r] else c[name][0, :0]


def paged_decode_attn(q, rows_k, rows_v, scale):
    """q [L, H_q, D], rows_k / rows_v: lists of [len, D].  (out [L, H_q, D], lse [L, H_q], list of the
    rows' group-summed probabilities, and sum_t p_t |v_t| [L, H_q, D], which error bounds are made of)."""
    q = _as_f64(q)
    L, Hq, D = q.shape
    R = len(rows_k)
    G = L * Hq // R
    out, mag, lse = np.zeros((L, Hq, D)), np.zeros((L, Hq, D)), np.full((L, Hq), -np.inf)
    mass = []
    for r in range(R):
        k, v = _as_f64(rows_k[r]), _as_f64(rows_v[r])
        mass.append(np.zeros(k.shape[0]))
        if k.shape[0] == 0:
            continue
        for g in range(G):
            l, h = divmod(r * G + g, Hq)
            s = (k @ q[l, h]) * scale
            top = s.max()
            e = np.exp(s - top)
            lse[l, h] = top + np.log(e.sum())
            p = e / e.sum()
            out[l, h] = p @ v
            mag[l, h] = p @ np.abs(v)
            mass[r] += p
    return out, lse, mass, mag
