"""Decode steps of forked sequences whose rows have lost tokens: queries and keys turned to positions of their own, and kept
keys turned back to positions that close up, against attention in 64 bits over the kept tokens' projections.

Bounds (fp32).  Norm and rotation are off by 2^-20 of the row's length at most (some ten roundings of 2^-24, pairs mixed), so a
dot product by 2^-19 |q| |k|; turned a second time, a key by as much again; the rest as in test_gpu_prefix.
"""
import math

import numpy as np
import pytest
import torch

import learned_kv_cache_gb300 as kvp
from oracle import rope as oracle

pytestmark = pytest.mark.gpu

N, H_KV, G, D, PS = 5, 2, 3, 64, 16
R, HEADS = N * H_KV, H_KV * (G + 2)
PROMPT = 150


def turned(raw, weight, positions, rope):
    return oracle.norm_rope(raw, weight.double().cpu().numpy(), 1e-6, np.asarray(positions), rope.inv_freq, gain=rope.gain)


class Book:
    """The rows' tokens as projections (key, value, position), beside the cache."""

    def __init__(self, scaling, extra):
        self.gen = torch.Generator("cuda").manual_seed(7)
        self.rope = kvp.Rope(D, theta=1e4, scaling=scaling, **extra)
        self.w = torch.rand(D, device="cuda", generator=self.gen) + 0.5
        self.cache = kvp.PagedCache.empty(R, 24, 200, PS, D, torch.float32, positions=True)
        self.lead = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.position = torch.full((N, 1), PROMPT, dtype=torch.int32, device="cuda")      # of the next token
        x = torch.randn(N, PROMPT, HEADS, D, device="cuda", generator=self.gen).transpose(1, 2)
        counts = torch.zeros(R, dtype=torch.int32, device="cuda")
        counts[:H_KV] = PROMPT
        _, k = kvp.kvp_qk_norm_rope(x[:, :H_KV * G], x[:, H_KV * G:H_KV * (G + 1)], self.w, self.w, rope=self.rope)
        kvp.kvp_paged_append(self.cache, k, x[:, H_KV * (G + 1):], counts=counts)
        src = torch.full((N, H_KV), -1, dtype=torch.int32, device="cuda")
        src[1:] = torch.arange(H_KV, device="cuda", dtype=torch.int32)
        kvp.kvp_paged_fork(self.cache, src.view(-1))
        x = x.double().cpu().numpy()
        self.rows = [[(x[0, H_KV * G + r % H_KV, t], x[0, H_KV * (G + 1) + r % H_KV, t], t) for t in range(PROMPT)] for r in range(R)]

    def step(self):
        """Norms, rotation, append, attention over what the rows hold."""
        x = torch.randn(N, 1, HEADS, D, device="cuda", generator=self.gen).transpose(1, 2)
        q, k = kvp.kvp_qk_norm_rope(x[:, :H_KV * G], x[:, H_KV * G:H_KV * (G + 1)], self.w, self.w, rope=self.rope,
                                    positions=self.position)
        kvp.kvp_paged_append(self.cache, k, x[:, H_KV * (G + 1):], new_pos=self.position.repeat(1, H_KV).view(-1))
        out, lse = kvp.kvp_paged_prefix_decode_attn(q[:, :, 0], self.cache, self.lead, return_lse=True)
        kvp.kvp_check_device_status()
        x, at = x.double().cpu().numpy(), self.position.view(-1).tolist()
        for r in range(R):
            n, h = divmod(r, H_KV)
            self.rows[r].append((x[n, H_KV * G + h, 0], x[n, H_KV * (G + 1) + h, 0], at[n]))
            keys, values, positions = (np.stack(c) for c in zip(*self.rows[r]))
            k64 = turned(keys, self.w, positions, self.rope)
            q64 = turned(x[n, h * G:(h + 1) * G, 0], self.w, [at[n]] * G, self.rope)
            logits = q64 @ k64.T / math.sqrt(D)
            top = logits.max(-1, keepdims=True)
            p = np.exp(logits - top)
            want_lse = (top + np.log(p.sum(-1, keepdims=True)))[:, 0]
            p = p / p.sum(-1, keepdims=True)
            e = (2.0 ** -21 * np.abs(q64) @ np.abs(k64).T + 3 * 2.0 ** -20 * np.linalg.norm(q64, axis=-1)[:, None] *
                 np.linalg.norm(k64, axis=-1)[None]).max() / math.sqrt(D)
            tol = (4 * e + 2.0 ** -21) * (p @ np.abs(values)) + 2.0 ** -24 * np.abs(p @ values)
            got = out[n, h * G:(h + 1) * G].double().cpu().numpy()
            assert (np.abs(got - p @ values) <= tol).all(), (r, np.abs(got - p @ values).max(), tol.max())
            got = lse[n, h * G:(h + 1) * G].double().cpu().numpy()
            assert (np.abs(got - want_lse) <= 2 * e + 2.0 ** -20 + 2.0 ** -23 * np.abs(want_lse)).all()
        self.position += 1

    def keep(self, choice):
        """Evict: choice[r] the kept tokens of row r (None: all)."""
        most = max(len(c) for c in choice if c is not None)
        idx, count = torch.zeros(R, most, dtype=torch.int32), torch.full((R,), -1, dtype=torch.int32)
        for r, c in enumerate(choice):
            if c is not None:
                idx[r, :len(c)], count[r] = torch.tensor(c, dtype=torch.int32), len(c)
                self.rows[r] = [self.rows[r][i] for i in c]
        kvp.kvp_paged_compact(self.cache, idx.cuda(), count.cuda())
        kvp.kvp_check_device_status()


def some(seed, rows):
    rng = np.random.default_rng(seed)
    return [sorted(rng.choice(len(x), int(rng.integers(40, 120)), replace=False).tolist()) for x in rows]


SCALINGS = [("none", {}), ("yarn", {"factor": 4.0, "original_len": 64})]


@pytest.mark.parametrize("scaling,extra", SCALINGS)
def test_steps_after_an_eviction(scaling, extra):
    """Heads keep different numbers of tokens; the next tokens' positions go on where they were."""
    book = Book(scaling, extra)
    for _ in range(3):
        book.step()
    choice = some(1, book.rows)
    choice[2 * H_KV:3 * H_KV] = [None] * H_KV              # one sequence keeps everything
    book.keep(choice)
    for _ in range(3):
        book.step()
    assert book.cache.lens.view(N, H_KV)[0, 0] != book.cache.lens.view(N, H_KV)[0, 1]
    assert (book.cache.lens.view(N, H_KV)[3:] < book.position[3:]).all()


@pytest.mark.parametrize("scaling,extra", SCALINGS)
def test_positions_that_close_up(scaling, extra):
    """Kept keys turned back in their pages, by the difference of their old and new positions and with a gain of 1 (they
    have the rotation's already)."""
    book = Book(scaling, extra)
    for _ in range(2):
        book.step()
    # every row loses a token of its first page, so that it shares no page with another any more
    book.keep([[i for i in c if i > 0] for c in some(2, book.rows)])
    cache = book.cache
    # (the row's new positions; the sequence goes on behind its longest row)
    new = torch.arange(24 * PS, device="cuda", dtype=torch.int32)
    held = torch.arange(24, device="cuda") * PS < cache.lens[:, None]
    back = torch.zeros(200, PS, dtype=torch.int32, device="cuda")
    back[cache.table[held].long()] = (cache.pos - new).view(R, 24, PS)[held]
    assert (cache.refs <= 1).all()
    turn = kvp.Rope(D, inv_freq=book.rope.inv_freq)
    assert turn.gain == 1.0
    x = cache.k_pool[:, None]                             # [pages, 1, page_size, D]
    assert kvp.kvp_rope(x, turn, positions=back, inverse=True, out=x) is x
    cache.pos.copy_(new.expand(R, -1))
    book.rows = [[(k, v, i) for i, (k, v, _) in enumerate(row)] for row in book.rows]
    book.position.copy_(cache.lens.view(N, H_KV).amax(1, keepdim=True))
    for _ in range(3):
        book.step()
