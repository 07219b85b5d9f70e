"""The paged KV cache's operators, as cases to measure: decode attention over pages, append, compact, fork, free.

A cache row is one (sequence or layer, KV head); its tokens live in pages of ``page_size`` tokens that a row of ``table``
names.  Every operator stands here in its plain form (elementary torch operations in 32 bits) and, where ``own`` is true,
as the call a user makes of the package.  Operators that change the cache's books get them rolled back at the start of a
pass (one copy), so that a pass can be repeated; the tokens themselves are written to the same places every time.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BASE = {"dtype": "bf16", "head_dim": 128, "page_size": 64, "n_layers": 1, "h_q": 8, "h_kv": 2, "len_min": 1, "len_max": 1,
        "forks": 1, "side": False, "n_new": 0, "new_min": 0, "keep_min": 0, "keep_max": 0, "out16": False, "copy": False}


def _case(name, op, **kw):
    return {"name": name, "op": op, **BASE, **kw}


def listed():
    return [
        # the smallest call: one fp32 layer of 2 query heads on one KV head, 64 kept tokens; only latency counts
        _case("decode tiny f32", "decode", dtype="f32", head_dim=64, page_size=16, h_q=2, h_kv=1, len_min=64, len_max=64),
        # a pruned 28-layer cache at a uniform budget, every slot's attention accumulated for the next eviction
        _case("decode pruned f16 + scores", "decode", dtype="f16", n_layers=28, h_q=12, h_kv=2, len_min=4096, len_max=4096,
              side=True),
        # head-wise budgets (about 15 % of 32768): ragged rows, small pages, the output in the model's type
        _case("decode head-wise bf16", "decode", page_size=32, n_layers=32, h_q=32, h_kv=8, len_min=1000, len_max=8800,
              out16=True),
        # the control run before an eviction: the whole 120000-token cache of 28 layers (the largest case)
        _case("decode full f16", "decode", dtype="f16", n_layers=28, h_q=12, h_kv=2, len_min=120000, len_max=120000),
        # one decode step's new token in every row, half of the rows forked a moment ago (their tail page is still shared)
        _case("append step bf16", "append", page_size=32, n_layers=32, h_q=32, h_kv=8, len_min=1000, len_max=8800, n_new=1,
              new_min=1, forks=2, side=True),
        # one chunk of a chunked prefill behind rows of different lengths
        _case("append chunk f16", "append", dtype="f16", n_layers=28, h_q=12, h_kv=2, len_min=0, len_max=4096, n_new=8192,
              new_min=4096),
        # eviction of the whole 120000-token cache to 4096 tokens a row, with scores and positions
        _case("compact full f16", "compact", dtype="f16", n_layers=28, h_q=12, h_kv=2, len_min=120000, len_max=120000,
              keep_min=4096, keep_max=4096, side=True),
        # eviction to head-wise budgets of rows that share their pages in pairs (fresh pages are needed)
        _case("compact head-wise shared bf16", "compact", page_size=32, n_layers=32, h_q=32, h_kv=8, len_min=8800,
              len_max=16384, keep_min=1000, keep_max=8800, forks=2),
        # eight rows of a 131072-token prompt, each forked to seven more sequences
        _case("fork share bf16", "fork", page_size=128, n_layers=8, h_q=32, h_kv=8, len_min=131072, len_max=131072, forks=8),
        # a layer of 8192 tokens copied to rows that will be evicted on their own
        _case("fork copy bf16", "fork", n_layers=2, h_q=32, h_kv=8, len_min=8192, len_max=8192, forks=2, copy=True, side=True),
        # half of the rows of the 120000-token cache released
        _case("free rows f16", "free", dtype="f16", n_layers=28, h_q=12, h_kv=2, len_min=120000, len_max=120000),
        # rejected drafts: up to 64 tokens cut from the ends of rows that share their pages in pairs
        _case("free cut bf16", "free", page_size=32, n_layers=32, h_q=32, h_kv=8, len_min=1000, len_max=8800, forks=2,
              keep_min=1, keep_max=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "compact", "fork", "free"])
    c = dict(BASE, op=op)
    c["dtype"] = rng.choice(["f32", "bf16", "f16", "bf16", "f16"])
    c["head_dim"] = rng.choice([64, 128, 128])
    c["page_size"] = rng.choice([16, 32, 64, 64, 128, 256])
    c["h_kv"] = rng.choice([1, 2, 3, 4, 8])
    c["h_q"] = c["h_kv"] * rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
    c["n_layers"] = _log(rng, 1, 64)
    c["side"] = rng.random() < 0.4
    c["forks"] = rng.choice([1, 1, 2, 3]) if op != "fork" else rng.choice([2, 3, 5, 8])
    if op == "fork":
        c["copy"] = rng.random() < 0.5
        c["n_layers"] *= c["forks"]
    rows = c["n_layers"] * c["h_kv"]
    most = int(2.5e9 / (rows * 2 * c["head_dim"] * (4 if c["dtype"] == "f32" else 2)))
    if op != "decode":
        most //= 4
    c["len_max"] = _log(rng, 1, max(1, min(131072, most)))
    c["len_min"] = rng.choice([0, 1, c["len_max"], (c["len_max"] + 1) // 2])
    if op == "decode":
        c["out16"] = c["dtype"] != "f32" and rng.random() < 0.5
    if op == "append":
        c["n_new"] = rng.choice([1, 1, _log(rng, 1, max(1, min(8192, most)))])
        c["new_min"] = rng.randint(0, c["n_new"])
    if op in ("compact", "free"):
        c["keep_max"] = _log(rng, 1, c["len_max"])
        c["keep_min"] = rng.randint(0, c["keep_max"])
    return c


def _randint(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def prepare(case, seed):
    c, ps, D = case, case["page_size"], case["head_dim"]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, R, F = DTYPES[c["dtype"]], c["n_layers"] * c["h_kv"], c["forks"]
    lens = _randint(host, c["len_min"], c["len_max"], R)
    family = torch.arange(R) // F * F                     # rows of a family share the first one's pages
    if c["op"] == "fork":                                 # ... from this call on: the others are empty before it
        family = torch.arange(R)
        heads = R // F
        lens[heads:] = 0
        src = torch.where(family < heads, -1, family % max(heads, 1))
    else:
        lens = lens[family]
    new = _randint(host, c["new_min"], c["n_new"], R) if c["op"] == "append" else torch.zeros(R, dtype=torch.int64)
    pages = (lens + ps - 1) // ps
    # sizes go by the case's longest rows, so that every seed has the same ones
    max_pages = -(-(c["len_max"] + c["n_new"]) // ps) + 1
    owner = (family == torch.arange(R)).long()
    used = -(-R // F) * -(-c["len_max"] // ps)
    spare = R * (1 + -(-c["n_new"] // ps)) + (R * -(-c["keep_max"] // ps) if c["op"] == "compact" and F > 1 else 0)
    if c["op"] == "fork" and c["copy"]:
        spare += used * F
    n_pages = used + spare + 3
    place = torch.randperm(n_pages, generator=host)       # as in a server that has run for a while
    start = torch.cumsum(pages * owner, 0) - pages * owner
    col = torch.arange(max_pages)
    at = start[family][:, None] + col
    table = torch.where(col < pages[:, None], place[at.clamp(max=n_pages - 1)], -1)
    refs = torch.zeros(n_pages, dtype=torch.int64)
    refs.scatter_add_(0, table.clamp(min=0).reshape(-1), (table >= 0).long().reshape(-1))
    words = -(-n_pages // 32)
    # the cache's books in one buffer, so that a pass can roll them back with one copy
    parts = [R * max_pages, R, n_pages, words]
    parts = [-(-n // 4) * 4 for n in parts]
    books = torch.zeros(sum(parts), dtype=torch.int32, device=DEV)
    t, l, r, f = books.split(parts)
    s = {"case": c, "books": books, "table": t[:R * max_pages].view(R, max_pages), "lens": l[:R], "refs": r[:n_pages],
         "free_mask": f[:words], "n_pages": n_pages}
    s["table"].copy_(table)
    s["lens"].copy_(lens)
    s["refs"].copy_(refs)
    s["free_mask"].copy_(_mask_of(s["refs"]))
    s["books0"] = books.clone()
    # one page more than the cache has: the plain forms put there what goes nowhere
    pool = [torch.randn(n_pages + 1, ps, D, generator=gen, device=DEV, dtype=torch.float32 if c["dtype"] == "f32" else dt)
            for _ in range(2)]
    s["k_pool"], s["v_pool"] = pool
    cap = max_pages * ps
    if c["side"]:
        s["score"] = torch.rand(R, cap, generator=gen, device=DEV)
        s["pos"] = torch.arange(cap, device=DEV, dtype=torch.int32).expand(R, cap) * 3
        s["pos"] = s["pos"].contiguous()
    else:
        s["score"] = s["pos"] = None
    if c["op"] == "decode":
        _decode_inputs(c, s, gen, host, table, lens, R, F)
    if c["op"] == "append":
        s["new_k"], s["new_v"] = (torch.randn(R, c["n_new"], D, generator=gen, device=DEV, dtype=torch.float32).to(dt)
                                  for _ in range(2))
        s["counts"] = new.to(torch.int32).to(DEV)
        s["new_pos"] = (lens * 3).to(torch.int32).to(DEV)
    if c["op"] == "fork":
        s["src"] = src.to(torch.int32).to(DEV)
    if c["op"] == "free":
        if c["keep_max"]:                                 # that many tokens are cut from the row's end
            keep = (lens - _randint(host, c["keep_min"], c["keep_max"], R)).clamp(min=0)
        else:                                             # half of the rows go, the others stay
            keep = -_randint(host, 0, 1, R)
        s["keep"] = keep.to(torch.int32).to(DEV)
    if c["op"] == "compact":
        _compact_inputs(c, s, gen, host, lens, R)
    if own:
        import learned_kv_cache_gb300 as kvp
        # the handle a user's program keeps: it wraps the buffers above
        s["cache"] = kvp.PagedCache(s["k_pool"][:n_pages], s["v_pool"][:n_pages], s["table"], s["lens"], s["refs"],
                                    s["free_mask"], score=s["score"], pos=s["pos"])
    return s


def _decode_inputs(c, s, gen, host, table, lens, R, F):
    """Queries; keys of a per-head scale; the first tokens' keys along the group's mean query; NaN behind every row's end."""
    ps, D, G = c["page_size"], c["head_dim"], c["h_q"] // c["h_kv"]
    dt = DTYPES[c["dtype"]]
    q = torch.randn(c["n_layers"], c["h_q"], D, generator=gen, device=DEV)
    s["q"] = q.to(dt)
    n_slots = (s["n_pages"] + 1) * ps
    slot = s["table"].long().clamp(min=0)[:, :, None] * ps + torch.arange(ps, device=DEV)
    here = torch.arange(s["table"].shape[1] * ps, device=DEV) < s["lens"][:, None]
    slot = torch.where(here, slot.reshape(R, -1), n_slots - 1)
    live = torch.zeros(n_slots, dtype=torch.bool, device=DEV)
    live[slot.reshape(-1)] = True
    live[n_slots - 1] = False
    scale = torch.rand(s["n_pages"] + 1, generator=gen, device=DEV) * 1.5 + 0.5
    s["k_pool"].mul_(scale[:, None, None].to(s["k_pool"].dtype))
    heads = torch.arange(0, R, F, device=DEV)             # a family's prompt is its first row's
    qbar = q.reshape(R, G, D).mean(1)[heads]
    sink = qbar * (3.0 * math.sqrt(D) / qbar.norm(dim=-1, keepdim=True))
    for name in ("k_pool", "v_pool"):
        flat = s[name].view(n_slots, D)
        if name == "k_pool":
            first = slot[heads][:, :min(4, slot.shape[1])]
            flat[first.reshape(-1)] = sink[:, None].expand(-1, first.shape[1], -1).reshape(-1, D).to(dt)
        flat.masked_fill_(~live[:, None], float("nan"))


def _compact_inputs(c, s, gen, host, lens, R):
    """Kept tokens: 4 sinks, up to 32 recent ones, the best of random scores; ascending, -1 behind them."""
    count = torch.minimum(_randint(host, c["keep_min"], c["keep_max"], R), lens)
    width, T = c["keep_max"], int(lens.max())
    n, cnt = lens.to(DEV)[:, None], count.to(DEV)[:, None]
    col = torch.arange(T, device=DEV)
    score = torch.rand(R, T, generator=gen, device=DEV)
    score = torch.where((col < 4) | (col >= n - 32), 2.0, score)
    score = torch.where(col < n, score, -1.0)
    best = torch.topk(score, min(width, T), dim=1).indices
    if best.shape[1] < width:
        best = torch.nn.functional.pad(best, (0, width - best.shape[1]))
    best = torch.where(torch.arange(width, device=DEV) < cnt, best, T + 1).sort(dim=1).values
    s["idx"] = torch.where(best > T, -1, best).to(torch.int32)
    s["count"] = count.to(torch.int32).to(DEV)


def run(state):
    op = state["case"]["op"]
    if op != "decode":
        state["books"].copy_(state["books0"])
    return OPS[op](state)


def _books(s):
    out = {k: s[k] for k in ("table", "lens", "refs", "free_mask")}
    out["k_pool"], out["v_pool"] = s["k_pool"][:s["n_pages"]], s["v_pool"][:s["n_pages"]]
    if s["score"] is not None:
        out["score"], out["pos"] = s["score"], s["pos"]
    return out


def _decode(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        out, lse = kvp.kvp_paged_decode_attn(s["q"], s["cache"], out_dtype=s["q"].dtype if c["out16"] else None,
                                             add_scores=c["side"], return_lse=True)
        return {"out": out, "lse": lse, **({"score": s["score"]} if c["side"] else {})}
    ps, D, L, Hq = c["page_size"], c["head_dim"], c["n_layers"], c["h_q"]
    R = s["lens"].shape[0]
    G = L * Hq // R
    P = max(1, -(-c["len_max"] // ps))
    T = P * ps
    ids = s["table"][:, :P].clamp(min=0).long()
    live = torch.arange(T, device=s["lens"].device) < s["lens"][:, None]
    k = s["k_pool"][ids].view(R, T, D).float()
    x = torch.matmul(s["q"].float().view(R, G, D), k.transpose(1, 2)) * D ** -0.5
    x = torch.where(live[:, None], x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l > 0, l, 1.0)
    v = s["v_pool"][ids].view(R, T, D)
    v = torch.where(live[:, :, None], v, torch.zeros((), dtype=v.dtype, device=v.device)).float()
    out = torch.matmul(p, v).view(L, Hq, D)
    r = {"out": out.to(s["q"].dtype) if c["out16"] else out, "lse": (m + torch.log(l)).view(L, Hq)}
    if c["side"]:
        s["score"][:, :T] += torch.where(live, p.sum(1), 0.0)
        r["score"] = s["score"]
    return r


def _mask_of(refs):
    """The bits of the pages nobody holds: bit p % 32 of word p // 32."""
    n = refs.shape[0]
    bits = torch.nn.functional.pad((refs == 0).long(), (0, -n % 32)).view(-1, 32)
    word = (bits << torch.arange(32, device=refs.device)).sum(1)
    return ((word ^ (1 << 31)) - (1 << 31)).to(torch.int32)


def _take(s, need):
    """The i-th page needed (rows in order) is the i-th lowest free one: (that order, each row's first, rows served)."""
    off = torch.cumsum(need, 0) - need
    order = torch.argsort((s["refs"] != 0).to(torch.int32), stable=True)
    ok = (need == 0) | (off + need <= (s["refs"] == 0).sum())
    return order, off, ok


def _ids(order, off, k):
    """Page off + k of the free ones (anything where that is past the end)."""
    return order[(off[:, None] + k).clamp(0, order.shape[0] - 1)]


def _ref(s, ids, change):
    s["refs"].scatter_add_(0, ids.clamp(min=0).reshape(-1).long(), change.reshape(-1).to(torch.int32))


def _move(s, src, dst, ok):
    """Token slots src -> dst where ok, both pools; the rest goes to the page behind the cache."""
    trash = s["n_pages"] * s["case"]["page_size"]
    src = torch.where(ok, src, trash).reshape(-1)
    dst = torch.where(ok, dst, trash).reshape(-1)
    for name in ("k_pool", "v_pool"):
        flat = s[name].view(-1, s["case"]["head_dim"])
        flat[dst] = flat[src]


def _append(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        kvp.kvp_paged_append(s["cache"], s["new_k"], s["new_v"], counts=s["counts"],
                             new_pos=s["new_pos"] if c["side"] else None)
        return _books(s)
    ps, n_new = c["page_size"], c["n_new"]
    table, n, cnt = s["table"], s["lens"].long(), s["counts"].long()
    max_pages = table.shape[1]
    tail = table.gather(1, (n // ps).clamp(max=max_pages - 1)[:, None])[:, 0].long()
    cow = (cnt > 0) & (n % ps > 0) & (s["refs"][tail.clamp(min=0)] > 1)
    first = torch.where(cow, n // ps, (n + ps - 1) // ps)
    end = torch.where(cnt > 0, (n + cnt + ps - 1) // ps, first)
    order, off, ok = _take(s, end - first)
    col = torch.arange(max_pages, device=table.device)
    fresh = (col >= first[:, None]) & (col < end[:, None]) & ok[:, None]
    ids = _ids(order, off, col - first[:, None])
    _ref(s, ids, fresh)
    _ref(s, tail, -(cow & ok).int())
    table.copy_(torch.where(fresh, ids, table))
    o = torch.arange(ps, device=table.device)
    _move(s, tail[:, None] * ps + o, _ids(order, off, torch.zeros_like(col[:1])) * ps + o, (cow & ok)[:, None] & (o < (n % ps)[:, None]))
    i = torch.arange(n_new, device=table.device)
    at = n[:, None] + i
    here = (i < cnt[:, None]) & ok[:, None]
    slot = table.long().gather(1, (at // ps).clamp(max=max_pages - 1)) * ps + at % ps
    slot = torch.where(here, slot, s["n_pages"] * ps).reshape(-1)
    for pool, new in (("k_pool", "new_k"), ("v_pool", "new_v")):
        s[pool].view(-1, c["head_dim"])[slot] = s[new].view(-1, c["head_dim"])
    if c["side"]:
        cap = torch.arange(max_pages * ps, device=table.device)
        added = (cap >= n[:, None]) & (cap < (n + cnt)[:, None]) & ok[:, None]
        s["score"].copy_(torch.where(added, 0.0, s["score"]))
        s["pos"].copy_(torch.where(added, s["new_pos"][:, None] + (cap - n[:, None]).int(), s["pos"]))
    s["lens"].copy_(torch.where(ok, n + cnt, n))
    s["free_mask"].copy_(_mask_of(s["refs"]))
    return _books(s)


def _compact(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        kvp.kvp_paged_compact(s["cache"], s["idx"], s["count"])
        return _books(s)
    ps, idx, cnt = c["page_size"], s["idx"].long(), s["count"].long()
    table, n = s["table"], s["lens"].long()
    R, max_pages = table.shape
    width = idx.shape[1]
    old = (n + ps - 1) // ps
    new = (cnt + ps - 1) // ps
    col = torch.arange(max_pages, device=table.device)
    last = torch.minimum((col + 1) * ps, cnt[:, None]) - 1       # the last kept token of each new page
    moved = idx.gather(1, last.clamp(0, width - 1)) != last
    held = table.long().clamp(min=0)
    fresh = (col < new[:, None]) & moved & (s["refs"][held] > 1)
    order, off, ok = _take(s, fresh.sum(1))
    fresh &= ok[:, None]
    ids = torch.where(fresh, _ids(order, off, torch.cumsum(fresh, 1) - 1), table.long())
    m = torch.arange(width, device=table.device)
    here = (m < cnt[:, None]) & ok[:, None]
    src = held.gather(1, (idx.clamp(min=0) // ps)) * ps + idx.clamp(min=0) % ps
    dst = ids.gather(1, (m // ps).clamp(max=max_pages - 1).expand(R, -1)) * ps + m % ps
    _move(s, src, dst, here)
    gone = (col >= new[:, None]) & (col < old[:, None]) & ok[:, None]
    _ref(s, ids, fresh)
    _ref(s, held, -(fresh | gone).int())
    table.copy_(torch.where(gone, -1, ids))
    if c["side"]:
        cap = torch.arange(max_pages * ps, device=table.device)
        back = (cap < cnt[:, None]) & ok[:, None]
        at = torch.where(back, torch.nn.functional.pad(idx, (0, max(0, cap.shape[0] - width)))[:, :cap.shape[0]], cap)
        s["score"].copy_(s["score"].gather(1, at))
        s["pos"].copy_(s["pos"].gather(1, at))
    s["lens"].copy_(torch.where(ok, cnt, n))
    s["free_mask"].copy_(_mask_of(s["refs"]))
    return _books(s)


def _fork(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        kvp.kvp_paged_fork(s["cache"], s["src"], copy=c["copy"])
        return _books(s)
    ps, table, n, src = c["page_size"], s["table"], s["lens"].long(), s["src"].long()
    from_ = src.clamp(min=0)
    length = torch.where(src >= 0, n[from_], 0)
    pages = (length + ps - 1) // ps
    col = torch.arange(table.shape[1], device=table.device)
    theirs = table[from_].long()
    ok = src >= 0
    ids = theirs
    if c["copy"]:
        order, off, served = _take(s, pages)
        ok = ok & served
        ids = _ids(order, off, col)
        o = torch.arange(ps, device=table.device)
        token = col[:, None] * ps + o
        _move(s, theirs[:, :, None] * ps + o, ids[:, :, None] * ps + o, ok[:, None, None] & (token < length[:, None, None]))
    mine = (col < pages[:, None]) & ok[:, None]
    _ref(s, ids, mine)
    table.copy_(torch.where(mine, ids, table.long()))
    if c["side"]:
        here = (torch.arange(s["score"].shape[1], device=table.device) < length[:, None]) & ok[:, None]
        s["score"].copy_(torch.where(here, s["score"][from_], s["score"]))
        s["pos"].copy_(torch.where(here, s["pos"][from_], s["pos"]))
    s["lens"].copy_(torch.where(ok, length, n))
    s["free_mask"].copy_(_mask_of(s["refs"]))
    return _books(s)


def _free(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        kvp.kvp_paged_free(s["cache"], keep=s["keep"])
        return _books(s)
    ps, table, n, keep = c["page_size"], s["table"], s["lens"].long(), s["keep"].long()
    keep = torch.where(keep < 0, n, keep)
    col = torch.arange(table.shape[1], device=table.device)
    gone = (col >= ((keep + ps - 1) // ps)[:, None]) & (col < ((n + ps - 1) // ps)[:, None])
    _ref(s, table.long(), -gone.int())
    table.copy_(torch.where(gone, -1, table))
    s["lens"].copy_(keep)
    s["free_mask"].copy_(_mask_of(s["refs"]))
    return _books(s)


OPS = {"decode": _decode, "append": _append, "compact": _compact, "fork": _fork, "free": _free}


def work(case):
    """Bytes and operations of one pass at the mean of the case's drawn lengths."""
    c = case
    R, D, ps = c["n_layers"] * c["h_kv"], c["head_dim"], c["page_size"]
    elt = 4 if c["dtype"] == "f32" else 2
    n = (c["len_min"] + c["len_max"]) / 2
    token = 2 * D * elt + (8 if c["side"] else 0)          # K and V (score and position) of one token, one way
    heads = c["n_layers"] * c["h_q"]
    if c["op"] == "decode":
        rows = R * n / c["forks"]                          # a shared prompt is read once
        out = heads * D * (2 if c["out16"] else 4) + heads * 4
        return {"bytes": rows * 2 * D * elt + R * n / ps * 4 + heads * D * elt + out + (R * n * 8 if c["side"] else 0),
                "flops": 4 * heads * n * D}
    if c["op"] == "append":
        new = (c["new_min"] + c["n_new"]) / 2
        return {"bytes": R * (new * 2 * token + 16 * (1 + new / ps)), "flops": 0}
    keep = (c["keep_min"] + c["keep_max"]) / 2
    if c["op"] == "compact":
        keep = min(keep, n)
        return {"bytes": R * (keep * (2 * token + 4) + 16 * n / ps + 16), "flops": 0}
    if c["op"] == "fork":
        forked = R - R // c["forks"]
        moved = forked * n * 2 * token if c["copy"] else forked * n * (16 if c["side"] else 0)
        return {"bytes": moved + forked * (n / ps * 16 + 12), "flops": 0}
    cut = min(keep, n) if c["keep_max"] else n / 2
    return {"bytes": R * (cut / ps * 16 + 12), "flops": 0}


def exact(case, seed):
    """Decode attention row by row in 64 bits.  The other operators move tokens and count pages: they compute no numbers."""
    if case["op"] != "decode":
        return None
    s = prepare(case, seed)
    L, Hq, D = s["q"].shape
    R = s["lens"].shape[0]
    G = L * Hq // R
    out = torch.zeros(R, G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((R, G), -math.inf, dtype=torch.float64, device=DEV)
    score = s["score"].double() if case["side"] else None
    q = s["q"].double().reshape(R, G, D)
    for r, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        held = s["table"][r, : (n - 1) // case["page_size"] + 1].long()
        k = s["k_pool"].index_select(0, held).flatten(0, 1)[:n].double()
        logits = torch.einsum("gd,td->gt", q[r], k) / math.sqrt(D)
        lse[r] = torch.logsumexp(logits, 1)
        weight = torch.exp(logits - lse[r][:, None])
        out[r] = weight @ s["v_pool"].index_select(0, held).flatten(0, 1)[:n].double()
        if score is not None:
            score[r, :n] += weight.sum(0)
    return {"out": out.reshape(L, Hq, D), "lse": lse.reshape(L, Hq), **({"score": score} if score is not None else {})}
