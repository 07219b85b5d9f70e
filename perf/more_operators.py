"""Operators around the attention of a step, as cases to measure: position rotation, per-head norms of queries and keys
with the rotation in the same pass (and their gradients), and decode attention for sequences that share a long prompt.

Every operator stands here in its plain form (elementary torch operations in 32 bits, angles in 64) and, where ``own`` is
true, as the call a user makes of the package.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
ROPE = {"dtype": "bf16", "head_dim": 128, "rotary_dim": 128, "interleaved": False, "theta": 1e6, "scaling": "none",
        "factor": 1.0, "original_len": 8192, "batch": 1, "h_q": 32, "h_kv": 8, "seq": 1, "pos_max": 0, "inverse": False}
PREFIX = {"dtype": "bf16", "head_dim": 128, "page_size": 64, "n_layers": 1, "h_q": 32, "h_kv": 8, "families": 1, "members": 2,
          "prompt_min": 64, "prompt_max": 64, "own_min": 1, "own_max": 1, "strays": False}


def _case(name, op, **kw):
    return {"name": name, "op": op, **(PREFIX if op == "prefix" else ROPE), **kw}


def listed():
    return [
        # one decode step of a small batch deep in its context: queries and keys rotated where the projection left them
        _case("rope step f16", "rope", dtype="f16", batch=8, h_q=12, h_kv=2, pos_max=120000),
        # a 32768-token prefill with frequencies stretched by bands of wavelengths
        _case("rope prefill bands bf16", "rope", theta=5e5, scaling="bands", factor=8.0, seq=32768),
        # keys turned back to position 0 (an eviction that closes up its positions, or the gradient): half of each head
        # rotated, in neighbouring pairs, fp32, ragged batch
        _case("rope back interleaved f32", "rope", dtype="f32", head_dim=64, rotary_dim=32, interleaved=True, theta=1e4,
              batch=3, h_q=2, h_kv=1, seq=1001, pos_max=5000, inverse=True),
        # one decode step of 64 sequences: norms and rotation of 40 heads each
        _case("norm rope step bf16", "norm", batch=64, pos_max=40000),
        # a layer's prefill of 8192 tokens
        _case("norm rope prefill bf16", "norm", seq=8192),
        # a layer's prefill of 131072 tokens, positions stretched by interpolation in part of the spectrum
        _case("norm rope long yarn bf16", "norm", seq=131072, scaling="yarn", factor=4.0, original_len=32768),
        # the gradients of the 8192-token layer, weights' included
        _case("norm rope backward bf16", "norm_bwd", seq=8192),
        # the same of a small fp32 model with ragged sizes
        _case("norm rope backward f32", "norm_bwd", dtype="f32", head_dim=64, rotary_dim=64, theta=1e4, batch=3, h_q=2, h_kv=1,
              seq=333),
        # a draft and its parent on one short prompt: only latency counts
        _case("prefix tiny f32", "prefix", dtype="f32", head_dim=64, page_size=16, h_q=2, h_kv=1, own_max=9),
        # 32 answers sampled from one 32768-token prompt
        _case("prefix 32 answers bf16", "prefix", members=32, prompt_min=32768, prompt_max=32768, own_max=1000),
        # 7 of 28 layers, eight answers on a 120000-token prompt
        _case("prefix 8 answers f16", "prefix", dtype="f16", n_layers=7, h_q=12, h_kv=2, members=8, prompt_min=120000,
              prompt_max=120000, own_max=500),
        # several prompts evicted head by head before they were forked, 64 answers each; some answers evicted on their own since
        _case("prefix head-wise bf16", "prefix", page_size=32, families=4, members=64, prompt_min=1000, prompt_max=8800,
              own_max=300, strays=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "norm_bwd", "prefix", "prefix"])
    c = dict(PREFIX if op == "prefix" else ROPE, op=op)
    c["dtype"] = rng.choice(["f32", "bf16", "f16", "bf16", "f16"])
    elt = 4 if c["dtype"] == "f32" else 2
    c["head_dim"] = D = rng.choice([64, 128, 128])
    c["h_kv"] = rng.choice([1, 2, 3, 4, 8])
    c["h_q"] = c["h_kv"] * rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
    if op == "prefix":
        c["page_size"] = rng.choice([16, 32, 64, 64, 128, 256])
        c["families"] = _log(rng, 1, 16)
        c["members"] = _log(rng, 2, 64)
        c["n_layers"] = _log(rng, 1, 8)
        rows = c["n_layers"] * c["families"] * c["members"] * c["h_kv"]
        most = int(4e9 / (rows * D * 4)) if c["dtype"] != "f32" else int(1e9 / (rows * D * 4))
        most = max(2, min(most, int(1e12 / (rows * D * c["h_q"] // c["h_kv"]))))
        c["prompt_max"] = _log(rng, 1, min(131072, most))
        c["prompt_min"] = rng.choice([1, c["prompt_max"], (c["prompt_max"] + 1) // 2])
        c["own_max"] = _log(rng, 1, max(1, min(2000, most // 4)))
        c["own_min"] = rng.choice([0, 1, c["own_max"]])
        c["strays"] = rng.random() < 0.3
        return c
    c["rotary_dim"] = rng.choice([D, D, D // 2, D // 4, 3 * D // 4])
    c["interleaved"] = rng.random() < 0.4
    c["theta"] = rng.choice([1e4, 5e5, 1e6])
    c["scaling"] = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
    c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
    c["batch"] = _log(rng, 1, 64)
    row = (c["h_q"] + 2 * c["h_kv"]) * D * elt
    c["seq"] = rng.choice([1, _log(rng, 1, max(1, min(131072, int(5e8 / (c["batch"] * row)))))])
    c["pos_max"] = rng.choice([0, 1000, 120000])
    c["inverse"] = op == "rope" and rng.random() < 0.4
    return c


def prepare(case, seed):
    return _prepare_prefix(case, seed) if case["op"] == "prefix" else _prepare_rope(case, seed)


def _inv_freq(c):
    """Radians per position of every pair, and the factor on cosine and sine (fp64)."""
    r, scaling, factor = c["rotary_dim"], c["scaling"], c["factor"]
    e = torch.arange(0, r, 2, dtype=torch.float64) / r
    theta = c["theta"] * (factor ** (r / (r - 2)) if scaling == "ntk" else 1.0)
    inv, gain = theta ** -e, 1.0
    if scaling == "linear":
        inv = inv / factor
    if scaling == "bands":               # long waves are stretched, short ones stay, a ramp between wavelengths n / 4 and n
        smooth = ((c["original_len"] * inv / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)
        inv = (1 - smooth) * inv / factor + smooth * inv
    if scaling == "yarn":                # a ramp over the pairs that turn 32 times ... once within the original length
        def pair(turns):
            return r * math.log(c["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(c["theta"]))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        gain = 0.1 * math.log(factor) + 1.0
    return inv, gain


def _prepare_rope(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, D, B, S, Hq, Hkv = DTYPES[c["dtype"]], c["head_dim"], c["batch"], c["seq"], c["h_q"], c["h_kv"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32 if dt == torch.float32 else dt)

    # what a fused projection leaves: per token the query heads, the key heads, the value heads
    qkv = randn(B, S, Hq + 2 * Hkv, D)
    heads = torch.rand(Hq + 2 * Hkv, 1, generator=gen, device=DEV) * 3 + 0.2
    qkv.mul_(heads.to(qkv.dtype))
    start = torch.randint(0, c["pos_max"] + 1, (B, 1), generator=gen, device=DEV)
    s = {"case": c, "qkv": qkv, "positions": (start + torch.arange(S, device=DEV)).to(torch.int32)}
    s["inv"], s["gain"] = (_inv_freq(c)[0].to(DEV), _inv_freq(c)[1])
    if c["op"] != "rope":
        for name in ("q_weight", "k_weight"):
            s[name] = (torch.rand(D, generator=gen, device=DEV) * 2 + 0.1).to(dt)
    if c["op"] == "norm_bwd":
        s["dq"], s["dk"] = randn(B, Hq, S, D), randn(B, Hkv, S, D)
    if own:
        import learned_kv_cache_gb300 as kvp
        # the frequencies that a model keeps
        s["rope"] = kvp.Rope(c["rotary_dim"], theta=c["theta"], interleaved=c["interleaved"], scaling=c["scaling"],
                             factor=c["factor"], original_len=c["original_len"])
    return s


def _prepare_prefix(c, seed):
    ps, D, L, F, M, Hkv = c["page_size"], c["head_dim"], c["n_layers"], c["families"], c["members"], c["h_kv"]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, G = DTYPES[c["dtype"]], c["h_q"] // c["h_kv"]
    N = F * M                                             # sequences of a layer
    R = L * N * Hkv                                       # row = (layer, sequence, KV head)

    def randint(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=host)

    prompt = randint(c["prompt_min"], c["prompt_max"], L, F, 1, Hkv).expand(L, F, M, Hkv).reshape(R)
    new = randint(c["own_min"], c["own_max"], 1, F, M, 1).expand(L, F, M, Hkv).reshape(R)
    lens = prompt + new
    shared = prompt // ps                                 # pages of the prompt that stay shared once a row has grown
    member = torch.arange(M).view(1, 1, M, 1).expand(L, F, M, Hkv).reshape(R)
    if c["strays"]:                                       # every eighth row evicted by itself somewhere in its prompt
        stray = (randint(0, 7, R) == 0) & (member > 0)
        shared = torch.where(stray, (shared * torch.rand(R, generator=host)).long(), shared)
    pages = (lens + ps - 1) // ps
    max_pages = -(-(c["prompt_max"] + c["own_max"]) // ps) + 1
    first = torch.arange(R).view(L, F, M, Hkv)[:, :, :1].expand(L, F, M, Hkv).reshape(R)
    mine = torch.where(member == 0, pages, pages - shared)
    used = L * F * Hkv * (c["prompt_max"] // ps + 1) + R * (c["own_max"] // ps + 2)
    if c["strays"]:
        used += (R if R < 64 else R // 4) * (c["prompt_max"] // ps)
    used = max(used, int(mine.sum()))
    n_pages = used + 3
    place = torch.randperm(n_pages, generator=host)       # as in a server that has run for a while
    start = torch.cumsum(mine, 0) - mine
    col = torch.arange(max_pages)
    theirs = (member > 0)[:, None] & (col < shared[:, None])
    at = torch.where(theirs, start[first][:, None] + col, start[:, None] + col - torch.where(member > 0, shared, 0)[:, None])
    table = torch.where(col < pages[:, None], place[at.clamp(0, n_pages - 1)], -1)
    refs = torch.zeros(n_pages, dtype=torch.int64)
    refs.scatter_add_(0, table.clamp(min=0).reshape(-1), (table >= 0).long().reshape(-1))
    bits = torch.nn.functional.pad((refs == 0).long(), (0, -n_pages % 32)).view(-1, 32)
    word = (bits << torch.arange(32)).sum(1)
    s = {"case": c, "table": table.to(torch.int32).to(DEV), "lens": lens.to(torch.int32).to(DEV),
         "refs": refs.to(torch.int32).to(DEV), "free_mask": ((word ^ (1 << 31)) - (1 << 31)).to(torch.int32).to(DEV)}
    # the sequence that each one was forked from
    lead = torch.arange(L * N).view(L, F, M)[:, :, :1].expand(L, F, M).reshape(-1)
    s["lead"] = lead.to(torch.int32).to(DEV)
    q = torch.randn(L * N, c["h_q"], D, generator=gen, device=DEV)
    s["q"] = q.to(dt)
    # keys of a scale per page, the first tokens' along the queries' mean, NaN where no row has a token
    live = torch.zeros(n_pages, ps, dtype=torch.bool)
    ends = torch.where(col < pages[:, None], (lens[:, None] - col * ps).clamp(max=ps), 0)
    fill = torch.zeros(n_pages, dtype=torch.int64)
    fill.scatter_reduce_(0, table.clamp(min=0).reshape(-1), ends.reshape(-1), "amax")
    live = (torch.arange(ps) < fill[:, None]).to(DEV)
    scale = torch.rand(n_pages, 1, 1, generator=gen, device=DEV) * 1.5 + 0.5
    for name in ("k_pool", "v_pool"):
        pool = torch.randn(n_pages, ps, D, generator=gen, device=DEV, dtype=torch.float32 if c["dtype"] == "f32" else dt)
        if name == "k_pool":
            pool.mul_(scale.to(pool.dtype))
            qbar = q.view(L, F, M, Hkv, G, D).mean((2, 4)).reshape(-1, D)
            sink = qbar * (3.0 * math.sqrt(D) / qbar.norm(dim=-1, keepdim=True))
            head = torch.arange(R).view(L, F, M, Hkv)[:, :, 0].reshape(-1)
            pool[s["table"][head, 0].long().clamp(min=0), 0] = sink.to(dt)
        s[name] = pool.masked_fill_(~live[:, :, None], float("nan"))
    if own:
        import learned_kv_cache_gb300 as kvp
        s["cache"] = kvp.PagedCache(s["k_pool"], s["v_pool"], s["table"], s["lens"], s["refs"], s["free_mask"])
    return s


def run(state):
    return OPS[state["case"]["op"]](state)


def _views(s):
    c = s["case"]
    x = s["qkv"].transpose(1, 2)                          # [B, heads, S, D], as the projection left it
    return x[:, :c["h_q"]], x[:, c["h_q"]:c["h_q"] + c["h_kv"]]


def _cos_sin(s, inverse=False):
    angle = s["positions"].double()[:, None, :, None] * s["inv"]
    sin = torch.sin(angle)
    return (torch.cos(angle) * s["gain"]).float(), ((-sin if inverse else sin) * s["gain"]).float()


def _rotate(x, cos, sin, c):
    """Rotates the pairs of the first rotary_dim values of every head (fp32)."""
    r = c["rotary_dim"]
    y = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _rope(s):
    c = s["case"]
    x = s["qkv"].transpose(1, 2)[:, :c["h_q"] + c["h_kv"]]
    if own:
        import learned_kv_cache_gb300 as kvp
        return kvp.kvp_rope(x, s["rope"], positions=s["positions"], inverse=c["inverse"])
    cos, sin = _cos_sin(s, c["inverse"])
    return _rotate(x.float(), cos, sin, c).to(x.dtype)


def _norm(s):
    c = s["case"]
    q, k = _views(s)
    if own:
        import learned_kv_cache_gb300 as kvp
        return kvp.kvp_qk_norm_rope(q, k, s["q_weight"], s["k_weight"], EPS, s["rope"], positions=s["positions"])
    cos, sin = _cos_sin(s)

    def one(x, w):
        x32 = x.float()
        x32 = x32 * torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS) * w.float()
        return _rotate(x32, cos, sin, c).to(x.dtype)
    return one(q, s["q_weight"]), one(k, s["k_weight"])


def _norm_bwd(s):
    c = s["case"]
    q, k = _views(s)
    if own:
        import learned_kv_cache_gb300 as kvp
        return kvp.kvp_qk_norm_rope_backward(s["dq"], s["dk"], q, k, s["q_weight"], s["k_weight"], EPS, s["rope"],
                                             positions=s["positions"])
    cos, sin = _cos_sin(s, inverse=True)

    def one(dy, x, w):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
        n = x32 * r
        dz = _rotate(dy.float(), cos, sin, c)
        dw = (dz * n).sum((0, 1, 2), dtype=torch.float64).float()
        dn = dz * w.float()
        return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype), dw
    dq, dwq = one(s["dq"], q, s["q_weight"])
    dk, dwk = one(s["dk"], k, s["k_weight"])
    return dq, dk, dwq, dwk


def _prefix(s):
    c = s["case"]
    if own:
        import learned_kv_cache_gb300 as kvp
        out, lse = kvp.kvp_paged_prefix_decode_attn(s["q"], s["cache"], s["lead"], return_lse=True)
        return {"out": out, "lse": lse}
    ps, D, Hq = c["page_size"], c["head_dim"], c["h_q"]
    R, N = s["lens"].shape[0], s["q"].shape[0]
    G = N * Hq // R
    P = max(1, -(-(c["prompt_max"] + c["own_max"]) // ps))
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
    return {"out": torch.matmul(p, v).view(N, Hq, D).to(s["q"].dtype), "lse": (m + torch.log(l)).view(N, Hq)}


OPS = {"rope": _rope, "norm": _norm, "norm_bwd": _norm_bwd, "prefix": _prefix}


def work(case):
    """Bytes and operations of one pass at the mean of the case's drawn lengths."""
    c = case
    elt, D = 4 if c["dtype"] == "f32" else 2, c["head_dim"]
    if c["op"] == "prefix":
        lone = c["n_layers"] * c["families"] * c["h_kv"]  # prompts, a row each
        rows = lone * c["members"]
        prompt, new = (c["prompt_min"] + c["prompt_max"]) / 2, (c["own_min"] + c["own_max"]) / 2
        queries = rows * (c["h_q"] // c["h_kv"])
        tokens = lone * prompt + rows * new               # a prompt is read once for all that share it
        if c["strays"]:
            tokens += (rows - lone) * prompt / 16
        return {"bytes": tokens * 2 * D * elt + rows * (prompt + new) / c["page_size"] * 4 + queries * (2 * D * elt + 4),
                "flops": 4 * D * queries * (prompt + new)}
    n = c["batch"] * c["seq"] * (c["h_q"] + c["h_kv"]) * D
    turned = n * c["rotary_dim"] / D
    tensors = 3 if c["op"] == "norm_bwd" else 2
    flops = {"rope": 3 * turned, "norm": 3 * turned + 4 * n, "norm_bwd": 3 * turned + 11 * n}[c["op"]]
    return {"bytes": tensors * n * elt + c["batch"] * c["seq"] * 4, "flops": flops}


def _turns(c):
    """The definition pair by pair: (radians per position, gain)."""
    r, out = c["rotary_dim"], []
    f, n = c["factor"], c["original_len"]
    for i in range(r // 2):
        w = c["theta"] ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            w /= f
        elif c["scaling"] == "ntk":
            w = (c["theta"] * f ** (r / (r - 2.0))) ** (-2.0 * i / r)
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / w
            if wave > n:
                w /= f
            elif wave > n / 4:
                t = (n / wave - 1.0) / 3.0
                w = (1 - t) * w / f + t * w
        elif c["scaling"] == "yarn":
            lo = max(math.floor(r * math.log(n / (32 * 2 * math.pi)) / (2 * math.log(c["theta"]))), 0)
            hi = min(math.ceil(r * math.log(n / (2 * math.pi)) / (2 * math.log(c["theta"]))), r - 1)
            t = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = t * w / f + (1 - t) * w
        out.append(w)
    return out, (0.1 * math.log(f) + 1.0 if c["scaling"] == "yarn" else 1.0)


def _exact_turn(x, s, sign):
    """x (fp64, [B, H, S, D]) with its pairs multiplied by gain * e^(i sign angle)."""
    c = s["case"]
    r = c["rotary_dim"]
    w, gain = _turns(c)
    angle = s["positions"].double()[:, None, :, None] * torch.tensor(w, dtype=torch.float64, device=DEV) * sign
    turn = torch.polar(torch.full_like(angle, gain), angle)
    part = x[..., :r]
    pairs = part.unflatten(-1, (r // 2, 2)) if c["interleaved"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z if c["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., r:]], -1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "prefix":
        return _exact_prefix(s)
    D, sign = c["head_dim"], -1.0 if c["inverse"] else 1.0
    if c["op"] == "rope":
        return _exact_turn(s["qkv"].transpose(1, 2)[:, :c["h_q"] + c["h_kv"]].double(), s, sign)
    done = []
    for x, name in zip(_views(s), ("q", "k")):
        x, w = x.double(), s[name + "_weight"].double()
        length = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
        if c["op"] == "norm":
            done.append(_exact_turn(x / length * w, s, 1.0))
            continue
        back = _exact_turn(s["d" + name].double(), s, -1.0)
        inner = (back * w * x).sum(-1, keepdim=True)
        done.append((back * w - x * inner / (D * length * length)) / length)
        done.append((back * x / length).sum((0, 1, 2)))
    return tuple(done) if c["op"] == "norm" else (done[0], done[2], done[1], done[3])


def _exact_prefix(s):
    """Row by row in 64 bits; the rows' tokens gathered one row at a time."""
    c = s["case"]
    N, Hq, D = s["q"].shape
    R = s["lens"].shape[0]
    if R * (c["prompt_max"] + c["own_max"]) > 3e7:
        return None
    G = N * Hq // R
    q = s["q"].double().reshape(R, G, D)
    out = torch.zeros(R, G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((R, G), -math.inf, dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        held = s["table"][r, : (n - 1) // c["page_size"] + 1].long()
        k = s["k_pool"].index_select(0, held).flatten(0, 1)[:n].double()
        logits = torch.einsum("gd,td->gt", q[r], k) / math.sqrt(D)
        lse[r] = torch.logsumexp(logits, 1)
        out[r] = torch.exp(logits - lse[r][:, None]) @ s["v_pool"].index_select(0, held).flatten(0, 1)[:n].double()
    return {"out": out.reshape(N, Hq, D), "lse": lse.reshape(N, Hq)}
