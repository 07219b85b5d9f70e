"""How exact decode over shared prefixes is, on inputs whose dot products are exact in any order (queries and keys are small
multiples of 1/8, so that every partial sum of q . k fits 24 bits), against 64 bits.

What is left are the steps behind the logit, each bounded by its own roundings (h(x): half a step of a float of x's size,
E = 2^-24):

* a logit in base 2 is s times a float scale, less the maximum: the scale (E of the logit), the product and the difference,
  the last two one rounding on the tensor cores; for a weight and for the normaliser's largest each, 3 h(X) with X = max
  |logit| + |largest logit|, twice;
* exp2 is off by 2^-22; a weight's two 16-bit parts leave 2^-16 (bf16) or 2^-22 of it, and f16 parts never less than 2^-39 of
  the row's largest weight;
* the tensor cores add 16 products to what stood there and cut each term off at 2^-23 of the largest: 17 a step at worst.
  Steps are counted over the tokens that stay in one sum (64 tiles of 128 in f16, all in bf16), two for every 16 keys; those sums are added in
  fp32;
* parts of a row are merged in fp32: at most one from every SM, 5 sums over lanes, a weight (2^-22) each;
* the output is rounded once, half a step of its type (below its normal values: half of their smallest step).
"""
import math

import pytest
import torch

import learned_kv_cache_gb300 as kvp
from tests.test_gpu_prefix import DT

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
LN2 = math.log(2)


def half_step(x):
    return 2.0 ** (math.floor(math.log2(x)) - 24)


def eighths(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda") / 8.0


def cache_of(k, v, members, ps):
    """`members` sequences that hold the rows k, v [h_kv, n, D] together."""
    h_kv, n, D = k.shape
    P = -(-n // ps)
    k, v = (torch.nn.functional.pad(x, (0, 0, 0, P * ps - n), value=math.nan).view(h_kv * P, ps, D) for x in (k, v))
    ids = torch.arange(h_kv * P, dtype=torch.int32, device="cuda")
    return kvp.PagedCache(k, v, ids.view(1, h_kv, P).expand(members, h_kv, P).reshape(-1, P).contiguous(),
                          torch.full((members * h_kv,), n, dtype=torch.int32, device="cuda"),
                          torch.full((h_kv * P,), members, dtype=torch.int32, device="cuda"),
                          torch.zeros((h_kv * P + 31) // 32, dtype=torch.int32, device="cuda"))


def tolerance(dtype, n, span, mag, values, want):
    """Bound on the outputs; span: X above, mag: sum p |v|, values: sum |v| over the weight of the row's largest token."""
    segment = {torch.float32: 1 << 30, torch.bfloat16: 1 << 30, torch.float16: 64 * 128}[dtype]
    exponent = 6 * LN2 * half_step(max(span, 2.0 ** -20)) + 2.0 ** -22
    part = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}[dtype]
    steps = 2 * -(-min(n, segment) // 16) if dtype != torch.float32 else 0
    chain = min(17, steps * 16 + 1) * 2.0 ** -23 + (steps + 1) * 2.0 ** -23
    merge = 160 * E + 6 * 2.0 ** -22
    if dtype == torch.float32:
        chain = min(n, segment) * E                          # one after the other
    info = torch.finfo(dtype)
    rounding = info.eps / 2 * (1 + 2 ** -7) * want.abs()
    # below the smallest normal value (f16: 2^-14, outputs beside a sink of value 0) a type's steps stay as they are there:
    # half of one is eps / 2 times that value, 2^-25 in f16
    rounding = rounding.clamp(min=info.eps / 2 * info.tiny)
    tol = (2 * exponent + part + chain + 2 * merge) * mag + rounding
    return tol + 2.0 ** -39 * values if dtype == torch.float16 else tol


def check(q, cache, members, n, heads):
    """q [h_kv, G, D] is every member's; the rows of `heads` are looked at."""
    h_kv, G, D = q.shape
    dtype = q.dtype
    queries = q.reshape(1, h_kv * G, D).expand(members, h_kv * G, D).contiguous()
    lead = torch.zeros(members, dtype=torch.int32, device="cuda")
    out, lse = kvp.kvp_paged_prefix_decode_attn(queries, cache, lead, return_lse=True)
    kvp.kvp_check_device_status()
    out, lse = out.view(members, h_kv, G, D), lse.view(members, h_kv, G)
    for h in heads:
        k, v = (pool[cache.table[h].long()].view(-1, D)[:n].double() for pool in (cache.k_pool, cache.v_pool))
        x = q[h].double() @ k.T * D ** -0.5
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top)
        L = e.sum(-1, keepdim=True)
        want = e / L @ v
        span = (x.abs().max() + top.abs().max()).item() / LN2
        tol = tolerance(dtype, n, span, e / L @ v.abs(), v.abs().sum(0) / L, want)
        err = (out[:, h].double() - want).abs()
        assert (err <= tol).all(), (h, (err / tol).max().item(), (err / want.abs().clamp(min=1e-300)).max().item())
        err = (lse[:, h].double() - (top + L.log())[:, 0]).abs()
        bound = 6 * LN2 * half_step(span + 40) + 2.0 ** -22 + (160 + min(n, 8192)) * E + 6 * 2.0 ** -22
        assert (err <= bound).all(), (h, err.max().item(), bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("members,h_kv,n,D", [
    (2, 1, 300, 128), (2, 160, 3000, 128), (2, 4, 30000, 64), (40, 3, 30000, 128), (70, 160, 2500, 128), (70, 2, 30000, 64)])
@pytest.mark.parametrize("gap", [64, 128, 192, 208, 224])
def test_beside_a_sink(dtype, members, h_kv, n, D, gap):
    """The first token's dot product is `gap` above the others' (5.7, 11, 17, 18 and 20 in the exponent at head_dim 128): their
    weights are small, many and of values of one sign, so that what each loses adds up.  The sink's own value is 0 in every
    second row.  Prefixes and own tokens, up to 128 queries and more, cut over all SMs and whole in one of them."""
    G, dt = 4, DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(n + gap)
    sign = torch.where(torch.rand(h_kv, 1, D, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    size = torch.tensor([1.0, 0.875, 1.0, 0.75], device="cuda")[None, :, None]
    k = eighths(gen, -1, 1, h_kv, n, D)
    k[:, 0] = sign[:, 0] * (gap / D)
    v = eighths(gen, 6, 8, h_kv, n, D)
    v[::2, 0] = 0
    check((sign * size).to(dt), cache_of(k.to(dt), v.to(dt), members, 64), members, n, range(0, h_kv, -(-h_kv // 6)))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("members,n,D", [(1, 262144, 128), (16, 262144, 64), (40, 131072, 128), (1, 16384, 64), (40, 8193, 64),
                                         (16, 16385, 128), (16, 16384 + 128, 64), (40, 16500, 128)])
def test_long_rows_whole_in_one_place(dtype, members, n, D):
    """About as many rows (prefixes) as SMs, so that each is one CTA's whole: values of one sign, whose sums the tensor cores
    would cut at every step.  All rows lie on the same few pages, each in an order of its own."""
    G, h_kv, ps, pages, dt = 4, 152, 1024, 100, DT[dtype]
    if dt == torch.float32:
        h_kv = 12
    gen = torch.Generator(device="cuda").manual_seed(n + members)
    k, v = eighths(gen, -2, 2, pages, ps, D).to(dt), eighths(gen, 6, 8, pages, ps, D).to(dt)
    P = -(-n // ps)
    table = torch.randint(0, pages, (1, h_kv, P), generator=gen, device="cuda", dtype=torch.int32)
    cache = kvp.PagedCache(k, v, table.expand(members, h_kv, P).reshape(-1, P).contiguous(),
                           torch.full((members * h_kv,), n, dtype=torch.int32, device="cuda"),
                           torch.ones(pages, dtype=torch.int32, device="cuda"),
                           torch.zeros((pages + 31) // 32, dtype=torch.int32, device="cuda"))
    check(eighths(gen, -8, 8, h_kv, G, D).to(dt), cache, members, n, range(0, h_kv, -(-h_kv // 8)))


@pytest.mark.parametrize("members,D", [(2, 64), (40, 64), (40, 128)])
def test_the_maximum_grows_from_sum_to_sum(members, D):
    """One row over all SMs, some 200 tiles each, whose logits rise by sqrt(D) / 8 every 2000 tokens and start again after 32000: the sums
    that a place keeps go by smaller and smaller maxima."""
    G, ps = 4, 1024
    n = 152 * 200 * 128 + 77
    gen = torch.Generator(device="cuda").manual_seed(members + D)
    t = torch.arange(n, device="cuda")
    sign = torch.where(torch.rand(D, generator=gen, device="cuda") < 0.5, -1.0, 1.0).half()
    k = sign * (t // 2000 % 16).half()[:, None]
    k[:, 0] = eighths(gen, -4, 4, n).half()
    v = eighths(gen, 2, 8, n, D).half()
    size = torch.tensor([0.125, 0.125, 0.0625, 0.03125], dtype=torch.float16, device="cuda")
    check((sign * size[:, None])[None], cache_of(k[None], v[None], members, ps), members, n, [0])
