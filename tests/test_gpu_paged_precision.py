"""How exact paged decode is: fp32 outputs against 64 bits, on inputs whose dot products are exact in any order.

Queries and keys are small multiples of 1/8, so that every partial sum of q . k fits 24 bits: what is left are the steps
behind the logit, each bounded by its own roundings (h(x): half a step of a float of x's size, E = 2^-24):

* a logit is s * (c2 + c2_low) in base 2, kept as a float and what it rounds off (fp32 caches: as the float alone);
  the maximum is taken off and the remainder added: three roundings of at most h(X), X = max |logit| + |largest logit|;
* exp2 is off by 2^-22; a weight's 16-bit parts leave 2^-24 of it (bf16), or 2^-22 and never more than 2^-39 of the row's
  largest weight (f16);
* a product of parts and values on the tensor cores adds up to 16 terms and what stood there, each cut off at E of the
  largest at worst; steps of 16 keys are added up over the tiles of a CTA, tiles by the parts of a row;
* the normaliser keeps what its sums round off, so that the tiles do not show in it: only the merging does.
"""
import math

import pytest
import torch

from tests.test_gpu_paged import DT, i32, kvp  # noqa: F401 (kvp is the fixture)

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
LN2 = math.log(2)


def half_step(x):
    return 2.0 ** (math.floor(math.log2(x)) - 24)


def cache_of(kvp, k, v, ps, spare_pages=0):  # noqa: F811
    """A cache of rows k, v [R, n, D]; spare_pages: room in the table behind them."""
    R, n, D = k.shape
    held = -(-n // ps)
    c = kvp.PagedCache.empty(R, held + spare_pages, R * held, ps, D, k.dtype, scores=True)
    kvp.kvp_paged_append(c, k, v)
    kvp.kvp_check_device_status()
    return c


def reference(q, k, v, scale):
    """Row by row in 64 bits: outputs and lse [R, G, ...], probabilities [R, n], sum p |v|, |logit| and logit maxima (base 2),
    and sum |v| over the weight of the row's largest token (what an absolute error of a weight is worth)."""
    R, n, D = k.shape
    G = q.shape[1] // R
    x = q.double().view(R, G, D) @ k.double().transpose(1, 2) * scale
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    L = e.sum(-1, keepdim=True)
    p = e / L
    v = v.double()
    span = (x.abs().max() + top.abs().max()).item() / LN2
    return p @ v, (top + L.log())[..., 0], p.sum(1), p @ v.abs(), span, v.abs().sum(1)[:, None] / L


def check(kvp, q, k, v, ps, spare_pages, sm_scale=None):  # noqa: F811
    R, n, D = k.shape
    G = q.shape[1] // R
    dtype = k.dtype
    scale = D ** -0.5 if sm_scale is None else sm_scale
    c = cache_of(kvp, k, v, ps, spare_pages)
    out, lse = kvp.kvp_paged_decode_attn(q, c, sm_scale=sm_scale, return_lse=True, add_scores=True)
    kvp.kvp_check_device_status()
    again = kvp.kvp_paged_decode_attn(q, c, sm_scale=sm_scale)
    ref, ref_lse, mass, mag, span, values = reference(q, k, v, scale)

    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    total = R * -(-n // 64)
    tiles = min(total // min(-(-total // 2), ctas) + 1, -(-n // 64))   # of a row, in one CTA
    parts = 1 if n <= 64 else -(-(-(-n // 64)) // tiles) + 1
    exponent = 3 * LN2 * half_step(max(span, 2.0 ** -20))
    weight = exponent + 2.0 ** -22 + {torch.float32: 0.0, torch.bfloat16: E, torch.float16: 4 * E}[dtype]
    # merging: lanes (5), states or warps (up to 16, with a weight of their own each if the row has more than 16 tokens),
    # parts (4 in a lane, 5 over the lanes, 8 steps of 128)
    merge = (5 + min(n, 16)) * E + (2.0 ** -22 if n > 16 else 0) + ((min(parts, 16) + 13) * E + 2.0 ** -22 if parts > 1 else 0)
    normal = exponent + 2.0 ** -22 + 2 * E + merge
    terms = (min(n, 16) + 3) * E if dtype != torch.float32 else 0
    chain = (tiles if dtype != torch.float32 else min(n, 16 * tiles)) * E
    eps = weight + normal + terms + chain + merge + 3 * E
    tol = eps * mag
    if dtype == torch.float16:
        tol = tol + 2.0 ** -39 * values                         # the parts of a weight end at 2^-24, 2^14 above it
    for got in (out, again):
        err = (got.double().view(R, G, D) - ref).abs()
        assert (err <= tol).all(), (eps, (err / mag.clamp(min=1e-300)).max().item())
    err = (lse.double().view(R, G) - ref_lse).abs()
    assert (err <= normal + 2 * LN2 * half_step(span + 40) + 2 * half_step(span + 40)).all(), err.max().item()
    # a score's logit is the float alone, and the row's lse in base 2 a float too
    score = c.score[:, :n].double()
    err = (score - mass).abs()
    seps = weight + normal + 3 * LN2 * half_step(span + 40) + G * E
    assert (err <= seps * mass).all(), (seps, (err / mass).max().item())
    return out.view(R, G, D), ref


def eighths(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda") / 8.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 8), (128, 16), (64, 1)])
@pytest.mark.parametrize("spare", [0, 40])
def test_every_bit_of_a_weight(kvp, dtype, D, G, spare):  # noqa: F811
    """Two tokens, the heavier one of value 0: the output is the other one's weight, so that nothing hides what its parts
    leave out (two bf16 parts leave 2^-18)."""
    R, dt = 128, DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(D + G)
    q = eighths(gen, -8, 8, 1, R * G, D)
    k = eighths(gen, -4, 4, R, 2, D)
    x = (q.view(R, G, D) @ k.transpose(1, 2)) * D ** -0.5
    first = x[:, :1, :1] >= x[:, :1, 1:]                        # the heavier one for the group's first head
    v = torch.where(first.expand(R, 2, D) == torch.tensor([True, False], device="cuda")[None, :, None], 0.0, 1.0)
    check(kvp, q.to(dt), k.to(dt), v.to(dt), 16, spare)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,R,D", [(300, 6, 128), (4096, 48, 128), (4096, 1, 64), (30000, 2, 128)])
@pytest.mark.parametrize("gap", [64, 128, 224])
def test_beside_a_sink(kvp, dtype, n, R, D, gap):  # noqa: F811
    """The first token's dot product is `gap` above the others' (5.7, 11 and 20 in the exponent at head_dim 128): their weights
    are small, many and of values of one sign, so that what each loses adds up.  The sink's own value is 0 in every second row."""
    G, dt = 4, DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(n + gap)
    sign = torch.where(torch.rand(R, 1, D, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    size = torch.tensor([1.0, 0.875, 1.0, 0.75], device="cuda")[None, :, None]
    q = (sign * size).reshape(1, R * G, D)
    k = eighths(gen, -1, 1, R, n, D)
    k[:, 0] = sign[:, 0] * (gap / D)
    v = eighths(gen, 6, 8, R, n, D)
    v[::2, 0] = 0
    check(kvp, q.to(dt), k.to(dt), v.to(dt), 64, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_normaliser_of_a_very_long_row(kvp, dtype):  # noqa: F811
    """2^25 tokens of one weight, every 256th a heavier one: the log-sum-exp in closed form.  Every warp adds up some 1700
    tiles; a sum that forgot what it rounds off would be off by 8e-6 to 1.5e-5 (but for m = 1)."""
    n, D, ps, dt = 1 << 25, 64, 1024, DT[dtype]
    c = kvp.PagedCache.empty(1, n // ps, n // ps, ps, D, dt)
    c.table.copy_(torch.arange(n // ps, device="cuda")[None])
    c.lens.fill_(n)
    c.k_pool.fill_(0.125)
    c.k_pool[:, 0:64:16] = 0.25                                 # one for each warp
    c.v_pool.fill_(1.0)
    heavy = n // ps * 4
    for m in (0.375, 0.5, 0.625, 0.875, 1.0):
        q = torch.full((1, 1, D), m, dtype=dt, device="cuda")
        out, lse = kvp.kvp_paged_decode_attn(q, c, return_lse=True)
        kvp.kvp_check_device_status()
        x, top = D * m * 0.125 / 8, D * m * 0.25 / 8
        ref = top + math.log(heavy + (n - heavy) * math.exp(x - top))
        # the exponent and exp2; the kept remainder, lanes (3), warps (4), parts (2 a thread, 5 over lanes, 7 over warps), their
        # weights; the lse in base 2 (log2, the sum) and as it is returned
        total = (2 + 3 + 4 + 2 + 5 + 7) * E + 2 * 2.0 ** -22
        tol = 3 * LN2 * half_step(2 * top / LN2) + 2.0 ** -22 + total + 3 * LN2 * half_step(ref / LN2) + half_step(ref)
        assert abs(float(lse.double()) - ref) <= tol, (m, float(lse.double()) - ref, tol)
        tiles = n // 64 // 300 + 1                              # outputs are added up tile by tile
        assert ((out.double() - 1).abs() <= 2 * tol + (tiles + 30) * E).all()
