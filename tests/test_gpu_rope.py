"""Rotary positions and the norms of queries and keys against the fp64 oracle.

Bounds count roundings.  A step is 2^-24 (half the spacing of float32 at 1).  A turned value a c - b s: cosine and sine
are off by 2 steps of 1 (the angle's remainder, the function) and one more by the gain, two products and a sum add 3:
8 steps of gain (|a| + |b|) are allowed.  A normalised value has in it the sum of squares (D / 16 lanes of 16 terms:
20 additions, halved by the root), the mean, the root and two products: 16 steps.  Gradients multiply such values: 64
steps of what the terms sum to in absolute value.  The result's own rounding is half a step of its type.
"""
import numpy as np
import pytest
import torch

import learned_kv_cache_gb300 as kvp
import oracle

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def np64(t):
    return t.detach().cpu().double().numpy()


def half(t):
    return torch.finfo(t.dtype).eps / 2


def mixed(x, rope):
    """|a| + |b| of the pair that every value is in (|a| behind them)."""
    x, r, y = np.abs(x), rope.rotary_dim if rope else 0, np.abs(x).copy()
    n = r // 2
    if rope and rope.interleaved:
        y[..., 0:r:2] = y[..., 1:r:2] = x[..., 0:r:2] + x[..., 1:r:2]
    elif rope:
        y[..., :n] = y[..., n:r] = x[..., :n] + x[..., n:r]
    return y * (max(1.0, abs(rope.gain)) if rope else 1.0)


def close(got, want, bound):
    got64 = np64(got)
    err = np.abs(got64 - want)
    worst = (err - (bound + half(got) * np.abs(want) * (1 + 2 ** -10) + torch.finfo(got.dtype).tiny)).max()
    assert np.isfinite(got64).all() and worst <= 0, (err.max(), worst)


def spec(rope):
    return dict(inv_freq=rope.inv_freq, interleaved=rope.interleaved, gain=rope.gain) if rope else {}


def randn(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


ROPES = [dict(rotary_dim=64), dict(rotary_dim=64, interleaved=True), dict(rotary_dim=16, theta=1e6),
         dict(rotary_dim=48, interleaved=True, scaling="yarn", factor=4.0, original_len=4096)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D,kw", [(64, k) for k in ROPES] + [
    (128, dict(rotary_dim=128, theta=1e6)), (128, dict(rotary_dim=128, interleaved=True)), (128, dict(rotary_dim=96)),
    (128, dict(rotary_dim=32, interleaved=True, scaling="bands", factor=8.0, original_len=8192))])
@pytest.mark.parametrize("B,H,S", [(1, 1, 1), (3, 5, 1), (2, 3, 77), (1, 42, 333)])
def test_rope(dtype, D, kw, B, H, S):
    gen = torch.Generator("cuda").manual_seed(S + D)
    rope = kvp.Rope(**kw)
    x = randn(gen, B, H, S, D, dtype=DT[dtype])
    pos = torch.randint(-1000, 200000, (B, S), generator=gen, device="cuda").to(torch.int32)
    for inverse in (False, True):
        y = kvp.kvp_rope(x, rope, positions=pos, inverse=inverse)
        assert y.shape == x.shape and y.dtype == x.dtype
        want = oracle.rotate(np64(x), pos.cpu().numpy()[:, None], inverse=inverse, **spec(rope))
        close(y, want, 8 * STEP * mixed(np64(x), rope))
        assert torch.equal(y[..., rope.rotary_dim:], x[..., rope.rotary_dim:])


def test_far_positions_and_starts():
    gen = torch.Generator("cuda").manual_seed(1)
    rope = kvp.Rope(128, theta=1e6)
    x = randn(gen, 1, 2, 6, 128, dtype=torch.float32)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 0, 2 ** 24 + 1, 131071], dtype=torch.int32, device="cuda")
    want = oracle.rotate(np64(x), pos.cpu().numpy(), rope.inv_freq)
    close(kvp.kvp_rope(x, rope, positions=pos), want, 8 * STEP * mixed(np64(x), rope))
    for start in (0, 120001, 2 ** 31 - 6, -2 ** 31):
        want = oracle.rotate(np64(x), start + np.arange(6), rope.inv_freq)
        close(kvp.kvp_rope(x, rope, start=start), want, 8 * STEP * mixed(np64(x), rope))


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_in_place_and_shared_positions(dtype):
    """A fused projection's slice, a token-major output, the input itself, one row of positions, x without a batch."""
    gen = torch.Generator("cuda").manual_seed(2)
    rope = kvp.Rope(64)
    B, H, S, D = 3, 4, 19, 64
    qkv = randn(gen, B, S, (H + 3) * D, dtype=DT[dtype])
    x = qkv[..., 2 * D:(H + 2) * D].view(B, S, H, D).transpose(1, 2)
    pos = torch.arange(5, 5 + S, dtype=torch.int32, device="cuda")
    want = kvp.kvp_rope(x.contiguous(), rope, positions=pos.expand(B, S).contiguous())
    out = torch.full((B, S, H, D), 7.0, dtype=x.dtype, device="cuda")
    kvp.kvp_rope(x, rope, positions=pos, out=out.transpose(1, 2))
    assert torch.equal(out.transpose(1, 2), want)
    wide = pos.repeat(B, 2)[:, :S]                        # rows of positions further apart than they are long
    assert torch.equal(kvp.kvp_rope(x, rope, positions=wide), want)
    assert torch.equal(kvp.kvp_rope(x, rope, positions=pos.expand(B, S)), want)
    assert torch.equal(kvp.kvp_rope(x[1], rope, start=5), want[1])
    shared = x[:1].expand(B, H, S, D)                     # an input that is broadcast
    assert torch.equal(kvp.kvp_rope(shared, rope, start=5), want[:1].expand(B, H, S, D))
    before = qkv.clone()
    assert kvp.kvp_rope(x, rope, positions=pos, out=x) is x
    assert torch.equal(x, want)
    rest = torch.cat([qkv[..., :2 * D], qkv[..., (H + 2) * D:]], -1)
    assert torch.equal(rest, torch.cat([before[..., :2 * D], before[..., (H + 2) * D:]], -1))


def test_infinities_stay_in_their_pairs():
    rope = kvp.Rope(32)
    x = torch.ones(1, 1, 4, 64, device="cuda")
    x[0, 0, 0, 40] = float("inf")                         # behind the rotated part
    x[0, 0, 1, 3] = float("inf")
    y = kvp.kvp_rope(x, rope, start=1)
    bad = ~torch.isfinite(y[0, 0])
    assert bad[0].nonzero().flatten().tolist() == [40] and set(bad[1].nonzero().flatten().tolist()) == {3, 19}
    assert not bad[2:].any()


NORMS = [("f32", 64, 2, 1, dict(rotary_dim=32)), ("f32", 128, 5, 3, dict(rotary_dim=128, interleaved=True)), ("f32", 64, 1, 1, None),
         ("bf16", 128, 32, 8, dict(rotary_dim=128, theta=1e6)), ("bf16", 64, 3, 7, dict(rotary_dim=48, interleaved=True)),
         ("f16", 128, 12, 2, None), ("f16", 64, 16, 1, dict(rotary_dim=64)), ("f16", 128, 40, 40, dict(rotary_dim=16))]


def norm_case(dtype, D, Hq, Hkv, kw, B, S, seed=0, weight="same"):
    gen = torch.Generator("cuda").manual_seed(seed + S)
    qkv = randn(gen, B, S, (Hq + 2 * Hkv) * D, dtype=DT[dtype]) * 3
    heads = qkv.view(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
    w = [None, None]
    if weight != "none":
        w = [(torch.rand(D, generator=gen, device="cuda") * 2 - 0.5).to(torch.float32 if weight == "f32" else DT[dtype])
             for _ in range(2)]
    pos = torch.randint(0, 100000, (B, S), generator=gen, device="cuda").to(torch.int32)
    return heads[:, :Hq], heads[:, Hq:Hq + Hkv], w, (kvp.Rope(**kw) if kw else None), pos, gen


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("B,S,weight", [(1, 1, "same"), (5, 1, "f32"), (2, 67, "same"), (1, 700, "none")])
def test_norm_rope(case, B, S, weight):
    dtype, D, Hq, Hkv, kw = case
    q, k, w, rope, pos, _ = norm_case(dtype, D, Hq, Hkv, kw, B, S, weight=weight)
    outs = kvp.kvp_qk_norm_rope(q, k, w[0], w[1], 1e-5, rope, positions=pos)
    p = pos.cpu().numpy()[:, None]
    for x, y, wt in zip((q, k), outs, w):
        wt = None if wt is None else np64(wt)
        z = oracle.norm_rope(np64(x), wt, 1e-5)
        close(y, oracle.norm_rope(np64(x), wt, 1e-5, p, **spec(rope)), 24 * STEP * mixed(z, rope))
    # in place, from the same inputs
    a, b = q.contiguous(), k.contiguous()
    kvp.kvp_qk_norm_rope(a, b, w[0], w[1], 1e-5, rope, positions=pos, q_out=a, k_out=b)
    assert torch.equal(a, outs[0]) and torch.equal(b, outs[1])


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("B,S,weight", [(1, 1, "same"), (5, 1, "f32"), (2, 67, "none"), (3, 700, "same")])
def test_norm_rope_backward(case, B, S, weight):
    dtype, D, Hq, Hkv, kw = case
    q, k, w, rope, pos, gen = norm_case(dtype, D, Hq, Hkv, kw, B, S, 9, weight)
    gq = randn(gen, B, S, Hq, D, dtype=q.dtype).transpose(1, 2)
    gk = randn(gen, B, Hkv, S, D, dtype=q.dtype)
    dq, dk, dwq, dwk = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], 1e-5, rope, positions=pos)
    p = pos.cpu().numpy()[:, None]
    for x, g, wt, dx, dw in ((q, gq, w[0], dq, dwq), (k, gk, w[1], dk, dwk)):
        x, g, wt = np64(x), np64(g), None if wt is None else np64(wt)
        want, want_w = oracle.norm_rope_backward(g, x, wt, 1e-5, p, **spec(rope))
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        n, dz = np.abs(x * r), mixed(g, rope)
        wdz = dz * (1.0 if wt is None else np.abs(wt))
        close(dx, want, 64 * STEP * r * (wdz + n * (wdz * n).mean(-1, keepdims=True)))
        # every lane adds its rows one by one (fewer than 64 here), then 40 sums of sums
        terms = (dz * n).reshape(-1, D).sum(0)
        close(dw, want_w, (64 + 64 + 40) * STEP * terms)
    again = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], 1e-5, rope, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))
    a, b = gq.contiguous(), gk.clone()                    # in the gradients' places
    kvp.kvp_qk_norm_rope_backward(a, b, q, k, w[0], w[1], 1e-5, rope, positions=pos, dq=a, dk=b)
    assert torch.equal(a, dq) and torch.equal(b, dk)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,S", [("f32", 64, 2, 1, 9001), ("bf16", 128, 1, 1, 4501)])
def test_more_tokens_than_run_at_once(dtype, D, Hq, Hkv, S):
    q, k, w, rope, pos, gen = norm_case(dtype, D, Hq, Hkv, dict(rotary_dim=D), 3, S, 4)
    outs = kvp.kvp_qk_norm_rope(q, k, w[0], w[1], 1e-5, rope, positions=pos)
    gq, gk = randn(gen, *q.shape, dtype=q.dtype), randn(gen, *k.shape, dtype=q.dtype)
    grads = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], 1e-5, rope, positions=pos)
    turned = kvp.kvp_rope(q, rope, positions=pos)
    p = pos.cpu().numpy()[:, None]
    close(turned, oracle.rotate(np64(q), p, **spec(rope)), 8 * STEP * mixed(np64(q), rope))
    for x, g, wt, y, dx, dw in ((q, gq, w[0], outs[0], grads[0], grads[2]), (k, gk, w[1], outs[1], grads[1], grads[3])):
        x, g, wt = np64(x), np64(g), np64(wt)
        close(y, oracle.norm_rope(x, wt, 1e-5, p, **spec(rope)), 24 * STEP * mixed(oracle.norm_rope(x, wt, 1e-5), rope))
        want, want_w = oracle.norm_rope_backward(g, x, wt, 1e-5, p, **spec(rope))
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        n, dz = np.abs(x * r), mixed(g, rope)
        wdz = dz * np.abs(wt)
        close(dx, want, 64 * STEP * r * (wdz + n * (wdz * n).mean(-1, keepdims=True)))
        close(dw, want_w, (64 + 64 + 40) * STEP * (dz * n).reshape(-1, D).sum(0))


def test_gradient_matches_differences():
    q, k, w, rope, pos, gen = norm_case("f32", 64, 2, 1, dict(rotary_dim=32), 1, 3)
    q, k = q.contiguous() / 3, k.contiguous() / 3
    gq, gk = randn(gen, 1, 2, 3, 64, dtype=torch.float32), randn(gen, 1, 1, 3, 64, dtype=torch.float32)
    dq, dk, dwq, dwk = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, w[0], w[1], 1e-5, rope, positions=pos)

    def loss(q, k, w):
        a, b = kvp.kvp_qk_norm_rope(q, k, w[0], w[1], 1e-5, rope, positions=pos)
        return float((a.double() * gq).sum() + (b.double() * gk).sum())
    h = 2.0 ** -7
    for t, d in ((q, dq), (k, dk), (w[0], dwq), (w[1], dwk)):
        flat, grad = t.view(-1), d.reshape(-1)
        for i in (0, 17, flat.numel() - 1):
            x = float(flat[i])
            flat[i] = x + h
            up = loss(q, k, w)
            flat[i] = x - h
            down = loss(q, k, w)
            flat[i] = x
            # the loss's roundings (some 600 terms of up to 10, 2^-22 of each, over 2h: below 2e-2 together), and a
            # third derivative times h^2 / 6
            assert abs((up - down) / (2 * h) - float(grad[i])) < 2e-2


def test_zero_rows_and_no_eps():
    q = torch.zeros(1, 2, 3, 64, device="cuda")
    q[0, 0, 0] = 1.0
    y, _ = kvp.kvp_qk_norm_rope(q, q.clone(), None, None, 1e-6)
    assert torch.isfinite(y).all() and (y[0, 1] == 0).all()
    y, _ = kvp.kvp_qk_norm_rope(q, q.clone(), None, None, 0.0)
    assert (y[0, 0, 0] == 1).all() and torch.isnan(y[0, 1]).all()


def test_streams_and_graphs():
    q, k, w, rope, pos, gen = norm_case("bf16", 128, 8, 2, dict(rotary_dim=128), 2, 65)
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    want = kvp.kvp_qk_norm_rope(q, k, *w, 1e-6, rope, positions=pos)
    want_b = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, *w, 1e-6, rope, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvp.kvp_qk_norm_rope(q, k, *w, 1e-6, rope, positions=pos, stream=side)
    got_b = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, *w, 1e-6, rope, positions=pos, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + want_b, got + got_b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kvp.kvp_qk_norm_rope(q, k, *w, 1e-6, rope, positions=pos)
        got_b = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, *w, 1e-6, rope, positions=pos)
        turned = kvp.kvp_rope(q, rope, positions=pos)
    q.mul_(0.5)
    pos.add_(3)
    want = kvp.kvp_qk_norm_rope(q, k, *w, 1e-6, rope, positions=pos)
    want_b = kvp.kvp_qk_norm_rope_backward(gq, gk, q, k, *w, 1e-6, rope, positions=pos)
    for _ in range(2):
        g.replay()
    assert all(torch.equal(a, b) for a, b in zip(want + want_b, got + got_b))
    assert torch.equal(turned, kvp.kvp_rope(q, rope, positions=pos))


def test_offsets_past_32_bits():
    """Heads more than 2^31 elements apart."""
    D, S = 64, 3
    far = 2 ** 31 + 64
    buf = torch.empty(far + S * D, dtype=torch.float16, device="cuda")
    x = buf.as_strided((1, 2, S, D), (0, far, D, 1))
    x.copy_(torch.randn(1, 2, S, D, device="cuda"))
    rope = kvp.Rope(64)
    want = kvp.kvp_rope(x.contiguous(), rope, start=9)
    assert torch.equal(kvp.kvp_rope(x, rope, start=9), want)
    kvp.kvp_rope(x, rope, start=9, out=x)
    assert torch.equal(x, want)


def test_refusals():
    rope = kvp.Rope(64)
    x = torch.zeros(2, 4, 8, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    bad = [(TypeError, lambda: kvp.kvp_rope(x, None)), (TypeError, lambda: kvp.kvp_rope([1], rope)),
           (TypeError, lambda: kvp.kvp_rope(x, [1.0])),
           (ValueError, lambda: kvp.kvp_rope(x[0, 0], rope)), (ValueError, lambda: kvp.kvp_rope(x.long(), rope)),
           (ValueError, lambda: kvp.kvp_rope(x.transpose(2, 3), rope)), (ValueError, lambda: kvp.kvp_rope(x, rope, positions=pos.long())),
           (ValueError, lambda: kvp.kvp_rope(x, rope, positions=pos[:, :7])), (ValueError, lambda: kvp.kvp_rope(x, rope, positions=pos.cpu())),
           (ValueError, lambda: kvp.kvp_rope(x, rope, positions=pos.T.contiguous().T)),
           (ValueError, lambda: kvp.kvp_rope(x, rope, out=x[:, :3])), (ValueError, lambda: kvp.kvp_rope(x, rope, out=x.float())),
           (kvp.KvpError, lambda: kvp.kvp_rope(x, kvp.Rope(128))), (kvp.KvpError, lambda: kvp.kvp_rope(x, rope, out=x[:1].expand_as(x))),
           (kvp.KvpError, lambda: kvp.kvp_rope(x, rope, start=2 ** 31 - 2)),
           (kvp.KvpError, lambda: kvp.kvp_rope(x.view(-1)[4:4 + 4 * 64 * 8].view(1, 4, 8, 64), rope)),
           (ValueError, lambda: kvp.kvp_qk_norm_rope(x, x.float())), (TypeError, lambda: kvp.kvp_qk_norm_rope(x, None)),
           (ValueError, lambda: kvp.kvp_qk_norm_rope(x, x[:1])),
           (ValueError, lambda: kvp.kvp_qk_norm_rope(x, x, torch.ones(32, device="cuda"))),
           (ValueError, lambda: kvp.kvp_qk_norm_rope(x, x, torch.ones(64, device="cuda").half())),
           (ValueError, lambda: kvp.kvp_qk_norm_rope(x, x, torch.ones(64, device="cuda"), x.new_ones(64))),
           (kvp.KvpError, lambda: kvp.kvp_qk_norm_rope(x, x, eps=-1.0)),
           (ValueError, lambda: kvp.kvp_qk_norm_rope_backward(x, x[:, :2], x, x)),
           (kvp.KvpError, lambda: kvp.kvp_qk_norm_rope_backward(x, x, x, x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()
