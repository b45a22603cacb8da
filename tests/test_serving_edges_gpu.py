"""The serving operators at their edges, on the GPU against 64-bit arithmetic."""
import math
import os

import numpy as np
import pytest
import torch

from helpers import ROOT, spa
from test_serving_gpu import (BF16, F32, I32, U, gen, make_cache, no_wait_ran_out, projected,  # noqa: F401
                              randn, run_evict)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ shared-prefix decode
def exact_decode(q, P, cache, lens, prefix=None):
    """Outputs and weights in 64 bits, and how far fp32 scores, probabilities and sums may be from
    them, key by key: a key counts by its own probability."""
    B, H, d = q.shape
    Hk, _, m = P.shape
    kc, mul, v = cache
    out = torch.zeros((B, H, v.shape[-1]), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    weights = torch.zeros(kc.shape[:3], dtype=torch.float64, device="cuda")
    wtol = torch.zeros_like(weights)
    lens = lens.tolist()
    for b in range(B):
        for h in range(H):
            hk, n = h // (H // Hk), lens[b]
            K = kc[b, hk, :n].view(torch.float16).double() * mul[b, hk, :n, None].double()
            V = v[b, hk, :n].double()
            if prefix is not None:
                K = torch.cat((prefix[0][hk].view(torch.float16).double() * prefix[1][hk, :, None].double(), K))
                V = torch.cat((prefix[2][hk].double(), V))
            if len(K) == 0:
                continue
            s = (q[b, h].double() @ P[hk].double()) @ K.T / math.sqrt(m)
            p = torch.softmax(s, -1)
            mag = q[b, h].double().abs() @ P[hk].double().abs()
            # a score: d and m fp32 products and sums, counted as 2(d + m) + 8 roundings of the sum of
            # magnitudes; the query in 22 bits of its largest entry (2^-23 each); the key's entries to
            # 2^-24 of its largest; four roundings on the way to its exponential
            off = (mag @ K.abs().T * (2 * d + 2 * m + 8) * 2.0 ** -24 +
                   mag.max() * (K.abs().sum(-1) * 2.0 ** -23 + m * K.abs().amax(-1) * 2.0 ** -24)) / math.sqrt(m)
            rel = torch.expm1(torch.clamp(off, max=1.0)) + 4 * 2.0 ** -24 * (s.abs() + s.max().abs()) + 2.0 ** -20
            all_ = (p * rel).sum()
            # probabilities in two bf16 parts (2^-16), on the prefix kernel in one (2^-8); sums of 16
            # products each
            one = torch.full_like(p, 2.0 ** -16)
            one[:len(K) if H // Hk > 32 else len(K) - n] = 2.0 ** -8
            out[b, h] = p @ V
            tol[b, h] = (p * (rel + one)) @ V.abs() + (all_ + (len(K) / 16 + 64) * 2.0 ** -23) * (p @ V.abs())
            weights[b, hk, :n] += p[len(K) - n:]
            wtol[b, hk, :n] += (p * (rel + all_ + (len(K) / 16 + 64) * 2.0 ** -23))[len(K) - n:]
    return out, 1.01 * tol, weights, 1.01 * wtol


def check_exact(pkg, q, P, cache, lens, prefix=None, weights=True):
    acc = torch.zeros(cache[1].shape, device="cuda") if weights else None
    got = pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, acc=acc)
    out, tol, want, wtol = exact_decode(q, P, cache, lens, prefix)
    over = (got.double() - out).abs() - (U[BF16] * (out.abs() + tol) + tol + 1e-30)
    assert float(over.max()) <= 0, f"{float(over.max())} over, of {float(out.abs().max())}"
    if weights and acc.numel():
        inside = torch.arange(acc.shape[2], device="cuda")[None, None] < lens[:, None, None]
        over = (acc.double() - want).abs() - wtol - 4 * q.shape[1] / P.shape[0] * U[F32] * want - 1e-30
        assert float(over[inside.expand_as(over)].amax() if bool(inside.any()) else 0) <= 0
    return got


@pytest.mark.parametrize("shape", [
    # B, H, Hk, d, m, dv, lens: few keys, so that each one's probability shows
    (3, 4, 2, 64, 32, 64, [40, 7, 1]),
    (16, 8, 8, 64, 16, 64, [5 + i for i in range(16)]),
    (4, 8, 1, 128, 64, 128, [24, 3, 17, 30]),
    (8, 4, 4, 128, 128, 128, [17, 5] * 4),
    (3, 32, 1, 64, 32, 128, [33, 9, 4]),
])
def test_decode_probabilities_keep_their_bits(shape):
    """On the sequences' own rows an output is off by its own rounding alone, not by the
    probabilities'."""
    pkg = spa()
    B, H, Hk, d, m, dv, lens = shape
    g = gen(B + H + m)
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, 40, m=m, dv=dv, d=d)
    check_exact(pkg, q, P, cache, torch.tensor(lens, dtype=I32, device="cuda"))


def rows_of(x):
    """Rows as the appends write them: fp16 bits and a power of two, 1 for a row of zeros."""
    top = x.abs().amax(-1)
    mul = torch.where(top > 0, torch.exp2((torch.frexp(top)[1] - 14).double()), torch.ones_like(top))
    return (x / mul[..., None]).to(torch.float16).view(torch.int16), mul.float()


@pytest.mark.parametrize("kind", ["zero rows", "a far larger row", "all kinds"])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("m", [16, 32, 64, 128])
def test_decode_keys_of_other_magnitudes_in_a_tile(m, own, kind):
    """Small keys keep their scores beside rows of zeros (multiplier 1) and beside rows 2^25 as
    large: in the prefix, and in the own rows of a group that runs on the prefix kernel."""
    pkg = spa()
    g = gen(m + own)
    B, H, Hk, d, dv, n = (1, 40, 1, 64, 64, 300) if own else (3, 8, 2, 64, 64, 300)
    # queries of 2^14 against keys of 2^-14: scores of a few units
    one = randn(g, 1, 1, d)
    q = ((one + 0.3 * randn(g, B, H, d)) * 2.0 ** 14).to(BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    x = torch.randn((Hk, n, m), generator=g, device="cuda", dtype=torch.float64) * math.sqrt(d / m) * 2.0 ** -14
    if kind == "all kinds":  # and rows down to 2^-30 of that: any factor within a tile
        x[:, 140:] *= torch.exp2(-torch.randint(0, 31, (Hk, n - 140, 1), generator=g, device="cuda").double())
    if kind != "a far larger row":
        x[:, [3, 130, n - 1]] = 0
    if kind != "zero rows":  # against all queries: its own probability is 0
        far = torch.einsum("d,hdm->hm", one[0, 0].double(), P.double())
        x[:, 17] = -2.0 ** 11 * far
    kc, mul = rows_of(x)
    v = randn(g, Hk, n, dv, dtype=BF16)
    if own:
        cache, prefix = (kc[None], mul[None], v[None]), None
        lens = torch.tensor([n], dtype=I32, device="cuda")
    else:
        cache = make_cache(g, B, Hk, 8, m=m, dv=dv, d=d)
        cache[1].mul_(2.0 ** -14)
        prefix, lens = (kc, mul, v), torch.tensor([8, 0, 5], dtype=I32, device="cuda")
    check_exact(pkg, q, P, cache, lens, prefix)


@pytest.mark.parametrize("m", [16, 64, 128])
def test_decode_many_tiles_with_and_without_one_range(m):
    """Some twenty tiles one behind the other on every SM, at random with a row of zeros or without:
    each key's weight is that of its own multiplier."""
    pkg = spa()
    g = gen(110 + m)
    B, H, Hk, d, dv, n = 1, 40, 1, 64, 64, 400000
    q = (randn(g, B, H, d) * 2.0 ** 14).to(BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    x = torch.randn((Hk, n, m), generator=g, device="cuda", dtype=torch.float64) * math.sqrt(d / m) * 2.0 ** -14
    x *= torch.exp2(-torch.randint(0, 3, (Hk, n, 1), generator=g, device="cuda").double())
    wide = torch.nonzero(torch.rand(n // 128, generator=g, device="cuda") < 0.5)[:, 0]
    x[:, wide * 128 + torch.randint(0, 128, wide.shape, generator=g, device="cuda")] = 0
    kc, mul = rows_of(x)
    del x
    check_exact(pkg, q, P, (kc[None], mul[None], randn(g, B, Hk, n, dv, dtype=BF16)),
                torch.tensor([n - 5], dtype=I32, device="cuda"))


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("m", [16, 64, 128])
def test_decode_scores_that_grow_along_the_keys(m, own):
    """Later tiles of the prefix kernel move a row's maximum: its sums follow."""
    pkg = spa()
    g = gen(60 + m)
    B, H, Hk, d, dv, n = (1, 40, 1, 64, 128, 1500) if own else (3, 8, 2, 64, 128, 1500)
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    x = torch.randn((Hk, n, m), generator=g, device="cuda", dtype=torch.float64) * math.sqrt(d / m)
    x *= torch.exp2(torch.arange(n, device="cuda").double()[:, None] // 250)  # up to 2^5
    kc, mul = rows_of(x)
    v = randn(g, Hk, n, dv, dtype=BF16)
    if own:
        cache, prefix = (kc[None], mul[None], v[None]), None
        lens = torch.tensor([n], dtype=I32, device="cuda")
    else:
        cache = make_cache(g, B, Hk, 20, m=m, dv=dv, d=d)
        prefix, lens = (kc, mul, v), torch.tensor([20, 0, 5], dtype=I32, device="cuda")
    check_exact(pkg, q, P, cache, lens, prefix)


def test_decode_long_own_caches():
    """Own caches of 131072 and 32769 rows, and of one."""
    pkg = spa()
    g = gen(70)
    B, H, Hk, d, m, dv, cap = 3, 4, 2, 128, 32, 128, 131072
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    check_exact(pkg, q, P, cache, torch.tensor([cap, 32769, 1], dtype=I32, device="cuda"))


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("cap", [380000, 1 << 20])
def test_evict_longest_caches(cap):
    """A bit per row in shared memory: 46 to 128 KB, with the kernel's own beside it."""
    pkg = spa()
    g = gen(cap)
    acc = torch.floor(torch.rand((1, 1, cap), generator=g, device="cuda") * 5000)
    row_pos = torch.argsort(torch.rand((1, 1, cap), generator=g, device="cuda"), dim=-1).to(I32)
    run_evict(pkg, g, 1, 1, 16, 64, cap, cap - 5000, 4, 300, [cap - 1], acc, row_pos, True)


def test_decode_one_workspace_with_changing_queries_and_lengths():
    """Calls one behind the other on one workspace, without a pause: each sees the queries and
    lengths of its own call."""
    pkg = spa()
    g = gen(80)
    B, H, Hk, d, m, dv, cap, plen, calls = 24, 8, 2, 64, 32, 64, 700, 3000, 60
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache, prefix = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d), make_cache(g, Hk, plen, m=m, dv=dv, d=d)
    ws = torch.empty(pkg.spa_attention_decode_shared_workspace_size(B, H, Hk, plen, d, m, dv, cap),
                     dtype=torch.uint8, device="cuda")
    qs = randn(g, calls, B, H, d, dtype=BF16)
    lens = torch.randint(0, cap + 1, (calls, B), generator=g, device="cuda", dtype=I32)
    outs = torch.empty((calls, B, H, dv), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    for i in range(calls):
        pkg.spa_attention_decode_shared(qs[i], P, *cache, lens[i], prefix=prefix, out=outs[i], workspace=ws)
    torch.cuda.synchronize()
    for i in range(calls):
        want = pkg.spa_attention_decode_shared(qs[i], P, *cache, lens[i], prefix=prefix)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want), i


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_angle(interleaved):
    """The angle to 2^-32 of a turn: near half turns, where the sine shows it."""
    pkg = spa()
    g = gen(90)
    d, N = 64, 8192
    table = pkg.rope_table(pkg.rope_frequencies(d))
    pos = torch.randint(-(1 << 20), 1 << 20, (1, N), generator=g, device="cuda", dtype=I32)
    x = torch.zeros((1, 1, N, d), device="cuda")
    a, b = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    x[..., a] = 1.0
    y = pkg.spa_rope(x, table, pos, interleaved=interleaved)
    # the table's fraction of a turn, in wrapping 64-bit integers as the entry says
    turn = pos[0, :, None].to(torch.int64) * table
    angle = turn.double() * (2 * math.pi * 2.0 ** -64)
    # 2 pi 2^-32 for the angle, the sine and cosine to 2 steps of fp32
    for got, want in ((y[0, 0][:, a], torch.cos(angle)), (y[0, 0][:, b], torch.sin(angle))):
        assert bool(((got.double() - want).abs() <= 2 * math.pi * 2.0 ** -32 + 4 * U[F32] * want.abs()).all())


# ------------------------------------------------------------------ ragged append
@pytest.mark.parametrize("terms", [16, 60])
@pytest.mark.parametrize("d", [256, 200])
def test_append_multiplier_of_cancelling_sums(d, terms):
    """Row maxima just beside a power of two, to which d terms of up to 60 times that in all cancel."""
    pkg = spa()
    g = torch.Generator().manual_seed(d)
    m, T = 32, 400
    n = d // 2 - 2
    r = torch.rand((T, n), generator=g, dtype=torch.float64) + 0.5
    r *= torch.exp2(-torch.randint(0, 16, (T, n), generator=g).double())  # so that fp32 sums round
    r = (r * ((terms - 1.2) / 2 / r.sum(-1, keepdim=True))).to(BF16).double()
    k = torch.zeros((T, d), dtype=torch.float64)
    k[:, 2:n + 2], k[:, n + 2:2 * n + 2] = r, -r                  # sums grow first and shrink then
    k[:, 0] = 1.0
    k[:, 1] = torch.exp2(-(torch.arange(T) % 12) - 15.0) * torch.where(torch.rand(T, generator=g) < 0.5, 1.0, -1.0)
    k = k.to(BF16)[None, None].cuda()
    P = torch.zeros((1, d, m), device="cuda", dtype=BF16)
    P[0, :, 5] = 1.0
    kc, mul = pkg.kcache_new(1, 1, T, m)
    vc = torch.zeros((1, 1, T, 64), dtype=BF16, device="cuda")
    pkg.spa_kcache_append_ragged(k, vc.clone(), P, kc, mul, vc, torch.zeros(1, dtype=I32, device="cuda"))
    x, want, mag = projected(k, P)
    assert float((mag.amax(-1) / x.abs().amax(-1)).max()) < 1.01 * terms
    assert torch.equal(mul.double(), want)


# ------------------------------------------------------------------ the README's step
def test_readme_decode_steps():
    """The README's loop: every new row has a position of its own, the next one."""
    pkg = spa()
    text = open(os.path.join(ROOT, "README.md")).read()
    code = next(c for c in text.split("```python\n")[1:] if "spa_rope" in c).split("```")[0]
    g = gen(99)
    B, H, Hk, d, m, dv, cap, plen, n = 2, 4, 2, 64, 32, 64, 300, 50, 5
    kc, kc_mul, vc = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    names = dict(d=d, P=(randn(g, Hk, d, m) / math.sqrt(m)).to(BF16), kc=kc, kc_mul=kc_mul, vc=vc, budget=256,
                 prefix=make_cache(g, Hk, plen, m=m, dv=dv, d=d), acc=torch.zeros((B, Hk, cap), device="cuda"),
                 row_pos=torch.zeros((B, Hk, cap), dtype=I32, device="cuda"),
                 lens=torch.zeros(B, dtype=I32, device="cuda"), pos=torch.tensor([plen, plen + 7], dtype=I32, device="cuda"),
                 steps=[[randn(g, B, h, 1, c, dtype=BF16) for h, c in ((H, d), (Hk, d), (Hk, dv))] for _ in range(n)])
    exec(code, names)
    assert names["lens"].tolist() == [n, n]
    for b, first in enumerate((plen, plen + 7)):
        for h in range(Hk):
            assert names["row_pos"][b, h, :n].tolist() == list(range(first, first + n))
    assert bool(torch.isfinite(names["out"]).all())


# ------------------------------------------------------------------ accumulated weights
@pytest.mark.parametrize("shape", [
    # B, H, Hk, d, m, plen: many queries, so that the errors' mean does not hang on a few of them
    (64, 8, 8, 128, 16, 0),
    (100, 16, 4, 200, 32, 0),
    (64, 32, 4, 128, 32, 300),
])
def test_decode_weights_are_as_near_as_plain_fp32(shape):
    """Weights of large scores: as near to 64 bits, in the mean, as fp32 arithmetic on fp32 scores."""
    pkg = spa()
    B, H, Hk, d, m, plen = shape
    g = gen(B + m)
    cap, dv, G = 48, 64, H // Hk
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    prefix = make_cache(g, Hk, plen, m=m, dv=dv, d=d) if plen else None
    acc = torch.zeros((B, Hk, cap), device="cuda")
    pkg.spa_attention_decode_shared(q, P, *cache, torch.full((B,), cap, dtype=I32, device="cuda"), prefix=prefix, acc=acc)

    def plain(t):
        qt = torch.matmul(q.to(t).view(B, Hk, G, d), P.to(t)) / math.sqrt(m)
        s = torch.matmul(qt, (cache[0].view(torch.float16).to(t) * cache[1].to(t)[..., None]).transpose(-1, -2))
        if plen:
            k = (prefix[0].view(torch.float16).to(t) * prefix[1].to(t)[..., None]).transpose(-1, -2)
            s = torch.cat((s, torch.matmul(qt, k)), dim=-1)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        return (e / e.sum(-1, keepdim=True)).sum(2)[..., :cap]

    want = plain(torch.float64)
    own, fp32 = (float((x.double() - want).norm() / want.norm()) for x in (acc, plain(torch.float32)))
    # a quarter more at most: both round each score at its size and a probability a few times
    assert own <= 1.25 * fp32, (own, fp32)
