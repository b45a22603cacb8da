"""The serving operators on the GPU against plain 64-bit implementations: rotary
positions, ragged append, shared-prefix decode with weights, eviction, and a
decode loop of all of them."""
import math
import threading
import time

import numpy as np
import pytest
import torch

from helpers import spa

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = {BF16: 2.0 ** -8, torch.float16: 2.0 ** -11, F32: 2.0 ** -24}  # half a step


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert spa().device_error() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ rotary positions
def rope_ref(x, freq, pos, interleaved, inverse, scale):
    """64 bits; also the bound |a| + |b| of each rotated feature."""
    x = x.double()
    rot = 2 * freq.numel()
    ang = pos.double()[:, None, :, None] * freq.to(x.device)
    c, s = torch.cos(ang), torch.sin(ang) * (-1 if inverse else 1)
    y, bound = x.clone(), torch.zeros_like(x)
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = scale * (a * c - b * s)
    y[..., ib] = scale * (a * s + b * c)
    bound[..., ia] = bound[..., ib] = abs(scale) * (a.abs() + b.abs())
    return y, bound


def check_rope(got, x, freq, pos, interleaved, inverse=False, scale=1.0, angle=0.0):
    ref, bound = rope_ref(x, freq, pos, interleaved, inverse, scale)
    # rounding of the result; the angle to 2^-25 of a half turn (pi 2^-25), the sine to two
    # steps (2^-22), two products, a sum and the scale (4 x 2^-24): below 2^-20 of |a| + |b|
    tol = U[got.dtype] * ref.abs() + (2.0 ** -20 + angle) * bound + 1e-30
    assert bool(((got.double() - ref).abs() <= tol).all()), float(((got.double() - ref).abs() - tol).max())


ROPE = [
    # B, H, Hk, N, d, rot
    (1, 1, 0, 1, 2, 2),
    (2, 3, 1, 5, 64, 64),
    (3, 4, 2, 7, 96, 38),      # a half of 19 features
    (1, 5, 5, 33, 80, 80),
    (2, 2, 1, 9, 33, 20),      # an odd width
    (1, 8, 2, 130, 128, 64),
    (2, 1, 1, 3, 1024, 1024),
    (64, 32, 8, 1, 128, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ROPE)
def test_rope(shape, interleaved, dtype):
    pkg = spa()
    B, H, Hk, N, d, rot = shape
    g = gen(N * d + rot)
    freq = pkg.rope_frequencies(rot)
    table = pkg.rope_table(freq)
    q, k = randn(g, B, H, N, d, dtype=dtype), randn(g, B, Hk, N, d, dtype=dtype)
    pos = torch.randint(-5, 1 << 20, (B, N), generator=g, device="cuda", dtype=I32)
    if Hk:
        a, b = pkg.spa_rope(q, table, pos, k=k, interleaved=interleaved, scale=1.25)
        check_rope(b, k, freq, pos, interleaved, scale=1.25)
    else:
        a = pkg.spa_rope(q, table, pos, interleaved=interleaved, scale=1.25)
    check_rope(a, q, freq, pos, interleaved, scale=1.25)
    assert torch.equal(a[..., rot:], q[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_in_place_and_broadcast(interleaved):
    pkg = spa()
    g = gen(3)
    B, H, Hk, N, d = 2, 4, 2, 37, 64
    freq = pkg.rope_frequencies(d, scaling=pkg.SPA_ROPE_LINEAR, factor=8.0)
    table = pkg.rope_table(freq)
    pos = torch.arange(N, device="cuda", dtype=I32).expand(B, N).contiguous() + 11
    x = randn(g, B, N, H + 2 * Hk, d, dtype=BF16)           # token-major, with values behind
    keep = x.clone()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    a, b = pkg.spa_rope(q, table, k=k, pos0=11, interleaved=interleaved)
    check_rope(a, q, freq, pos, interleaved)
    check_rope(b, k, freq, pos, interleaved)
    # in place, strided: the same bits, and nothing else is touched
    pkg.spa_rope(q, table, pos, k=k, interleaved=interleaved, out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(x[:, :, H + Hk:], keep[:, :, H + Hk:])
    # an offset that only allows single features; one row for all sequences (stride 0)
    y = randn(g, 1, H, N, d + 1, dtype=BF16)[..., 1:].expand(B, H, N, d)
    check_rope(pkg.spa_rope(y, table, pos, interleaved=interleaved), y, freq, pos, interleaved)
    with pytest.raises(pkg.SpaError):
        pkg.spa_rope(y, table, pos, out=y)                   # sequences that share an output row
    with pytest.raises(ValueError):
        pkg.spa_rope(x.transpose(2, 3)[:, :, :, :N], table, pos)


def test_rope_far_positions():
    pkg = spa()
    g = gen(4)
    freq = pkg.rope_frequencies(64)
    pos = torch.tensor([[0, 1, -1, 2**31 - 1, -2**31, 2**30 + 1, 10**9 + 7]], device="cuda", dtype=I32)
    x = randn(g, 1, 2, 7, 64)
    got = pkg.spa_rope(x, pkg.rope_table(freq), pos)
    # 2^31 rad: the reference's own product is off by 2^-53 of it, the table by the rounding of f / 2pi
    # and of 2pi (2^-53 each)
    check_rope(got, x, freq, pos, False, angle=3 * 2.0 ** 31 * 2.0 ** -53)
    assert torch.equal(got[:, :, 0], x[:, :, 0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    pkg = spa()
    g = gen(5)
    B, H, N, d, rot = 1, 2, 6, 20, 12
    freq = pkg.rope_frequencies(rot)
    table = pkg.rope_table(freq)
    pos = torch.randint(0, 5000, (B, N), generator=g, device="cuda", dtype=I32)
    x, dy = randn(g, B, H, N, d), randn(g, B, H, N, d)
    dx = pkg.spa_rope(dy, table, pos, interleaved=interleaved, inverse=True, scale=0.75)
    # the formula's: the transposed rotation
    check_rope(dx, dy, freq, pos, interleaved, inverse=True, scale=0.75)
    dx_tail, dy_tail = dx[..., rot:], dy[..., rot:]
    assert torch.equal(dx_tail, dy_tail)
    # differences of <rope(x), dy>, which is linear in x: step 1, each feature in turn
    def f(z):
        return (pkg.spa_rope(z, table, pos, interleaved=interleaved, scale=0.75).double() * dy.double())
    for c in range(d):
        e = torch.zeros_like(x)
        e[..., c] = 0.5
        diff = (f(x + e) - f(x - e)).sum(-1)
        # 2d terms of about 1, each off by fp32 roundings (2^-22 of |x| + 1/2 < 6, times |dy| < 6)
        assert float((diff - dx[..., c].double()).abs().max()) <= 2 * d * 2.0 ** -22 * 36


# ------------------------------------------------------------------ ragged append
def projected(k, P):
    """K~ in 64 bits, the multipliers of the row maxima, and the sums of magnitudes."""
    x = torch.einsum("bhtd,hdm->bhtm", k.double(), P.double())
    mag = torch.einsum("bhtd,hdm->bhtm", k.double().abs(), P.double().abs())
    top = x.abs().amax(-1)
    e = torch.frexp(top)[1] - 14
    mul = torch.where(top > 0, torch.exp2(e.double()), torch.ones_like(top))
    return x, mul, mag


APPEND = [
    # B, H, T, d, m, dv, cap
    (1, 1, 1, 1, 16, 64, 1),
    (5, 2, 1, 64, 32, 128, 20),
    (3, 3, 17, 100, 64, 64, 40),   # a width that is no multiple of 8
    (2, 1, 33, 256, 128, 128, 33),
    (64, 8, 1, 128, 32, 128, 16),
    (2, 2, 300, 96, 16, 64, 301),
]


@pytest.mark.parametrize("shape", APPEND)
def test_append_ragged(shape):
    pkg = spa()
    B, H, T, d, m, dv, cap = shape
    g = gen(sum(shape))
    k, v = randn(g, B, H, T, d, dtype=BF16), randn(g, B, H, T, dv, dtype=BF16)
    P = (randn(g, H, d, m) / math.sqrt(m)).to(BF16)
    if T > 1:
        k[0, 0, 1] = 0                         # a row without a magnitude
    kc = torch.full((B, H, cap, m), 77, dtype=torch.int16, device="cuda")
    mul, acc = torch.full((B, H, cap), 7.0, device="cuda"), torch.full((B, H, cap), 7.0, device="cuda")
    vc = torch.full((B, H, cap, dv), 7.0, dtype=BF16, device="cuda")
    row_pos = torch.full((B, H, cap), 7, dtype=I32, device="cuda")
    pos = torch.randint(0, cap - T + 1, (B,), generator=g, device="cuda", dtype=I32)
    count = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=I32)
    count[-1] = T
    token = pos + 1000
    pkg.spa_kcache_append_ragged(k, v, P, kc, mul, vc, pos, count, acc, row_pos, token)
    x, want_mul, mag = projected(k, P)
    fresh = torch.zeros((B, cap), dtype=torch.bool)
    for b in range(B):
        p, n = int(pos[b]), int(count[b])
        fresh[b, p:p + n] = True
        rows = kc[b, :, p:p + n].view(torch.float16).double()
        assert torch.equal(mul[b, :, p:p + n].double(), want_mul[b, :, :n])
        # fp16 rounding (2^-11, at least 2^-25 of the scaled unit) and d fp32 products and sums,
        # counted as 2d roundings
        scaled = want_mul[b, :, :n, None]
        tol = U[torch.float16] * x[b, :, :n].abs() + 2.0 ** -25 * scaled + 2 * d * U[F32] * mag[b, :, :n]
        assert bool(((rows * scaled - x[b, :, :n]).abs() <= 1.001 * tol).all())
        assert torch.equal(vc[b, :, p:p + n], v[b, :, :n])
        assert bool((acc[b, :, p:p + n] == 0).all())
        want = torch.arange(n, device="cuda", dtype=I32) + token[b]
        assert torch.equal(row_pos[b, :, p:p + n], want.expand(H, n))
    old = ~fresh.cuda()[:, None].expand(B, H, cap)
    assert bool((kc[old] == 77).all()) and bool((vc[old] == 7).all()) and bool((mul[old] == 7).all())
    assert bool((acc[old] == 7).all()) and bool((row_pos[old] == 7).all())


def test_append_rows_outside_the_cache_are_not_written():
    pkg = spa()
    g = gen(8)
    B, H, T, d, m, dv, cap = 4, 1, 6, 64, 32, 64, 8
    k, v, P = randn(g, B, H, T, d, dtype=BF16), randn(g, B, H, T, dv, dtype=BF16), randn(g, H, d, m, dtype=BF16)
    # one more sequence in front and behind takes what would run over
    kc, mul, vc = (torch.zeros((B + 2, H, cap, *s), dtype=t, device="cuda")
                   for s, t in (((m,), torch.int16), ((), F32), ((dv,), BF16)))
    pos = torch.tensor([-3, 5, 8, 2**31 - 2], device="cuda", dtype=I32)
    count = torch.tensor([6, 100, 6, 6], device="cuda", dtype=I32)
    pkg.spa_kcache_append_ragged(k, v, P, kc[1:-1], mul[1:-1], vc[1:-1], pos, count)
    there = mul[:, 0] != 0
    want = torch.zeros((B + 2, cap), dtype=torch.bool, device="cuda")
    want[1, :3] = True
    want[2, 5:] = True
    assert torch.equal(there, want)
    assert torch.equal(vc[1, 0, :3], v[0, 0, 3:]) and torch.equal(vc[2, 0, 5:], v[1, 0, :3])
    assert bool((vc[~want[:, None]] == 0).all())


def test_append_from_two_threads():
    """Calls of two widths at the same time, on a stream each: one thread's launches
    do not take the shared memory from the other's."""
    pkg = spa()
    B, H, T, m, dv, cap = 2, 2, 33, 128, 64, 40
    pos = torch.zeros(B, dtype=I32, device="cuda")
    work, errors = [], []
    for i, d in enumerate((256, 33)):
        g = gen(91 + i)
        k, v = randn(g, B, H, T, d, dtype=BF16), randn(g, B, H, T, dv, dtype=BF16)
        P = (randn(g, H, d, m) / math.sqrt(m)).to(BF16)
        caches = [(torch.zeros((B, H, cap, m), dtype=torch.int16, device="cuda"),
                   torch.zeros((B, H, cap), device="cuda"),
                   torch.zeros((B, H, cap, dv), dtype=BF16, device="cuda")) for _ in range(2)]
        work.append((k, v, P, caches, torch.cuda.Stream()))
        pkg.spa_kcache_append_ragged(k, v, P, *caches[0], pos)
    torch.cuda.synchronize()

    def run(k, v, P, caches, stream):
        try:
            for _ in range(200):
                pkg.spa_kcache_append_ragged(k, v, P, *caches[1], pos, stream=stream)
        except Exception as e:  # told to the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for _, _, _, (a, b), _ in work:
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_append_multiplier_at_powers_of_two():
    """Row maxima on, just under and just over a power of two, by sums that fp32 rounds."""
    pkg = spa()
    d, m = 64, 32
    rows = []
    for tail in (0.0, 2.0 ** -30, -2.0 ** -30, 2.0 ** -26, -2.0 ** -26, 2.0 ** -18, -2.0 ** -18):
        r = torch.zeros(d)
        r[0], r[1], r[2], r[3] = 1.0, 3.0, tail, -2.0   # 2 + tail
        rows.append(r)
    k = torch.stack(rows)[None, None].to(BF16).cuda()
    P = torch.zeros((1, d, m), device="cuda", dtype=BF16)
    P[0, :, 5] = 1.0
    T = k.shape[2]
    kc, mul = pkg.kcache_new(1, 1, T, m)
    vc = torch.zeros((1, 1, T, 64), dtype=BF16, device="cuda")
    pkg.spa_kcache_append_ragged(k, vc.clone(), P, kc, mul, vc, torch.zeros(1, dtype=I32, device="cuda"))
    _, want, _ = projected(k, P)
    assert torch.equal(mul.double(), want)


@pytest.mark.parametrize("m", [16, 32, 64, 128])
def test_append_agrees_with_the_dense_append(m):
    pkg = spa()
    g = gen(m)
    B, H, T, d, cap = 2, 3, 150, 128, 160
    k, v = randn(g, B, H, T, d, dtype=BF16), randn(g, B, H, T, 64, dtype=BF16)
    P = (randn(g, H, d, m) / math.sqrt(m)).to(BF16)
    a, b = pkg.kcache_new(B, H, cap, m), pkg.kcache_new(B, H, cap, m)
    vc = torch.zeros((B, H, cap, 64), dtype=BF16, device="cuda")
    pkg.spa_kcache_append(k, P, *a, 7)
    pkg.spa_kcache_append_ragged(k, v, P, *b, vc, torch.full((B,), 7, dtype=I32, device="cuda"))
    x = a[0].view(torch.float16).double() * a[1].double()[..., None]
    y = b[0].view(torch.float16).double() * b[1].double()[..., None]
    _, _, mag = projected(k, P)
    # two roundings to fp16, one at a multiplier twice the other's, and twice the fp32 sums' error
    tol = 2 * U[torch.float16] * torch.maximum(x.abs(), y.abs())[:, :, 7:157] + 4 * d * U[F32] * mag + \
        2.0 ** -24 * torch.maximum(a[1], b[1]).double()[:, :, 7:157, None]
    assert bool(((x - y)[:, :, 7:157].abs() <= tol).all())


# ------------------------------------------------------------------ shared-prefix decode
def make_cache(g, *shape, m, dv, d):
    x = randn(g, *shape, m) * math.sqrt(d / m)
    e = torch.frexp(x.abs().amax(-1))[1] - 14
    mul = torch.exp2(e.float())
    return (x / mul[..., None]).to(torch.float16).view(torch.int16), mul, randn(g, *shape, dv, dtype=BF16)


def decode_ref(q, P, cache, lens, prefix, plen):
    """Outputs, the weights per key head, and their tolerances' parts, in 64 bits."""
    B, H, d = q.shape
    Hk, _, m = P.shape
    G = H // Hk
    kc, mul, v = cache
    out, mag, rel = (torch.zeros((B, H, n), dtype=torch.float64) for n in (v.shape[-1], v.shape[-1], 1))
    weights = torch.zeros(kc.shape[:3], dtype=torch.float64)
    for b in range(B):
        for h in range(H):
            hk, n = h // G, min(max(int(lens[b]), 0), kc.shape[2])
            keys = [kc[b, hk, :n].view(torch.float16).double() * mul[b, hk, :n, None].double()]
            vals = [v[b, hk, :n].double()]
            if plen:
                keys.insert(0, prefix[0][hk, :plen].view(torch.float16).double() * prefix[1][hk, :plen, None].double())
                vals.insert(0, prefix[2][hk, :plen].double())
            K, V = torch.cat(keys), torch.cat(vals)
            if len(K) == 0:
                continue
            qd, Pd = q[b, h].double(), P[hk].double()
            p = torch.softmax((qd @ Pd) @ K.T / math.sqrt(m), -1)
            out[b, h], mag[b, h] = p @ V, p @ V.abs()
            # the score of a key: d and m fp32 products and sums, counted as 2(d + m) + 8 roundings of
            # the sum of magnitudes; a probability is off by twice that, relatively
            off = (qd.abs() @ Pd.abs()) @ K.abs().T / math.sqrt(m) * (2 * d + 2 * m + 8) * 2.0 ** -24
            rel[b, h] = 2 * off.max() + 2.0 ** -18
            weights[b, hk, :n] += p[len(K) - n:].cpu()
    return out, weights, mag, rel


def check_decode(pkg, q, P, cache, lens, prefix=None, plen=None, acc=None, what="", **kw):
    before = None if acc is None else acc.double().cpu()
    got = pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, plen=plen, acc=acc, **kw)
    n = 0 if prefix is None else prefix[0].shape[1] if plen is None else plen
    out, weights, mag, rel = decode_ref(q, P, cache, lens, prefix, n)
    # the result's rounding, and the probabilities' (bf16 operands of the value product)
    tol = U[BF16] * out.abs() + (U[BF16] + rel) * 1.01 * mag + 1e-30
    diff = (got.double().cpu() - out).abs()
    assert bool((diff <= tol).all()), f"{what}: {float((diff - tol).max())}"
    if acc is not None:
        new = (kw.get("acc_out", None) if kw.get("acc_out", None) is not None else acc).double().cpu()
        G = q.shape[1] // P.shape[0]
        r = float(rel.max())
        inside = torch.arange(acc.shape[2])[None, :] < lens.cpu()[:, None]
        d = (new - before - weights).abs()
        ok = d <= (r + G * U[F32]) * weights + 2 * U[F32] * (before + weights) + 1e-30
        assert bool((ok | ~inside[:, None]).all()), what
    return got


DECODE = [
    # B, H, Hk, d, m, dv, cap, plen, lens
    (1, 1, 1, 64, 16, 64, 1, 0, [1]),
    (1, 1, 1, 64, 32, 64, 4, 1, [0]),
    (3, 4, 2, 100, 32, 128, 130, 0, [0, 1, 130]),             # an empty row of the batch
    (2, 8, 1, 128, 64, 128, 300, 129, [300, 127]),
    (5, 5, 1, 33, 128, 64, 200, 127, [0, 128, 129, 1, 200]),
    (4, 12, 4, 128, 16, 128, 700, 1000, [700, 640, 3, 257]),
    (33, 8, 2, 64, 32, 64, 64, 513, list(range(33))),         # more than 128 query rows per key head
    (40, 16, 1, 128, 32, 128, 20, 700, [20] * 40),            # 640 rows
    (2, 6, 3, 128, 64, 64, 5000, 0, [5000, 4097]),
    (1, 40, 1, 128, 128, 128, 600, 300, [555]),               # a group wider than a warp
    (1, 200, 1, 64, 32, 64, 300, 20, [290]),                  # a group wider than a tile
    # many segments for every CTA, of one tile and of many, over several key heads
    (16, 8, 4, 128, 32, 64, 3000, 0, [17 + 187 * i for i in range(16)]),
    (24, 16, 8, 64, 64, 128, 700, 9000, [(97 * i) % 701 for i in range(24)]),
    (40, 48, 4, 64, 16, 64, 520, 4000, [(131 * i) % 521 for i in range(40)]),   # and several row tiles
    (3, 8, 4, 64, 128, 128, 4000, 20000, [4000, 1, 129]),                       # a ring of two slots
    # many short sequences, without and with a prefix, and few warps' work for many
    (1300, 2, 1, 64, 16, 64, 40, 0, [(7 * i) % 41 for i in range(1300)]),
    (1100, 2, 2, 64, 32, 64, 24, 300, [(5 * i) % 25 for i in range(1100)]),
    (70, 4, 4, 64, 16, 64, 2000, 0, [0] * 69 + [2000]),
    (70, 4, 4, 64, 32, 64, 2000, 6000, [2000] + [0] * 69),
    # no rows of the sequences' own at all, with and without a prefix
    (3, 4, 2, 64, 32, 64, 0, 700, [0, 0, 0]),
    (2, 40, 1, 64, 32, 64, 0, 130, [0, 0]),
    (2, 4, 2, 64, 32, 64, 0, 0, [0, 0]),
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("shape", DECODE)
def test_decode_shared(shape, weights):
    pkg = spa()
    B, H, Hk, d, m, dv, cap, plen, lens = shape
    g = gen(B * cap + plen)
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    prefix = make_cache(g, Hk, plen, m=m, dv=dv, d=d) if plen else None
    lens = torch.tensor(lens, dtype=I32, device="cuda")
    # what lies behind a length may be anything
    for b in range(B):
        n = int(lens[b])
        cache[0][b, :, n:] = 0x7e00        # NaN in fp16
        cache[1][b, :, n:] = math.inf
        cache[2][b, :, n:] = math.nan
    acc = torch.rand((B, Hk, cap), generator=g, device="cuda") if weights else None
    ws = torch.empty(pkg.spa_attention_decode_shared_workspace_size(B, H, Hk, plen, d, m, dv, cap, weights),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)                          # NaN wherever it is read before it is written
    acc_out = torch.full_like(acc, -5.0) if weights else None
    kw = dict(acc_out=acc_out) if weights else {}
    got = check_decode(pkg, q, P, cache, lens, prefix, acc=acc, what=str(shape), workspace=ws, **kw)
    for b in range(B):
        if plen == 0 and int(lens[b]) == 0:
            assert bool((got[b] == 0).all())
        if weights:
            assert bool((acc_out[b, :, int(lens[b]):] == -5).all())
    # again, from the library's own workspace: the same bits
    again = torch.full_like(got, math.nan)
    if weights:
        new = acc.clone()
        pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, acc=new, out=again)
        for b in range(B):
            assert torch.equal(new[b, :, :int(lens[b])], acc_out[b, :, :int(lens[b])])
    else:
        pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, out=again)
    assert torch.equal(got, again)


def test_decode_part_of_a_prefix_and_lengths_out_of_range():
    pkg = spa()
    g = gen(12)
    B, H, Hk, d, m, dv, cap, pcap = 3, 4, 2, 64, 32, 64, 150, 200
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    prefix = make_cache(g, Hk, pcap, m=m, dv=dv, d=d)
    for t, bad in zip(prefix, (0x7c00, math.nan, math.inf)):
        t[:, 133:] = bad
    lens = torch.tensor([-7, 2**31 - 1, 60], dtype=I32, device="cuda")
    check_decode(pkg, q, P, cache, lens, prefix, plen=133)
    with pytest.raises(pkg.SpaError):
        pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, plen=201)


def test_decode_large_and_peaked_scores():
    """Scores far beyond the exponent range of exp, of both signs, growing along the keys."""
    pkg = spa()
    g = gen(13)
    B, H, Hk, d, m, dv, cap, plen = 2, 4, 2, 64, 32, 64, 400, 300
    q, P = (8 * randn(g, B, H, d)).to(BF16), (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d)
    prefix = make_cache(g, Hk, plen, m=m, dv=dv, d=d)
    cache[1].mul_(torch.exp2(torch.arange(cap, device="cuda") // 64))
    lens = torch.tensor([400, 33], dtype=I32, device="cuda")
    got = pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix)
    out, _, mag, rel = decode_ref(q, P, cache, lens, prefix, plen)
    tol = U[BF16] * out.abs() + (U[BF16] + rel) * 1.01 * mag
    assert bool(((got.double().cpu() - out).abs() <= tol).all())
    assert bool(torch.isfinite(got).all())


def test_decode_agrees_with_the_single_length_decode():
    pkg = spa()
    g = gen(14)
    B, H, d, m, dv, cap = 2, 3, 128, 32, 128, 900
    q, P = randn(g, B, H, d, dtype=BF16), (randn(g, H, d, m) / math.sqrt(m)).to(BF16)
    cache = make_cache(g, B, H, cap, m=m, dv=dv, d=d)
    a = pkg.spa_attention_decode(q, P, *cache, 777).double().cpu()
    lens = torch.full((B,), 777, dtype=I32, device="cuda")
    b = check_decode(pkg, q, P, cache, lens).double().cpu()
    out, _, mag, rel = decode_ref(q, P, cache, lens, None, 0)
    assert bool(((a - b).abs() <= U[BF16] * out.abs() + (U[BF16] + 2 * rel) * 1.01 * mag).all())


# ------------------------------------------------------------------ eviction
def evict_ref(acc, row_pos, n, budget, sink, recent):
    """The rows in their new order: plain lists."""
    left = min(n, budget)
    a, p = acc[:n].tolist(), row_pos[:n].tolist()
    if n == 0:
        return []
    newest = max(p)
    def rank(i):
        if p[i] < sink or p[i] > newest - recent:
            return (0, 0.0, i)
        return (2, 0.0, i) if math.isnan(a[i]) else (1, -a[i], i)
    kept = set(sorted(range(n), key=rank)[:left])
    late = iter(sorted(i for i in kept if i >= left))
    return [i if i in kept else next(late) for i in range(left)]


def run_evict(pkg, g, B, H, m, dv, cap, budget, sink, recent, lens, acc, row_pos, in_place):
    kc = torch.randint(-30000, 30000, (B, H, cap, m), generator=g, device="cuda", dtype=torch.int16)
    mul, v = randn(g, B, H, cap), randn(g, B, H, cap, dv, dtype=BF16)
    lens = torch.tensor(lens, dtype=I32, device="cuda")
    old = [t.clone() for t in (kc, mul, v, acc, row_pos, lens)]
    out = {} if in_place else dict(acc_out=torch.full_like(acc, -3.0), row_pos_out=torch.full_like(row_pos, -3),
                                   lens_out=torch.full_like(lens, -3))
    src = pkg.spa_kcache_evict(kc, mul, v, acc, row_pos, lens, budget, sink=sink, recent=recent, **out)
    a, p, l = (acc, row_pos, lens) if in_place else out.values()
    if not in_place:
        assert torch.equal(acc.view(I32), old[3].view(I32)) and torch.equal(row_pos, old[4]) and torch.equal(lens, old[5])
    for b in range(B):
        n = min(max(int(old[5][b]), 0), cap)
        left = min(n, budget)
        assert int(l[b]) == left
        for h in range(H):
            rows = evict_ref(old[3][b, h].cpu(), old[4][b, h].cpu(), n, budget, sink, recent)
            assert src[b, h].tolist() == rows + [-1] * (budget - left), (b, h)
            r = torch.tensor(rows, dtype=torch.long, device="cuda")
            for new, was in ((kc, old[0]), (mul, old[1]), (v, old[2]), (a.view(I32), old[3].view(I32)), (p, old[4])):
                assert torch.equal(new[b, h, :left], was[b, h, r])
            # behind the new length nothing changes
            for new, was in ((kc, old[0]), (mul, old[1]), (v, old[2])):
                assert torch.equal(new[b, h, left:], was[b, h, left:])
            if in_place:
                assert torch.equal(a[b, h, left:].view(I32), old[3][b, h, left:].view(I32))
            else:
                assert bool((a[b, h, left:] == -3).all()) and bool((p[b, h, left:] == -3).all())


EVICT = [
    # B, H, m, dv, cap, budget, sink, recent, lens
    (1, 1, 16, 64, 1, 1, 0, 0, [1]),
    (4, 2, 32, 128, 40, 16, 2, 5, [40, 16, 17, 0]),
    (3, 1, 64, 64, 3000, 1000, 0, 0, [3000, 2049, 1001]),
    (2, 3, 128, 128, 1500, 1024, 4, 100, [1500, 1025]),
    (1, 2, 32, 64, 5000, 4999, 10, 4000, [5000]),
    (1, 1, 32, 64, 20000, 64, 0, 64, [20000]),
    (2, 1, 16, 64, 100, 100, 50, 50, [100, 2**31 - 1]),
    (1, 1, 32, 128, 70000, 30000, 4, 512, [70000]),           # keys that do not fit in shared memory
    (61, 5, 16, 64, 70, 33, 1, 8, [(i * 7) % 71 for i in range(61)]),
    (2, 3, 16, 64, 9000, 4000, 3, 64, [9000, 8191]),
    (2, 1, 16, 64, 30000, 29000, 3, 64, [30000, 29001]),      # keys in shared memory
    (1, 2, 16, 64, 8192, 8191, 3, 64, [8192]),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", EVICT)
def test_evict(shape, in_place):
    pkg = spa()
    B, H, m, dv, cap, budget, sink, recent, lens = shape
    g = gen(cap + budget)
    # few distinct weights (ties), and the values that no order of floats puts in its place by itself
    acc = torch.floor(torch.rand((B, H, cap), generator=g, device="cuda") * 37) / 8
    special = torch.tensor([math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-42], device="cuda")
    at = torch.rand((B, H, cap), generator=g, device="cuda") < 0.2
    pick = torch.randint(0, 8, (B, H, cap), generator=g, device="cuda")
    acc = torch.where(at, special[pick], acc)
    row_pos = torch.argsort(torch.rand((B, H, cap), generator=g, device="cuda"), dim=-1).to(I32) * 2
    run_evict(pkg, g, B, H, m, dv, cap, budget, sink, recent, lens, acc, row_pos, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_equal_weights_and_repeated_positions(in_place):
    pkg = spa()
    g = gen(21)
    B, H, cap = 2, 2, 2500
    acc = torch.zeros((B, H, cap), device="cuda")
    row_pos = torch.zeros((B, H, cap), dtype=I32, device="cuda")   # every row is protected
    run_evict(pkg, g, B, H, 32, 64, cap, 1300, 1, 1, [2500, 1301], acc, row_pos, in_place)
    row_pos[...] = torch.iinfo(I32).min                            # the window reaches below the lowest
    run_evict(pkg, g, B, H, 32, 64, cap, 1300, 0, 700, [2500, 1301], acc, row_pos, in_place)


# ------------------------------------------------------------------ streams, graphs, a loop
def test_side_stream_and_graph_replay():
    """All four in a graph on a side stream; replayed with other lengths and inputs."""
    pkg = spa()
    g = gen(30)
    B, H, Hk, d, m, dv, cap, plen, budget = 3, 4, 2, 64, 32, 64, 300, 200, 128
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    table = pkg.rope_table(pkg.rope_frequencies(d))
    cache, prefix = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d), make_cache(g, Hk, plen, m=m, dv=dv, d=d)
    q, k, v = (randn(g, B, n, 1, c, dtype=BF16) for n, c in ((H, d), (Hk, d), (Hk, dv)))
    pos, lens = torch.tensor([[205], [400], [330]], device="cuda", dtype=I32), torch.tensor([5, 200, 130], device="cuda", dtype=I32)
    acc = torch.rand((B, Hk, cap), generator=g, device="cuda")
    row_pos = torch.argsort(torch.rand((B, Hk, cap), generator=g, device="cuda"), dim=-1).to(I32)
    state = (*cache, acc, row_pos, lens, pos, q, k, v)
    out, src = torch.empty((B, H, dv), dtype=BF16, device="cuda"), torch.empty((B, Hk, budget), dtype=I32, device="cuda")
    qr, kr = torch.empty_like(q), torch.empty_like(k)

    def step(**kw):
        pkg.spa_rope(q, table, pos, k=k, out=qr, k_out=kr, **kw)
        pkg.spa_kcache_append_ragged(kr, v, P, *cache, lens, acc=acc, row_pos=row_pos, token=pos.view(B), **kw)
        s = kw.get("stream")
        with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
            lens.add_(1)
        pkg.spa_attention_decode_shared(qr.view(B, H, d), P, *cache, lens, prefix=prefix, acc=acc, out=out, **kw)
        pkg.spa_kcache_evict(*cache, acc, row_pos, lens, budget, sink=2, recent=8, src=src, **kw)

    saved = [t.clone() for t in state]
    step()
    want = [t.clone() for t in (*state, out, src)]
    assert lens.tolist() == [6, 128, 128]
    for t, o in zip(state, saved):
        t.copy_(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for t, w in zip((*state, out, src), want):
        assert torch.equal(t, w)
    for t, o in zip(state, saved):
        t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t, o in zip(state, saved):
            t.copy_(o)
        out.fill_(0)
        graph.replay()
        for t, w in zip((*state, out, src), want):
            assert torch.equal(t, w)
    # other values in the same buffers
    saved[5].copy_(torch.tensor([0, 17, 299]))
    saved[7].copy_(randn(g, B, H, 1, d, dtype=BF16))
    for t, o in zip(state, saved):
        t.copy_(o)
    step()
    want = [t.clone() for t in (*state, out, src)]
    for t, o in zip(state, saved):
        t.copy_(o)
    graph.replay()
    for t, w in zip((*state, out, src), want):
        assert torch.equal(t, w)


def test_two_graphs_share_a_workspace():
    pkg = spa()
    g = gen(31)
    B, H, Hk, d, m, dv, cap, plen = 2, 4, 2, 64, 32, 64, 400, 300
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    cache, prefix = make_cache(g, B, Hk, cap, m=m, dv=dv, d=d), make_cache(g, Hk, plen, m=m, dv=dv, d=d)
    lens = torch.tensor([400, 77], device="cuda", dtype=I32)
    ws = torch.empty(pkg.spa_attention_decode_shared_workspace_size(B, H, Hk, plen, d, m, dv, cap),
                     dtype=torch.uint8, device="cuda")
    qs = [randn(g, B, H, d, dtype=BF16) for _ in range(2)]
    outs = [torch.empty((B, H, dv), dtype=BF16, device="cuda") for _ in range(2)]
    graphs = []
    for q, o in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix, out=o, workspace=ws)
    want = [pkg.spa_attention_decode_shared(q, P, *cache, lens, prefix=prefix) for q in qs]
    for _ in range(3):
        for x in graphs:
            x.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_decode_loop():
    """Prompts of different lengths behind a shared prefix, then steps of rope, append, decode and
    eviction; a plain loop in 64 bits follows the same tokens."""
    pkg = spa()
    g = gen(40)
    B, H, Hk, d, m, dv, cap, budget, plen = 3, 4, 2, 64, 32, 64, 48, 24, 70
    G, sink, recent = H // Hk, 2, 6
    freq = pkg.rope_frequencies(d, scaling=pkg.SPA_ROPE_BASE, factor=2.0)
    table = pkg.rope_table(freq)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    kc, mul = pkg.kcache_new(B, Hk, cap, m)
    vc = torch.zeros((B, Hk, cap, dv), dtype=BF16, device="cuda")
    acc, row_pos = torch.zeros((B, Hk, cap), device="cuda"), torch.zeros((B, Hk, cap), dtype=I32, device="cuda")
    # the prefix, at positions 0 .. plen-1
    kp, vp = randn(g, 1, Hk, plen, d, dtype=BF16), randn(g, 1, Hk, plen, dv, dtype=BF16)
    pkc, pmul = pkg.kcache_new(1, Hk, plen, m)
    pkg.spa_kcache_append(pkg.spa_rope(kp, table), P, pkc, pmul, 0)
    prefix = (pkc[0], pmul[0], vp[0])
    # the prompts, padded to the longest
    T = 31
    count = torch.tensor([31, 1, 20], device="cuda", dtype=I32)
    k, v = randn(g, B, Hk, T, d, dtype=BF16), randn(g, B, Hk, T, dv, dtype=BF16)
    zero = torch.zeros(B, dtype=I32, device="cuda")
    pkg.spa_kcache_append_ragged(pkg.spa_rope(k, table, pos0=plen), v, P, kc, mul, vc, zero, count, acc,
                                 row_pos, torch.full_like(zero, plen))
    lens, at = count.clone(), count + plen
    for step in range(12):
        q, k, v = (randn(g, B, n, 1, c, dtype=BF16) for n, c in ((H, d), (Hk, d), (Hk, dv)))
        qr, kr = pkg.spa_rope(q, table, at[:, None].contiguous(), k=k)
        check_rope(qr, q, freq, at[:, None], False)
        pkg.spa_kcache_append_ragged(kr, v, P, kc, mul, vc, lens, acc=acc, row_pos=row_pos, token=at)
        lens += 1
        at += 1
        check_decode(pkg, qr[:, :, 0].contiguous(), P, (kc, mul, vc), lens, prefix, acc=acc, what=f"step {step}")
        old = [t.clone() for t in (kc, acc, row_pos, lens)]
        src = pkg.spa_kcache_evict(kc, mul, vc, acc, row_pos, lens, budget, sink=sink, recent=recent)
        for b in range(B):
            n = int(old[3][b])
            assert int(lens[b]) == min(n, budget)
            for h in range(Hk):
                rows = evict_ref(old[1][b, h].cpu(), old[2][b, h].cpu(), n, budget, sink, recent)
                assert src[b, h, :len(rows)].tolist() == rows
                assert torch.equal(kc[b, h, :len(rows)], old[0][b, h, torch.tensor(rows, device="cuda")])
                # the newest tokens are still there
                p = set(row_pos[b, h, :int(lens[b])].tolist())
                assert {int(at[b]) - 1 - i for i in range(min(recent, n))} <= p
    # every step gave each sequence's own rows at most G of weight in all
    assert float(acc.sum(-1).max()) <= 12 * G + 1e-3


@pytest.mark.parametrize("kernel", [0, 1])
def test_decode_kernels_report_a_wait_that_runs_out(kernel):
    """The prefix kernel withholds its first "scores ready", the kernel of the own
    rows leaves its first copies unissued: the waits give up after 50 ms, every
    role drains what it started, and the device error word reports it.  A decode
    afterwards is right."""
    pkg = spa()
    t0 = time.perf_counter()
    status = pkg.selftest_decode_wait_timeout(50, kernel)
    elapsed = time.perf_counter() - t0
    assert status == pkg.SPA_ERR_TIMEOUT, pkg.status_str(status)
    assert elapsed < 1.5, f"self-test took {elapsed:.2f} s"
    assert pkg.device_error() == 0
    g = gen(77)
    q, P = randn(g, 2, 4, 64, dtype=BF16), (randn(g, 1, 64, 32) / math.sqrt(32)).to(BF16)
    cache = make_cache(g, 2, 1, 200, m=32, dv=64, d=64)
    prefix = make_cache(g, 1, 1000, m=32, dv=64, d=64)
    check_decode(pkg, q, P, cache, torch.tensor([200, 99], dtype=I32, device="cuda"), prefix, 1000,
                 what="after the self-test")
