"""The projected cache in 8 bits on the GPU against plain 64-bit implementations: packing,
the decode over pages and open rows, and a serving loop of both."""
import math

import pytest
import torch

from helpers import spa

pytestmark = pytest.mark.gpu

BF16, F16, F32, I32, I16, F8 = (torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int16,
                                torch.float8_e4m3fn)
PAGE = 64
# place of token t of a page in a column of values
PLACE = [16 * (t % 8 // 2) + 2 * (t // 8) + t % 2 for t in range(PAGE)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def i32(values):
    return torch.tensor(values, dtype=I32, device="cuda")


def open_rows(g, B, Hk, cap, m, dv, spread=3):
    """16-bit rows: K~ of magnitudes around 1 times 2^-spread .. 2^spread a row, multipliers powers of two."""
    x = randn(g, B, Hk, cap, m) * torch.exp2(
        torch.randint(-spread, spread + 1, (B, Hk, cap, 1), generator=g, device="cuda").float())
    e = torch.frexp(x.abs().amax(-1))[1] - 14
    mul = torch.ldexp(torch.ones_like(e, dtype=F32), e)
    return (x / mul[..., None]).to(F16).view(I16).contiguous(), mul, randn(g, B, Hk, cap, dv, dtype=BF16)


def key_values(kc, mul):
    return kc.view(F16).double() * mul.double()[..., None]


def bytes_of(t):
    return t.view(torch.uint8)


# ------------------------------------------------------------------ packing
def scale_of(x):
    """By comparisons alone, in 64 bits."""
    if not bool(x.isfinite().all()):
        return math.nan
    top = float(x.abs().max())
    s = 2.0 ** -100
    while top > 448 * s:
        s *= 2
    return s


def pack_reference(kc, mul, vc, lens, pages, table, blocks):
    """New (kc8, ks, vc8, vs, kc, mul, vc, lens, blocks), the arguments as they are."""
    kc, mul, vc = kc.clone(), mul.clone(), vc.clone()
    kc8, ks, vc8, vs = (t.clone() for t in pages)
    B, Hk, cap, _ = kc.shape
    n_pages, width = kc8.shape[0], table.shape[1]
    lens, blocks = [min(max(int(n), 0), cap) for n in lens], [min(max(int(n), 0), width) for n in blocks]
    k, v = key_values(kc, mul), vc.double()
    for b in range(B):
        done = 0
        while (done + 1) * PAGE <= lens[b] and blocks[b] + done < width:
            page = int(table[b, blocks[b] + done])
            if not 0 <= page < n_pages:
                break
            rows = slice(done * PAGE, (done + 1) * PAGE)
            for h in range(Hk):
                x, y = k[b, h, rows], v[b, h, rows]
                sk, sv = scale_of(x), scale_of(y)
                ks[page, h], vs[page, h] = sk, sv
                bytes_of(kc8)[page, h] = bytes_of((x / sk).float().to(F8))
                cols = torch.empty_like(y.T)
                cols[:, PLACE] = y.T
                bytes_of(vc8)[page, h] = bytes_of((cols / sv).float().to(F8))
            done += 1
        left = lens[b] - done * PAGE
        for t in (kc, mul, vc):
            t[b, :, :left] = t[b, :, done * PAGE:lens[b]].clone()
        lens[b], blocks[b] = left, blocks[b] + done
    return kc8, ks, vc8, vs, kc, mul, vc, i32(lens), i32(blocks)


def same(a, b):
    if a.dtype == F8:
        a, b = bytes_of(a), bytes_of(b)
    elif a.is_floating_point():  # NaN by their bits
        a, b = a.contiguous().view(I32 if a.dtype == F32 else I16), b.contiguous().view(I32 if a.dtype == F32 else I16)
    return torch.equal(a, b)


def check_pack(pkg, kc, mul, vc, lens, pages, table, blocks, where=True):
    """Runs the call; everything but the open rows behind the new length has to be the reference's."""
    ref = pack_reference(kc, mul, vc, lens, pages, table, blocks)
    lens_out, blocks_out = torch.full_like(lens, -7), torch.full_like(blocks, -7)
    pkg.spa_kcache8_pack(kc, mul, vc, lens, pages, table, blocks, lens_out, blocks_out)
    for i in (0, 2):
        assert same(pages[i], ref[i])
    for i in (1, 3):
        assert torch.equal(torch.nan_to_num(pages[i], nan=-1.0), torch.nan_to_num(ref[i], nan=-1.0))
    assert torch.equal(lens_out, ref[7]) and torch.equal(blocks_out, ref[8])
    for got, want in zip((kc, mul, vc), ref[4:7]):
        assert same(got, want)  # rows behind the new length are left as well, where nothing moved over them
    return lens_out, blocks_out


@pytest.mark.parametrize("m", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [64, 128])
def test_pack(m, dv):
    pkg = spa()
    g = gen(m + dv)
    lens = [0, 1, 63, 64, 65, 127, 128, 200, 319, -5, 1000]
    B, Hk, cap, width = len(lens), 3, 320, 9
    kc, mul, vc = open_rows(g, B, Hk, cap, m, dv)
    pages = pkg.kcache8_new(B * width + 2, Hk, m, dv)
    table = torch.randperm(B * width, generator=g, device="cuda").to(I32).view(B, width).contiguous()
    blocks = i32([0, 1, 2, 3, 4, 0, 1, 2, 3, 0, -3])
    check_pack(pkg, kc, mul, vc, i32(lens), pages, table, blocks)


def test_pack_without_room():
    """Blocks in front of one that has no page are packed; the others stay open, moved in order."""
    pkg = spa()
    g = gen(5)
    B, Hk, cap, m, dv, width = 6, 2, 450, 32, 64, 7
    kc, mul, vc = open_rows(g, B, Hk, cap, m, dv)
    pages = pkg.kcache8_new(B * width, Hk, m, dv)
    table = torch.arange(B * width, device="cuda", dtype=I32).view(B, width).clone()
    table[0, 1] = -1            # one block, six left
    table[1, 0] = B * width     # none
    table[2, 3] = 2**31 - 1
    blocks = i32([0, 0, 0, 6, 7, 100])
    lens = i32([450, 450, 449, 400, 300, 64])
    n, done = check_pack(pkg, kc, mul, vc, lens, pages, table, blocks)
    assert n.tolist() == [386, 450, 257, 336, 300, 64] and done.tolist() == [1, 0, 3, 7, 7, 7]


def test_pack_scales():
    pkg = spa()
    m, dv = 16, 64
    values = [0.0, 448.0, 448.5, 449.0, 2.0 ** -100, 448 * 2.0 ** -100, 450 * 2.0 ** -100, 2.0 ** -130, 3.3e38,
              math.inf, math.nan, -math.inf, 1.75, 1.76, 2.0 ** -9]
    B = len(values)
    v = torch.zeros(B, 1, PAGE, dv, dtype=BF16, device="cuda")
    k = torch.zeros(B, 1, PAGE, m, dtype=F16, device="cuda")
    mul = torch.ones(B, 1, PAGE, device="cuda")
    for b, x in enumerate(values):
        v[b, 0, 17, 5] = x
        v[b, 0, 3, 7] = 0.3
        if x in (3.3e38, 2.0 ** -100, 448 * 2.0 ** -100, 450 * 2.0 ** -100, 2.0 ** -130):
            k[b, 0, 63, 15], mul[b, 0, 63] = 1.0, 2.0 ** min(127, round(math.log2(x)))
        else:
            k[b, 0, 63, 15] = x
    k[0, 0, 2, 2], mul[0, 0, 2] = 60000.0, 2.0 ** 120        # beyond fp32
    pages = pkg.kcache8_new(B, 1, m, dv)
    table = torch.arange(B, device="cuda", dtype=I32).view(B, 1).contiguous()
    kk = k.view(I16).contiguous()
    # fp32 holds every product here but the first block's: the reference's scale there is NaN too
    ref_k = k.double() * mul.double()[..., None]
    pkg.spa_kcache8_pack(kk, mul, v, i32([PAGE] * B), pages, table, i32([0] * B))
    for b, x in enumerate(values):
        for got, want in ((pages[1][b, 0], ref_k[b, 0]), (pages[3][b, 0], v[b, 0].double())):
            want = want.clone()
            want[want.abs() > 3.402823466e38] = math.inf
            s = scale_of(want)
            assert float(got) == s or math.isnan(s) and math.isnan(float(got)), (x, float(got), s)


def test_pack_in_place_and_again():
    """In place; a second call without a full block changes nothing."""
    pkg = spa()
    g = gen(9)
    B, Hk, cap, m, dv = 3, 2, 200, 64, 128
    kc, mul, vc = open_rows(g, B, Hk, cap, m, dv)
    pages = pkg.kcache8_new(12, Hk, m, dv)
    table = torch.arange(12, device="cuda", dtype=I32).view(3, 4).contiguous()
    lens, blocks = i32([130, 64, 199]), i32([0, 1, 0])
    ref = pack_reference(kc, mul, vc, lens, pages, table, blocks)
    ws = torch.empty(pkg.spa_kcache8_pack_workspace_size(B), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        pkg.spa_kcache8_pack(kc, mul, vc, lens, pages, table, blocks, workspace=ws)
        for got, want in zip((*pages, kc, mul, vc, lens, blocks), ref):
            assert same(got, want) if got.dtype != I32 else torch.equal(got, want)


# ------------------------------------------------------------------ decode
def decode_reference(q, P, pages, table, blocks, kc, mul, vc, lens, window, sink):
    """out in 64 bits, and for every value the tolerance of what is not its own rounding."""
    B, H, d = q.shape
    Hk, _, m = P.shape
    G, dv, width, cap = H // Hk, vc.shape[-1], table.shape[1], vc.shape[2]
    out, tol = (torch.zeros(B, H, dv, dtype=torch.float64, device="cuda") for _ in range(2))
    q, P = q.double(), P.double()
    for b in range(B):
        nb, r = min(max(int(blocks[b]), 0), width), min(max(int(lens[b]), 0), cap)
        n = PAGE * nb + r
        seen = lambda j: not window or j >= n - window or j < sink  # noqa: E731
        for h in range(Hk):
            ks, vs = [], []
            for i in range(nb):
                cut = [t for t in range(PAGE) if seen(PAGE * i + t)]
                page = int(table[b, i])
                if not cut or not 0 <= page < pages[0].shape[0]:
                    continue
                ks.append(pages[0][page, h].double()[cut] * pages[1][page, h].double())
                v = pages[2][page, h].double()[:, PLACE].T
                vs.append(v[cut] * pages[3][page, h].double())
            cut = [t for t in range(r) if seen(PAGE * nb + t)]
            ks.append(key_values(kc[b, h, cut], mul[b, h, cut]))
            vs.append(vc[b, h, cut].double())
            k, v = torch.cat(ks), torch.cat(vs)
            if len(k) == 0:
                continue
            rows = slice(h * G, (h + 1) * G)
            p = torch.softmax(q[b, rows] @ P[h] @ k.T / math.sqrt(m), -1)
            out[b, rows] = p @ v
            # A score is a sum of terms up to |q| |P| |k|: d roundings of 2^-24 in q~, m in the score, 2^-21 for
            # the parts of q~, the scales and the base-2 exponent.  A weight is off by twice that (its own
            # exponential and the sum) and by 2^-11, its rounding to fp16 for a page's values (2^-15 for the parts
            # of an open row's), and sums run over n / 8 keys per lane.
            size = (q[b, rows].abs() @ P[h].abs() @ k.abs().T / math.sqrt(m)).amax(-1, keepdim=True)
            size = size * ((d + m) * 2.0 ** -24 + 2.0 ** -21)
            tol[b, rows] = (2 * size + 2.0 ** -11 + len(k) * 2.0 ** -24) * (p @ v.abs())
    return out, tol


def check_decode(got, ref, tol):
    over = ((got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - tol - 1e-30).max()
    assert float(over) <= 0, float(over)


def pool(g, pkg, lens, Hk, m, dv, extra=3):
    """Pages for sequences of `lens` tokens, filled; table, blocks, open lengths."""
    B, width = len(lens), max(1, max(n // PAGE for n in lens))
    total = sum(n // PAGE for n in lens) + extra
    pages = pkg.kcache8_new(total, Hk, m, dv)
    for t in (pages[0], pages[2]):
        t.copy_((randn(g, *t.shape) * 100).clamp(-448, 448).to(F8))
    for t in (pages[1], pages[3]):
        t.copy_(torch.exp2(torch.randint(-10, -4, t.shape, generator=g, device="cuda").float()))
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table = torch.full((B, width), -1, dtype=I32)
    for b, n in enumerate(lens):
        for i in range(n // PAGE):
            table[b, i] = order.pop()
    for page in order:  # pages of nobody: NaN codes and scales
        bytes_of(pages[0])[page], bytes_of(pages[2])[page] = 0x7f, 0xff
        pages[1][page] = pages[3][page] = math.nan
    return pages, table.cuda(), i32([n // PAGE for n in lens]), i32([n % PAGE for n in lens])


def spoil(kc, mul, vc, lens, first):
    """NaN and infinities in open rows behind each length and in front of `first`."""
    for b, n in enumerate(lens.tolist()):
        for cut in (slice(n, None), slice(0, first[b])):
            kc[b, :, cut] = 0x7e00
            mul[b, :, cut] = math.inf
            vc[b, :, cut] = math.nan


DECODE = [
    # lens, G, Hk, d, m, dv, window, sink
    ([1], 1, 1, 32, 16, 64, 0, 0),
    ([0, 63, 64, 65, 0, 200], 4, 2, 64, 32, 128, 0, 0),
    ([700, 64, 1], 8, 1, 128, 64, 128, 0, 0),
    ([129, 513], 9, 2, 96, 32, 64, 0, 0),            # more than 8 heads: products of their own
    ([300, 128], 16, 1, 128, 128, 128, 0, 0),
    ([257, 70], 17, 1, 64, 64, 64, 0, 0),            # two parts of a group
    ([190, 191], 40, 1, 33, 16, 128, 0, 0),
    ([130] * 33, 3, 2, 200, 128, 64, 0, 0),
    ([1000, 5, 64, 128, 321], 2, 2, 64, 32, 64, 100, 0),
    ([1000, 5, 64, 128, 321], 2, 2, 64, 32, 64, 100, 7),
    ([1000, 65, 640], 4, 1, 64, 16, 128, 1, 0),      # the newest key alone
    ([1000, 65, 640], 10, 1, 64, 64, 128, 70, 130),
    ([1000, 447], 4, 1, 128, 128, 64, 448, 64),
    ([640, 704], 4, 2, 64, 32, 64, 128, 1),          # borders on pages
    ([90, 120], 4, 2, 64, 32, 64, 10, 70),           # the first keys reach into the open rows
    ([100, 127], 4, 2, 64, 32, 64, 10, 66),
    ([5000], 1, 2, 64, 32, 128, 2**31 - 1, 2**31 - 1),
    ([9000, 20000], 4, 1, 64, 32, 64, 0, 0),
]


@pytest.mark.parametrize("case", DECODE)
def test_decode(case):
    lens, G, Hk, d, m, dv, window, sink = case
    pkg = spa()
    g = gen(sum(lens) + m)
    B = len(lens)
    pages, table, blocks, left = pool(g, pkg, lens, Hk, m, dv)
    kc, mul, vc = open_rows(g, B, Hk, 80, m, dv, spread=1)
    q = randn(g, B, G * Hk, d, dtype=BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    first = [0] * B
    if window:
        for b, n in enumerate(lens):
            lo = n - window
            if lo > sink:  # open rows in front of the window that are not among the first keys
                a = max(0, sink - n // PAGE * PAGE)
                first[b] = max(0, lo - n // PAGE * PAGE) if a == 0 else 0
            for i in range(n // PAGE):  # pages that are not seen have gone to nobody
                if (i + 1) * PAGE <= lo and i * PAGE >= sink:
                    table[b, i] = -1 if i % 2 else pages[0].shape[0]
    spoil(kc, mul, vc, left, first)
    ref = decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, window, sink)
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left, window=window, sink=sink)
    check_decode(got, *ref)
    for b, n in enumerate(lens):
        if n == 0:
            assert not got[b].any()


def test_decode_scales_of_any_size():
    """Value scales that differ by far within a sequence, pages of zeros, blocks without pages, NaN scales."""
    pkg = spa()
    g = gen(21)
    lens, G, Hk, d, m, dv = [1030, 640, 512, 64], 4, 2, 64, 32, 64
    pages, table, blocks, left = pool(g, pkg, lens, Hk, m, dv)
    for i in range(16):
        pages[3][int(table[0, i])] = 2.0 ** (-100 + 9 * i)
        pages[1][int(table[0, i])] = 2.0 ** -(40 + i)
    zero = int(table[0, 3])
    bytes_of(pages[2])[zero] = 0
    pages[3][zero] = 1.37 * 2.0 ** -100                     # not a power of two
    table[1, 0], table[1, 4], table[1, 9] = -1, 10**6, -2**31
    table[2, :8] = -1                                       # no key at all
    pages[1][int(table[3, 0]), 1] = math.nan
    kc, mul, vc = open_rows(g, 4, Hk, 64, m, dv)
    q = randn(g, 4, G * Hk, d, dtype=BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left)
    ref = decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, 0, 0)
    check_decode(got[:3], ref[0][:3], ref[1][:3])
    assert not got[2].any()
    assert bool(got[3, G:].isnan().all())                   # the head whose scale is NaN shows it
    check_decode(got[3, :G], ref[0][3, :G], ref[1][3, :G])


def test_decode_growing_scores():
    """Every page's scores far above the ones before: the maximum moves each time."""
    pkg = spa()
    g = gen(22)
    lens, m, dv, d = [64 * 40 + 33], 16, 64, 32
    for wide in (4, 12):
        pages, table, blocks, left = pool(g, pkg, lens, 1, m, dv)
        for i in range(40):
            pages[1][int(table[0, i])] = 2.0 ** (-12 + i / 4)
        kc, mul, vc = open_rows(g, 1, 1, 64, m, dv)
        q = randn(g, 1, wide, d, dtype=BF16)
        P = (randn(g, 1, d, m) / math.sqrt(m)).to(BF16)
        got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left)
        check_decode(got, *decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, 0, 0))


def test_decode_shared_pages_and_empty_parts():
    """Pages that serve several sequences; no pages at all; no open rows at all."""
    pkg = spa()
    g = gen(23)
    m, dv, d, Hk = 32, 128, 64, 2
    pages, table, blocks, left = pool(g, pkg, [640], Hk, m, dv)
    table, blocks = table.expand(5, -1).contiguous(), i32([10, 3, 1, 0, 10])
    kc, mul, vc = open_rows(g, 5, Hk, 64, m, dv)
    q = randn(g, 5, 8, d, dtype=BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    left = i32([0, 5, 64, 0, 33])
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left)
    check_decode(got, *decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, 0, 0))
    none = pkg.kcache8_new(0, Hk, m, dv), torch.empty(5, 0, dtype=I32, device="cuda")
    got = pkg.spa_attention_decode8(q, P, *none, blocks, kc, mul, vc, left)
    check_decode(got, *decode_reference(q, P, *none, blocks, kc, mul, vc, left, 0, 0))
    # against the decode of 16-bit rows alone
    other = pkg.spa_attention_decode_shared(q, P, kc, mul, vc, left)
    check_decode(got, other.double(), 2.0 ** -8 * other.double().abs() + 1e-3)
    no = tuple(t[:, :, :0].contiguous() for t in (kc, mul, vc))
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, *no, left)
    check_decode(got, *decode_reference(q, P, pages, table, blocks, *no, left * 0, 0, 0))


def test_decode_many_sequences_and_repeats():
    """More sequences than threads of a block scan at once, most of them empty; the same bits on another stream."""
    pkg = spa()
    g = gen(24)
    B, Hk, m, dv, d = 700, 1, 16, 64, 32
    lens = [0] * B
    for b, n in ((3, 64), (4, 1), (255, 200), (256, 129), (511, 63), (699, 640)):
        lens[b] = n
    pages, table, blocks, left = pool(g, pkg, lens, Hk, m, dv)
    kc, mul, vc = open_rows(g, B, Hk, 64, m, dv)
    q = randn(g, B, 2, d, dtype=BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left)
    check_decode(got, *decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, 0, 0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = [pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left, stream=s)
            for s in (side, torch.cuda.current_stream(), side)]
    torch.cuda.synchronize()
    assert all(torch.equal(got, t) for t in both)


def test_long_cache_offsets():
    """Pages whose byte offsets pass 32 bits."""
    pkg = spa()
    g = gen(25)
    Hk, m, dv, d = 8, 64, 128, 64
    n = 2**32 // (Hk * PAGE * m) + 40                       # K~ beyond 4 GiB, V beyond 8
    pages = pkg.kcache8_new(n, Hk, m, dv)
    last = list(range(n - 9, n))
    for t in (pages[0], pages[2]):
        t[n - 9:] = (randn(g, 9, *t.shape[1:]) * 100).clamp(-448, 448).to(F8)
    pages[1][n - 9:] = pages[3][n - 9:] = 2.0 ** -7
    table, blocks, left = i32([last]), i32([9]), i32([64 + 30])
    kc, mul, vc = open_rows(g, 1, Hk, 128, m, dv)
    q = randn(g, 1, 2 * Hk, d, dtype=BF16)
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left)
    check_decode(got, *decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, 0, 0))
    table = i32([last[:8] + [n - 20, n - 9]])
    ref = pack_reference(kc, mul, vc, left, [t[n - 20:] for t in pages], i32([[0] * 9 + [11]]), blocks)
    blocks_out = blocks.clone()
    pkg.spa_kcache8_pack(kc, mul, vc, left, pages, table, blocks, blocks_out=blocks_out)
    assert same(pages[0][n - 9], ref[0][11]) and same(pages[2][n - 9], ref[2][11]) and int(blocks_out) == 10


# ------------------------------------------------------------------ a serving loop
def test_serving_loop_and_graph():
    """norm_rope, ragged append, decode8 and pack, step by step against 64 bits; a captured step replays."""
    pkg = spa()
    g = gen(31)
    B, H, Hk, d, m, dv, cap, steps, window, sink = 3, 8, 2, 64, 32, 64, 128, 150, 100, 3
    P = (randn(g, Hk, d, m) / math.sqrt(m)).to(BF16)
    wq, wk = ((1 + 0.2 * randn(g, d)).to(BF16) for _ in range(2))
    table = pkg.rope_table(pkg.rope_frequencies(d))
    x = [randn(g, steps, B, h, 1, w, dtype=BF16) for h, w in ((H, d), (Hk, d), (Hk, dv))]

    def fresh():
        pages = pkg.kcache8_new(3 * B, Hk, m, dv)
        pt = torch.arange(3 * B, device="cuda", dtype=I32).flip(0).view(B, 3).contiguous()
        kc, mul = pkg.kcache_new(B, Hk, cap, m)
        vc = torch.zeros(B, Hk, cap, dv, dtype=BF16, device="cuda")
        return pages, pt, i32([0] * B), kc, mul, vc, i32([0, 0, 0]), i32([5, 0, 77])

    def step(q, k, v, state, out):
        pages, pt, blocks, kc, mul, vc, lens, pos = state
        q, k = pkg.spa_norm_rope(q, wq, table, pos[:, None], k=k, wk=wk)
        pkg.spa_kcache_append_ragged(k, v, P, kc, mul, vc, lens)
        lens += 1
        pos += 1
        pkg.spa_attention_decode8(q[:, :, 0].contiguous(), P, pages, pt, blocks, kc, mul, vc, lens, window=window,
                                  sink=sink, out=out)
        pkg.spa_kcache8_pack(kc, mul, vc, lens, pages, pt, blocks)
        return q

    state, out = fresh(), torch.empty(B, H, dv, dtype=BF16, device="cuda")
    outs = []
    for t in range(steps):
        before = [a.clone() if torch.is_tensor(a) else [b.clone() for b in a] for a in state]
        q = step(x[0][t], x[1][t], x[2][t], state, out)
        outs.append(out.clone())
        if t % 7 == 0 or t in (63, 64, 127, 128):
            # the cache as the step's decode saw it: before, with the step's rows
            pages, pt, blocks, kc, mul, vc, lens, _ = before
            k = pkg.spa_norm_rope(x[1][t], wk, table, before[7][:, None])
            pkg.spa_kcache_append_ragged(k, x[2][t], P, kc, mul, vc, lens)
            check_decode(out, *decode_reference(q[:, :, 0], P, pages, pt, blocks, kc, mul, vc, lens + 1, window, sink))
    assert state[2].tolist() == [2] * B and state[6].tolist() == [steps - 128] * B

    again, fixed = fresh(), [a[0].clone() for a in x]
    other = torch.empty_like(out)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(*fixed, fresh(), other)  # warm
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*fixed, again, other)
    torch.cuda.synchronize()
    for a, b in zip(again, fresh()):  # capturing runs nothing
        assert all(same(m_, n_) for m_, n_ in zip(a, b)) if isinstance(a, tuple) else torch.equal(a, b)
    for t in range(steps):
        for a, b in zip(fixed, x):
            a.copy_(b[t])
        graph.replay()
        assert torch.equal(other, outs[t])
    assert all(torch.equal(a, b) for a, b in zip(again[2:], state[2:]))


@pytest.mark.parametrize("G", [3, 11])
def test_decode_small_scores_on_a_border(G):
    """Pages of zero keys, whose scale is the smallest, under queries so small that scale times query is nothing: the
    keys that a border hides stay hidden, the others weigh the same."""
    pkg = spa()
    g = gen(41 + G)
    d, m, dv, lens = 64, 32, 64, [300, 230, 129]
    pages, table, blocks, left = pool(g, pkg, lens, 1, m, dv)
    bytes_of(pages[0]).zero_()
    pages[1].fill_(2.0 ** -100)
    kc, mul, vc = open_rows(g, 3, 1, 64, m, dv)
    q = (randn(g, 3, G, d) * 2.0 ** -60).to(BF16)
    P = (randn(g, 1, d, m) / math.sqrt(m)).to(BF16)
    for window, sink in ((100, 0), (100, 7), (150, 70)):
        got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left, window=window, sink=sink)
        check_decode(got, *decode_reference(q, P, pages, table, blocks, kc, mul, vc, left, window, sink))


@pytest.mark.parametrize("G", [1, 4, 12])
@pytest.mark.parametrize("nats", [8, 12, 14, 16, 20])
def test_decode_one_key_far_above(nats, G):
    """A first key with most of the weight and a value of zero: the output is made of the small weights."""
    pkg = spa()
    g = gen(31 + nats + G)
    d, m, dv, lens = 64, 32, 64, [8192, 8192 + 37]
    pages, table, blocks, left = pool(g, pkg, lens, 1, m, dv)
    kc, mul, vc = open_rows(g, 2, 1, 64, m, dv)
    mul.mul_(2.0 ** -6)
    P = (randn(g, 1, d, m) / math.sqrt(m)).to(BF16)
    one = randn(g, d)
    q = (one * torch.linspace(1.0, 0.9, G, device="cuda")[:, None]).expand(2, G, d).to(BF16).contiguous()
    qp = one.double() @ P[0].double()
    code = (qp * (300 / qp.abs().max())).to(F8)
    for b in range(2):
        for page in table[b, :blocks[b]].tolist():  # the others' logits: a deviation of a half
            pages[1][page, 0] = 0.5 * math.sqrt(m) / (100 * float(qp.norm()))
        first = int(table[b, 0])
        bytes_of(pages[0])[first, 0] = 0
        bytes_of(pages[0])[first, 0, 0] = bytes_of(code)
        pages[1][first, 0] = nats * math.sqrt(m) / float(code.double() @ qp)
        bytes_of(pages[2])[first, 0, :, PLACE[0]] = 0
    got = pkg.spa_attention_decode8(q, P, pages, table, blocks, kc, mul, vc, left).double()
    for b in range(2):
        page = table[b, :blocks[b]].long()
        r = int(left[b])
        k = torch.cat((pages[0][page, 0].double().mul(pages[1][page, 0].double()[:, None, None]).flatten(0, 1),
                       key_values(kc[b, 0, :r], mul[b, 0, :r])))
        v = torch.cat((pages[2][page, 0].double()[:, :, PLACE].mul(pages[3][page, 0].double()[:, None, None])
                       .transpose(1, 2).flatten(0, 1), vc[b, 0, :r].double()))
        p = torch.softmax(q[b].double() @ P[0].double() @ k.T / math.sqrt(m), -1)
        assert not v[0].any() and float(p[:, 0].min()) > 0.05
        ref = p @ v
        # As in decode_reference, but the first key's score and the sum of weights, of n additions one after the other
        # at most, take all values by one factor.  A weight's own errors: its score, its rounding to fp16, and its
        # place in a page's sum of 64 and a segment's of n / 64 pages.
        size = (q[b].double().abs() @ P[0].double().abs() @ k.abs().T / math.sqrt(m)) * (
            (d + m) * 2.0 ** -24 + 2.0 ** -21)
        tol = (2 * size[:, :1] + len(k) * 2.0 ** -24) * ref.abs() + (
            2 * size[:, 1:].amax(-1, keepdim=True) + 2.0 ** -11 + (len(k) / 64 + 64) * 2.0 ** -24) * (p @ v.abs())
        check_decode(got[b], ref, tol)
