"""Norms of queries and keys with rotary positions in one pass, and the gradient, on the
GPU against 64-bit arithmetic."""
import math

import pytest
import torch

from helpers import spa

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # half a step
EPS = 1e-6
# Relative to the magnitudes that enter a feature.  A row's sum of squares: a chain of 16 products
# and sums in a thread, five shuffled sums, the mean and eps, 23 x 2^-24, halved by the root; the
# reciprocal root and the sine two steps each, 2^-22; six more roundings: below 2^-19.
FWD = 2.0 ** -19
# The gradient's sum of t x: chains of 16 features with three roundings each and five sums, below
# 2^-18; r^3 three times the root's 2^-20; sine and further roundings as above: below 2^-17.
BWD = 2.0 ** -17


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def turn(x, freq, pos, interleaved, back=False):
    """R(pos) x (or its transpose) in 64 bits."""
    rot = 2 * len(freq)
    if rot == 0:
        return x
    ang = pos.double()[:, None, :, None] * freq.to(x.device)
    c, s = torch.cos(ang), torch.sin(ang) * (-1 if back else 1)
    y = x.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


def pair_sum(x, rot, interleaved):
    """|a| + |b| of the pair of each rotated feature, |x| of the others."""
    y = x.abs()
    z = y.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    z[..., ia] = z[..., ib] = y[..., ia] + y[..., ib]
    return z


def reference(x, w, freq, pos, interleaved, eps=EPS):
    x, w = x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return turn(x * r * w, freq, pos, interleaved), pair_sum(x * r * w, 2 * len(freq), interleaved)


def gradient(dy, x, w, freq, pos, interleaved, eps=EPS):
    """dx, dw and what bounds their errors."""
    dy, x, w = dy.double(), x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = turn(dy, freq, pos, interleaved, back=True)
    most = pair_sum(dy, 2 * len(freq), interleaved)
    t = w * h
    dx = r * (t - x * r * r * (t * x).mean(-1, keepdim=True))
    of_dx = r * (w.abs() * most + x.abs() * r * r * (w.abs() * most * x.abs()).mean(-1, keepdim=True))
    return dx, (h * x * r).sum((0, 1, 2)), of_dx, (most * (x * r).abs()).sum((0, 1, 2))


def near(got, ref, bound, rel):
    tol = U[got.dtype] * ref.abs() + rel * bound + 1e-30
    over = ((got.double() - ref).abs() - tol).max() if ref.numel() else torch.tensor(-1.0)
    assert float(over) <= 0, float(over)


def summed(got, ref, bound, rows):
    # a thread adds its rows one after the other, a block its groups (256 at most), a warp the blocks (608 / 32
    # and five sums): no chain is longer than the rows it covers, or than rows / threads and these
    chain = min(rows, 320 + rows // 1024)
    assert bool(((got.double() - ref).abs() <= (BWD + chain * 2.0 ** -24) * bound + 1e-30).all())


SHAPES = [
    # B, H, Hk, N, d, rot
    (1, 1, 0, 1, 1, 0),
    (1, 1, 0, 1, 2, 2),
    (2, 3, 1, 5, 64, 64),
    (3, 4, 2, 7, 96, 38),      # a half of 19 features
    (1, 5, 5, 33, 80, 80),
    (2, 2, 1, 9, 33, 20),      # an odd width
    (1, 8, 2, 130, 128, 64),
    (1, 9, 3, 17, 128, 0),     # the norm alone
    (2, 1, 1, 3, 256, 256),
    (1, 2, 1, 3, 255, 2),      # a tail of single features
    (2, 7, 7, 2, 200, 136),
    (64, 32, 8, 1, 128, 128),
]


def inputs(shape, dtype, seed=0):
    B, H, Hk, N, d, rot = shape
    g = gen(N * d + rot + seed)
    pkg = spa()
    freq = pkg.rope_frequencies(rot) if rot else torch.zeros(0, dtype=torch.float64)
    table = pkg.rope_table(freq) if rot else None
    pos = torch.randint(-5, 1 << 20, (B, N), generator=g, device="cuda", dtype=I32)
    scale = torch.exp2(torch.randint(-8, 9, (B, 1, N, 1), generator=g, device="cuda").float())
    q, k = (randn(g, B, h, N, d) * scale for h in (H, Hk))
    w = [1 + 0.3 * randn(g, d) for _ in range(2)]
    dy = [randn(g, B, h, N, d) for h in (H, Hk)]
    return pkg, freq, table, pos, *(t.to(dtype) for t in (q, k, *w, *dy))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_rope(shape, interleaved, dtype):
    pkg, freq, table, pos, q, k, wq, wk, _, _ = inputs(shape, dtype)
    if shape[2]:
        a, b = pkg.spa_norm_rope(q, wq, table, pos, k=k, wk=wk, eps=EPS, interleaved=interleaved)
        near(b, *reference(k, wk, freq, pos, interleaved), FWD)
    else:
        a = pkg.spa_norm_rope(q, wq, table, pos, eps=EPS, interleaved=interleaved)
    near(a, *reference(q, wq, freq, pos, interleaved), FWD)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(1, 6, 2, 3001, 64, 32)])
def test_gradient(shape, interleaved, dtype):
    pkg, freq, table, pos, q, k, wq, wk, dyq, dyk = inputs(shape, dtype)
    if shape[2]:
        dq, dk, dwq, dwk = pkg.spa_norm_rope_bwd(dyq, q, wq, table, pos, dk_out=dyk, k=k, wk=wk, eps=EPS,
                                                 interleaved=interleaved)
        dx, dw, bx, bw = gradient(dyk, k, wk, freq, pos, interleaved)
        near(dk, dx, bx, BWD)
        summed(dwk, dw, bw, shape[0] * shape[2] * shape[3])
    else:
        dq, dwq = pkg.spa_norm_rope_bwd(dyq, q, wq, table, pos, eps=EPS, interleaved=interleaved)
    dx, dw, bx, bw = gradient(dyq, q, wq, freq, pos, interleaved)
    near(dq, dx, bx, BWD)
    summed(dwq, dw, bw, shape[0] * shape[1] * shape[3])


def test_gradient_against_differences():
    pkg, freq, table, pos, q, _, w, _, u, _ = inputs((2, 3, 0, 11, 64, 48), F32, seed=7)
    q = q / q.square().mean(-1, keepdim=True).sqrt()
    g = gen(8)
    v, vw = randn(g, *q.shape), randn(g, 64)
    h = 2.0 ** -7

    def loss(x, weight):
        return float((pkg.spa_norm_rope(x, weight, table, pos, eps=EPS).double() * u.double()).sum())

    dq, dw = pkg.spa_norm_rope_bwd(u, q, w, table, pos, eps=EPS)
    # rounding of the two losses, and of the perturbed inputs (2^-24 of a value, through the gradient)
    size = float((reference(q, w, freq, pos, False)[1] * u.double().abs()).sum())
    moved = float(dq.double().abs().mul(q.double().abs() + 1).sum()) * 2.0 ** -23
    rounding = (2 * size * FWD + moved) / (2 * h)
    # the third derivative of x / |x| along v is at most 6 (|v| / |x|)^3 (1 - h |v| / |x|)^-3
    a = v.double().norm(dim=-1) / q.double().norm(dim=-1)
    cut = h * h * float((a ** 3 / (1 - h * a) ** 3 * math.sqrt(64) * w.abs().max() * u.double().norm(dim=-1)).sum())
    found = (loss(q + h * v, w) - loss(q - h * v, w)) / (2 * h)
    assert abs(found - float((dq.double() * v.double()).sum())) <= rounding + cut
    # linear in the weights
    found = (loss(q, w + h * vw) - loss(q, w - h * vw)) / (2 * h)
    assert abs(found - float((dw.double() * vw.double()).sum())) <= rounding + size * 2.0 ** -23 / h


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_and_broadcast(interleaved):
    pkg = spa()
    g = gen(3)
    B, H, Hk, N, d = 2, 4, 2, 37, 64
    freq = pkg.rope_frequencies(d)
    table = pkg.rope_table(freq)
    pos = torch.arange(N, device="cuda", dtype=I32).expand(B, N).contiguous() + 11
    wq, wk = randn(g, d, dtype=BF16), randn(g, d, dtype=BF16)
    x = randn(g, B, N, H + 2 * Hk, d, dtype=BF16)            # token-major, with values behind
    keep = x.clone()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    call = dict(wk=wk, eps=EPS, interleaved=interleaved)
    a, b = pkg.spa_norm_rope(q, wq, table, k=k, pos0=11, **call)
    near(a, *reference(q, wq, freq, pos, interleaved), FWD)
    near(b, *reference(k, wk, freq, pos, interleaved), FWD)
    dyq, dyk = randn(g, B, H, N, d, dtype=BF16), randn(g, B, Hk, N, d, dtype=BF16)
    grads = pkg.spa_norm_rope_bwd(dyq, q, wq, table, pos, dk_out=dyk, k=k, **call)
    near(grads[0], *gradient(dyq, q, wq, freq, pos, interleaved)[::2], BWD)
    # the gradient over the upstream one, and over the inputs; the same bits
    over = dyq.clone(), dyk.clone()
    again = pkg.spa_norm_rope_bwd(over[0], q, wq, table, pos, dk_out=over[1], k=k, dq=over[0], dk=over[1], **call)
    assert all(torch.equal(m, n) for m, n in zip(grads, again)) and again[0] is over[0]
    y = x.clone()
    yq, yk = y[:, :, :H].transpose(1, 2), y[:, :, H:H + Hk].transpose(1, 2)
    again = pkg.spa_norm_rope_bwd(dyq, yq, wq, table, pos, dk_out=dyk, k=yk, dq=yq, dk=yk, **call)
    assert all(torch.equal(m, n) for m, n in zip(grads, again))
    assert torch.equal(y[:, :, H + Hk:], keep[:, :, H + Hk:])
    # in place, strided: the same bits, and nothing else is touched
    pkg.spa_norm_rope(q, wq, table, pos, k=k, out=q, k_out=k, **call)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(x[:, :, H + Hk:], keep[:, :, H + Hk:])
    # an offset that only allows single features; one row for all sequences (stride 0)
    y = randn(g, 1, H, N, d + 1, dtype=BF16)[..., 1:].expand(B, H, N, d)
    near(pkg.spa_norm_rope(y, wq, table, pos, eps=EPS, interleaved=interleaved),
         *reference(y, wq, freq, pos, interleaved), FWD)
    dx, dw = pkg.spa_norm_rope_bwd(y, y, wq, table, pos, eps=EPS, interleaved=interleaved)
    ref = gradient(y, y, wq, freq, pos, interleaved)
    near(dx, ref[0], ref[2], BWD)
    summed(dw, ref[1], ref[3], B * H * N)
    with pytest.raises(pkg.SpaError):
        pkg.spa_norm_rope(y, wq, table, pos, out=y)          # sequences that share an output row
    with pytest.raises(ValueError):
        pkg.spa_norm_rope(x.transpose(2, 3)[:, :, :, :N], wq, None)


def test_rows_of_zeros_and_far_positions():
    pkg = spa()
    freq = pkg.rope_frequencies(64)
    pos = torch.tensor([[0, 1, -1, 2**31 - 1, -2**31, 10**9 + 7]], device="cuda", dtype=I32)
    x = randn(gen(4), 1, 2, 6, 64)
    x[0, 0, 2] = 0
    got = pkg.spa_norm_rope(x, None, pkg.rope_table(freq), pos, eps=EPS)
    assert not got[0, 0, 2].any()
    one = torch.ones(64, device="cuda")
    # the reference's own product is off by 2^-53 of 2^31 rad, the table by the rounding of f / 2pi and of 2pi
    near(got, *reference(x, one, freq, pos, False), FWD + 3 * 2.0 ** 31 * 2.0 ** -53)
    dx, dw = pkg.spa_norm_rope_bwd(x, x, None, pkg.rope_table(freq), pos, eps=EPS)
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    # a row of zeros: dx = r R^T dy
    u = randn(gen(5), 1, 1, 1, 64)
    dx, dw = pkg.spa_norm_rope_bwd(u, torch.zeros_like(u), None, None, eps=EPS)
    assert bool(((dx.double() - u.double() * EPS ** -0.5).abs() <= BWD * u.double().abs() * EPS ** -0.5).all())
    assert not dw.any()


def test_no_rows():
    pkg = spa()
    w = torch.ones(32, device="cuda")
    dq, dw = pkg.spa_norm_rope_bwd(torch.zeros(2, 3, 0, 32, device="cuda"), torch.zeros(2, 3, 0, 32, device="cuda"), w,
                                   dwq=torch.full((32,), 7.0, device="cuda"))
    assert dq.shape == (2, 3, 0, 32) and not dw.any()
    assert pkg.spa_norm_rope(torch.zeros(0, 3, 4, 32, device="cuda"), w).shape == (0, 3, 4, 32)


def test_replay_streams_and_workspace():
    """The same bits each time, on another stream, and from a captured graph that lives beside eager calls."""
    shape = (3, 6, 2, 700, 96, 64)
    pkg, freq, table, pos, q, k, wq, wk, dyq, dyk = inputs(shape, BF16)
    def call(**more):
        return pkg.spa_norm_rope_bwd(dyq, q, wq, table, pos, dk_out=dyk, k=k, wk=wk, eps=EPS, **more)
    ref = call()
    ws = torch.empty(pkg.spa_norm_rope_bwd_workspace_size(96), dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(ref, call(workspace=ws)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    outs = [torch.empty_like(t) for t in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(workspace=ws, dq=outs[0], dk=outs[1], dwq=outs[2], dwk=outs[3])
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))
    with pytest.raises(pkg.SpaError):
        call(workspace=ws[:256])


@pytest.mark.parametrize("causal", [False, True])
def test_training_step(causal):
    """norm_rope, the attention and both backward passes against 64-bit derivatives of the whole."""
    pkg = spa()
    B, H, N, d, m, dv = 2, 2, 200, 64, 32, 64
    g = gen(11)
    q, k, v = (randn(g, B, H, N, w, dtype=BF16) for w in (d, d, dv))
    wq, wk = ((1 + 0.2 * randn(g, d)).to(BF16) for _ in range(2))
    P = (randn(g, H, d, m) / math.sqrt(m)).to(BF16)
    dO = randn(g, B, H, N, dv, dtype=BF16)
    freq = pkg.rope_frequencies(d)
    table = pkg.rope_table(freq)
    pos = torch.arange(N, device="cuda", dtype=I32).expand(B, N).contiguous()
    qn, kn = pkg.spa_norm_rope(q, wq, table, pos, k=k, wk=wk, eps=EPS)
    out, lse = pkg.spa_attention_fwd_lse(qn, kn, v, P, causal=causal)
    dqn, dkn, dvv, dP = pkg.spa_attention_bwd_lse(qn, kn, v, P, out, lse, dO, causal=causal)
    dq, dk, dwq, dwk = pkg.spa_norm_rope_bwd(dqn.to(BF16), q, wq, table, pos, dk_out=dkn.to(BF16), k=k, wk=wk, eps=EPS)
    x = [t.double().requires_grad_() for t in (q, k, wq, wk)]
    a, b = (reference(t, w, freq, pos, False)[0] for t, w in ((x[0], x[2]), (x[1], x[3])))
    s = (a @ P.double()) @ (b @ P.double()).transpose(-1, -2) / math.sqrt(m)
    if causal:
        s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -math.inf)
    ref = torch.autograd.grad(torch.softmax(s, -1) @ v.double(), x, dO.double())
    # the attention's own gradients are held to a relative 2-norm of 2e-2, and normed queries and keys in
    # bf16 are off by 2^-8, a logit of up to about 30 by 0.1 where one feature carries it: 5e-2 in all
    for got, want in zip((dq, dk, dwq, dwk), ref):
        assert float((got.double() - want).norm() / want.norm()) < 5e-2


def odd_rows(x):
    """x with rows whose addresses no vector fits: one feature between them."""
    B, H, N, d = x.shape
    y = torch.empty(B, H, N, d + 1, dtype=x.dtype, device="cuda")[..., :d]
    return y.copy_(x)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d, odd", [(96, False), (80, False), (200, False), (33, False), (96, True), (128, False)])
def test_a_row_that_is_not_finite_stays_alone(d, odd, dtype, interleaved):
    """NaN and infinities in one head's row reach no other row, forward or backward: the others keep their bits."""
    B, H, Hk, N, rot = 2, 9, 8, 10007, 32
    g = gen(d + odd)
    pkg = spa()
    table = pkg.rope_table(pkg.rope_frequencies(rot))
    q, k = (randn(g, B, h, N, d, dtype=dtype) for h in (H, Hk))
    dq_out, dk_out = randn(g, B, H, N, d, dtype=dtype), randn(g, B, Hk, N, d, dtype=dtype)
    w = (1 + 0.3 * randn(g, d)).to(dtype)
    bad = [(0, 0, 0), (1, 2, N - 1), (0, 1, 77), (1, 5, 4096)]  # (sequence, head, token)
    values = (math.nan, math.inf, -math.inf, math.nan)

    def calls(q, k):
        if odd:
            q, k = odd_rows(q), odd_rows(k)
        return (*pkg.spa_norm_rope(q, w, table, k=k, wk=w, interleaved=interleaved),
                *pkg.spa_norm_rope_bwd(dq_out, q, w, table, dk_out=dk_out, k=k, wk=w, interleaved=interleaved)[:2])

    want = calls(q, k)
    for (b, h, n), x in zip(bad, values):
        for t in (q, k):
            t[b, h, n, 3] = x
    got = calls(q, k)
    for x, y in zip(got, want):
        for b, h, n in bad:
            assert bool(x[b, h, n].isnan().any())
            x[b, h, n] = y[b, h, n] = 0
        assert torch.equal(x, y)
