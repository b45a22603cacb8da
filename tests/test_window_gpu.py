"""Attention under a sliding window with first keys that stay visible, forward and
gradients, on the GPU against 64-bit arithmetic."""
import math
import time

import pytest
import torch

from helpers import BF16_MAX_ABS, BF16_REL_F, spa

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert spa().device_error() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, *shape):
    """Rows of norm sqrt(d)."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * (math.sqrt(shape[-1]) / x.norm(dim=-1, keepdim=True))).to(BF16)


def inputs(B, H, Hk, N, d, m, dv, seed=0):
    g = gen(seed + N + d + m)
    q, k = rows(g, B, H, N, d), rows(g, B, Hk, N, d)
    v = torch.randn(B, Hk, N, dv, generator=g, device="cuda").to(BF16)
    P = (torch.randn(Hk, d, m, generator=g, device="cuda") / math.sqrt(m)).to(BF16)
    dO = torch.randn(B, H, N, dv, generator=g, device="cuda").to(BF16)
    return q, k, v, P, dO


def seen(N, window, sink):
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")
    s = j <= i
    return s & ((i - j < window) | (j < sink)) if window else s


def reference(q, k, v, P, dO, window, sink):
    """out, lse and the gradients in 64 bits."""
    B, H, N, d = q.shape
    Hk, _, m = P.shape
    G = H // Hk
    x = [t.double().requires_grad_() for t in (q, k, v, P)]
    qp = (x[0].view(B, Hk, G, N, d) @ x[3][:, None]).reshape(B, H, N, m)
    kp = (x[1] @ x[3]).repeat_interleave(G, 1)
    s = (qp @ kp.transpose(-1, -2) / math.sqrt(m)).masked_fill(~seen(N, window, sink), -math.inf)
    out = torch.softmax(s, -1) @ x[2].repeat_interleave(G, 1)
    return out.detach(), torch.logsumexp(s, -1).detach(), torch.autograd.grad(out, x, dO.double())


def check_out(got, ref):
    """The forward's own tolerances, and the rounding of the output to bf16."""
    d = got.double() - ref
    assert float(d.norm() / ref.norm()) <= BF16_REL_F + 2.0 ** -8
    assert float((d.abs() - 2.0 ** -8 * ref.abs()).max()) <= BF16_MAX_ABS


def check_grads(got, ref):
    # the fused backward's products take bf16 operands with relative roundings of 2^-8 each: P, dS, Q~, K~, and the
    # output's own; a relative 2-norm of 2e-2 is what the backward is held to
    for name, a, b in zip(("dq", "dk", "dv", "dP"), got, ref):
        assert a.dtype == BF16 and bool(a.isfinite().all()), name
        rel = float((a.double() - b).norm() / b.norm().clamp(min=1e-30)) if float(b.norm()) else float(a.double().norm())
        assert rel <= 2e-2, (name, rel)


CASES = [
    # B, H, Hk, N, d, m, dv, window, sink
    (1, 1, 1, 1, 64, 32, 64, 0, 0),
    (2, 2, 1, 3, 128, 16, 128, 1, 4),
    (1, 2, 2, 127, 64, 64, 64, 5, 0),
    (1, 2, 1, 128, 64, 32, 128, 128, 1),
    (1, 3, 1, 129, 128, 32, 64, 128, 0),
    (2, 4, 2, 300, 64, 16, 64, 129, 1),
    (1, 2, 1, 640, 128, 64, 128, 2, 3),        # whole tiles that a row does not see
    (1, 4, 4, 640, 64, 32, 64, 100, 0),
    (1, 6, 2, 1021, 64, 64, 64, 300, 130),     # first keys of more than a tile
    (1, 2, 1, 1100, 128, 16, 128, 256, 600),
    (1, 8, 1, 900, 128, 32, 128, 127, 64),
    (3, 5, 1, 513, 64, 32, 128, 0, 0),         # no window: causal
    (1, 4, 2, 700, 128, 32, 64, 699, 2),
    (1, 4, 2, 700, 128, 32, 64, 700, 2),
    (1, 2, 1, 384, 64, 64, 128, 64, 2**31 - 1),
    (1, 2, 1, 3000, 64, 32, 64, 200, 7),
]


@pytest.mark.parametrize("case", CASES)
def test_window(case):
    B, H, Hk, N, d, m, dv, window, sink = case
    pkg = spa()
    q, k, v, P, dO = inputs(B, H, Hk, N, d, m, dv)
    lse, lo = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, dv, dtype=BF16, device="cuda")
    out = pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink, out_lo=lo, lse=lse)
    ref, ref_lse, grads = reference(q, k, v, P, dO, window, min(sink, N))
    check_out(out, ref)
    # a logit of fp16 (or split bf16) operands is off by 2^-10 of the terms it sums at most, the log-sum-exp
    # no more than its largest logit's error
    size = (q.double().abs().view(B, Hk, H // Hk, N, d) @ P.double().abs()[:, None]).amax() * (
        k.double().abs() @ P.double().abs()).amax() * math.sqrt(m)
    assert float((lse.double() - ref_lse).abs().max()) <= 2.0 ** -10 * float(size)
    check_grads(pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, window=window, sink=sink), grads)
    # without what the gradient needs: other roundings; the same bits each time
    again = pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink)
    check_out(again, ref)
    assert torch.equal(again, pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink))


@pytest.mark.parametrize("case", [(40, 32, 32, 128, 0, 0), (41, 32, 16, 77, 9, 2), (700, 4, 2, 1, 0, 0),
                                  (5, 48, 8, 1400, 300, 4)])
def test_many_items_of_one_key_tile(case):
    """More items than blocks, whose scores take one key tile, alone or between longer ones."""
    B, H, Hk, N, window, sink = case
    pkg = spa()
    q, k, v, P, dO = inputs(B, H, Hk, N, 64, 32, 64)
    lse, lo = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, 64, dtype=BF16, device="cuda")
    ref = None
    for _ in range(20):
        got = (pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink),
               pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink, out_lo=lo, lse=lse), lo, lse)
        assert pkg.device_error() == 0
        if ref is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        ref = [t.clone() for t in got]
    b = B - 1
    want = reference(q[b:], k[b:], v[b:], P, dO[b:], window, sink)[0]
    check_out(ref[0][b:], want)
    check_out(ref[1][b:], want)


@pytest.mark.parametrize("m", [16, 32, 64])
def test_without_window_is_the_causal_forward(m):
    """One key head per query head and no window: the causal forward."""
    pkg = spa()
    q, k, v, P, dO = inputs(2, 3, 3, 1500, 128, m, 128)
    lse, lo = torch.empty(2, 3, 1500, device="cuda"), torch.empty(2, 3, 1500, 128, dtype=BF16, device="cuda")
    out = pkg.spa_attention_window_fwd(q, k, v, P, out_lo=lo, lse=lse)
    want, want_lse = pkg.spa_attention_fwd_lse(q, k, v, P, causal=True)
    # without what the gradient needs, the forward's bits, rounded
    assert torch.equal(pkg.spa_attention_window_fwd(q, k, v, P), want.to(BF16))
    # with it, the same scores and other roundings of the probabilities: 2^-8 of a term either way
    assert float((out.double() + lo.double() - want.double()).norm() / want.double().norm()) <= 2.0 ** -7
    assert bool((lo.double().abs() <= 2.0 ** -8 * out.double().abs() + 1e-30).all())
    assert float((lse - want_lse).abs().max()) <= 2.0 ** -8
    # every key among the first ones, and a window as long as the sequence: the same
    for more in (dict(window=1, sink=1500), dict(window=1500), dict(window=2**31 - 1, sink=2**31 - 1)):
        got = pkg.spa_attention_window_fwd(q, k, v, P, **more)
        check_out(got, want.double())


def test_a_window_of_one():
    """Each query sees its own key alone: the output is its value, and only dv is not zero."""
    pkg = spa()
    q, k, v, P, dO = inputs(1, 2, 2, 777, 64, 32, 64)
    lse, lo = torch.empty(1, 2, 777, device="cuda"), torch.empty_like(v)
    out = pkg.spa_attention_window_fwd(q, k, v, P, window=1, out_lo=lo, lse=lse)
    # p v / p: the reciprocal and the product are off by 2^-24 of the value each
    assert torch.equal(out, v) and bool((lo.double().abs() <= 2.0 ** -22 * v.double().abs()).all())
    dq, dk, dv, dP = pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, window=1)
    # the sum is that of the rounded probability, which is 2^-8 off the exponential; their quotient is rounded
    # again for the product, and the gradient itself: 3 x 2^-8
    assert bool(((dv.double() - dO.double()).abs() <= 3 * 2.0 ** -8 * dO.double().abs()).all())
    # dS = P (dP - D) is the difference of two fp32 sums of 64 products
    most = float((dO.double().abs() * v.double().abs()).sum(-1).max()) * 64 * 2.0 ** -22
    for g, other in ((dq, k), (dk, q)):
        size = float((other.double().abs() @ P.double().abs()).max() * P.double().abs().sum(-1).max())
        assert float(g.double().abs().max()) <= most * size


def test_extreme_input_ranges():
    """Queries and keys far from 1 with the same logits: score operands carry range exponents."""
    pkg = spa()
    q, k, v, P, dO = inputs(1, 4, 2, 400, 64, 32, 64)
    ref, _, _ = reference(q, k, v, P, dO, 70, 3)
    for e in (24, -24):
        out = pkg.spa_attention_window_fwd((q.float() * 2.0 ** e).to(BF16), (k.float() * 2.0 ** -e).to(BF16), v, P,
                                           window=70, sink=3)
        check_out(out, ref)


def test_scores_that_grow():
    """Logits that rise along the sequence, so that every tile moves the maximum, and fall."""
    pkg = spa()
    q, k, v, P, dO = inputs(1, 2, 1, 1200, 64, 32, 64)
    for up in (1, -1):
        ramp = torch.linspace(0.05, 6.0, 1200, device="cuda")[::up].contiguous() if up == 1 else torch.linspace(
            6.0, 0.05, 1200, device="cuda")
        kk = (q[:, :1].float() * ramp[:, None]).to(BF16)
        ref, _, _ = reference(q, kk, v, P, dO, 500, 10)
        out = pkg.spa_attention_window_fwd(q, kk, v, P, window=500, sink=10)
        d = out.double() - ref
        # logits of up to 6 |q~|^2 / sqrt(m) = 6 * 64 / 5.7: 2^-10 of their terms is 0.07
        assert float(d.norm() / ref.norm()) <= 0.1


def test_gradients_against_differences():
    """dv is linear: exact up to rounding; dq, dk, dP along a direction, from 64-bit losses of the 64-bit forward."""
    pkg = spa()
    B, H, Hk, N, d, m, dv, window, sink = 1, 4, 2, 260, 64, 32, 64, 90, 5
    q, k, v, P, dO = inputs(B, H, Hk, N, d, m, dv, seed=3)
    lse, lo = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, dv, dtype=BF16, device="cuda")
    out = pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink, out_lo=lo, lse=lse)
    grads = pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, window=window, sink=sink)
    h = 2.0 ** -12
    for i, x in enumerate((q, k, v, P)):
        # along the gradient itself: |g|^2, the direction in which a wrong gradient shows
        dirn = grads[i].double() / grads[i].double().norm()
        loss = []
        for s in (h, -h):
            args = [t.double() for t in (q, k, v, P)]
            args[i] = args[i] + s * dirn
            loss.append(float((reference(*args, dO, window, sink)[0] * dO.double()).sum()))
        found = (loss[0] - loss[1]) / (2 * h)
        # the gradient's own 2e-2, and h^2 of the third derivative, which is nothing at this h
        assert abs(found - float(grads[i].double().norm())) <= 2.1e-2 * abs(found)


def test_training_step():
    """Norms with positions, the windowed attention and both backward passes, captured, against 64-bit derivatives of
    the whole."""
    pkg = spa()
    B, H, Hk, N, d, m, dv, window, sink = 2, 4, 2, 400, 64, 32, 64, 90, 3
    g = gen(12)
    q, k, v = (torch.randn(B, h, N, w, generator=g, device="cuda").to(BF16) for h, w in ((H, d), (Hk, d), (Hk, dv)))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(BF16) for _ in range(2))
    P = (torch.randn(Hk, d, m, generator=g, device="cuda") / math.sqrt(m)).to(BF16)
    dO = torch.randn(B, H, N, dv, generator=g, device="cuda").to(BF16)
    freq = pkg.rope_frequencies(d)
    table = pkg.rope_table(freq)
    pos = torch.arange(N, device="cuda", dtype=torch.int32).expand(B, N).contiguous()
    lse, lo = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, dv, dtype=BF16, device="cuda")
    call = dict(window=window, sink=sink)

    def step():
        qn, kn = pkg.spa_norm_rope(q, wq, table, pos, k=k, wk=wk)
        out = pkg.spa_attention_window_fwd(qn, kn, v, P, out_lo=lo, lse=lse, **call)
        dqn, dkn, dvv, dP = pkg.spa_attention_window_bwd(qn, kn, v, P, out, lo, lse, dO, **call)
        return *pkg.spa_norm_rope_bwd(dqn, q, wq, table, pos, dk_out=dkn, k=k, wk=wk), dvv, dP

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dq, dk, dwq, dwk, dvv, dP = step()
    graph.replay()
    x = [t.double().requires_grad_() for t in (q, k, wq, wk, v, P)]
    ang = pos.double()[:, None, :, None] * freq.to("cuda")

    def normed(t, w):
        y = t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)

    qp = (normed(x[0], x[2]).view(B, Hk, H // Hk, N, d) @ x[5][:, None]).reshape(B, H, N, m)
    kp = (normed(x[1], x[3]) @ x[5]).repeat_interleave(H // Hk, 1)
    s = (qp @ kp.transpose(-1, -2) / math.sqrt(m)).masked_fill(~seen(N, window, sink), -math.inf)
    ref = torch.autograd.grad(torch.softmax(s, -1) @ x[4].repeat_interleave(H // Hk, 1), x, dO.double())
    # the attention's own gradients are held to a relative 2-norm of 2e-2, and normed queries and keys in
    # bf16 are off by 2^-8, a logit of up to about 30 by 0.1 where one feature carries it: 5e-2 in all
    for got, want in zip((dq, dk, dwq, dwk, dvv, dP), ref):
        assert float((got.double() - want).norm() / want.norm()) < 5e-2


def test_streams_workspace_and_graphs():
    """A workspace of the caller's, another stream, and two captured graphs beside eager calls."""
    pkg = spa()
    sizes = (2, 4, 2, 600, 128, 32, 64)
    q, k, v, P, dO = inputs(*sizes)
    call = dict(window=150, sink=9)
    lse, lo = torch.empty(2, 4, 600, device="cuda"), torch.empty(2, 4, 600, 64, dtype=BF16, device="cuda")
    ref = pkg.spa_attention_window_fwd(q, k, v, P, out_lo=lo, lse=lse, **call)
    grads = pkg.spa_attention_window_bwd(q, k, v, P, ref, lo, lse, dO, **call)
    need = [pkg.spa_attention_window_workspace_size(2, 4, 2, 600, 128, 32, 64, 150, 9, g) for g in (False, True)]
    assert 0 < need[0] < need[1]
    with pytest.raises(pkg.SpaError):
        pkg.spa_attention_window_fwd(q, k, v, P, workspace=torch.empty(need[0] - 1, dtype=torch.uint8, device="cuda"),
                                     **call)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [torch.empty(need[1], dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = pkg.spa_attention_window_fwd(q, k, v, P, workspace=ws[0], stream=side, **call)
    side.synchronize()
    assert torch.equal(got, pkg.spa_attention_window_fwd(q, k, v, P, **call))
    outs, graphs = [], []
    for w in ws:
        out, lo2, l2 = torch.empty_like(ref), torch.empty_like(ref), torch.empty_like(lse)
        g2 = [torch.empty_like(t) for t in (q, k, v, P)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.spa_attention_window_fwd(q, k, v, P, out=out, out_lo=lo2, lse=l2, workspace=w, **call)
            pkg.spa_attention_window_bwd(q, k, v, P, out, lo2, l2, dO, grads=g2, workspace=w, **call)
        outs.append((out, g2))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for out, g2 in outs:
        assert torch.equal(out, ref)
        for a, b in zip(g2, grads):  # fp32 sums in another order, before one rounding to bf16
            assert float((a.double() - b.double()).norm() / b.double().norm()) <= 2.0 ** -8


def test_decode_gives_the_last_row():
    """The rows that the decode over pages gives with the same window are the prompt's."""
    pkg = spa()
    B, H, Hk, N, d, m, dv, window, sink = 2, 8, 2, 500, 64, 32, 64, 120, 3
    q, k, v, P, _ = inputs(B, H, Hk, N, d, m, dv)
    out = pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink)
    kc, mul = pkg.kcache_new(B, Hk, N, m)
    vc = torch.zeros(B, Hk, N, dv, dtype=BF16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pkg.spa_kcache_append_ragged(k, v, P, kc, mul, vc, i32(0, 0))
    pages = pkg.kcache8_new(16, Hk, m, dv)
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8).contiguous()
    last = q[:, :, -1].contiguous()
    got = pkg.spa_attention_decode8(last, P, pages, table, i32(0, 0), kc, mul, vc, i32(N, N), window=window, sink=sink)
    check_out(got, out[:, :, -1].double())
    lens, blocks = i32(N, N), i32(0, 0)
    pkg.spa_kcache8_pack(kc, mul, vc, lens, pages, table, blocks)
    assert lens.tolist() == [N % 64] * 2
    got = pkg.spa_attention_decode8(last, P, pages, table, blocks, kc, mul, vc, lens, window=window, sink=sink)
    # e4m3 K~ and V are off by 2^-4 of a value at most: a mean over many of them by far less than that
    assert float((got.double() - out[:, :, -1].double()).norm() / out[:, :, -1].double().norm()) <= 2.0 ** -3


@pytest.mark.parametrize("kernel", [0, 1])
def test_a_withheld_arrival_is_reported(kernel):
    """The kernels' bounded waits: every block withholds its first "scores ready", the waits give up after 50 ms,
    and a call afterwards is right."""
    pkg = spa()
    assert pkg.device_error() == 0
    t0 = time.perf_counter()
    assert pkg.selftest_window_wait_timeout(50, kernel) == pkg.SPA_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 1.5
    assert pkg.device_error() == 0
    q, k, v, P, dO = inputs(1, 4, 2, 700, 64, 32, 64)
    lse, lo = torch.empty(1, 4, 700, device="cuda"), torch.empty_like(dO)
    out = pkg.spa_attention_window_fwd(q, k, v, P, window=150, sink=3, out_lo=lo, lse=lse)
    ref, _, grads = reference(q, k, v, P, dO, 150, 3)
    check_out(out, ref)
    check_grads(pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, window=150, sink=3), grads)


def test_two_calls_at_once():
    """Forwards and gradients on two streams at the same time: the results of calls alone."""
    pkg = spa()
    sets = [inputs(1, 8, 4, 1500, 64, 32, 64, seed=s) for s in (1, 2)]
    call = dict(window=200, sink=5)

    def step(q, k, v, P, dO):
        lse, lo = torch.empty(1, 8, 1500, device="cuda"), torch.empty_like(dO)
        out = pkg.spa_attention_window_fwd(q, k, v, P, out_lo=lo, lse=lse, **call)
        return out, lo, lse, *pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, **call)

    alone = [step(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for stream, x in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append([step(*x) for _ in range(3)])
        torch.cuda.synchronize()
        for steps, ref in zip(got, alone):
            for one in steps:
                assert all(torch.equal(a, b) for a, b in zip(one[:3], ref[:3]))
                for a, b in zip(one[3:], ref[3:]):  # fp32 sums in another order, before one rounding to bf16
                    assert float((a.double() - b.double()).norm() / b.double().norm()) <= 2.0 ** -8


def test_key_heads_without_queries():
    """No query head on two key heads: their gradients are zero, and are written."""
    pkg = spa()
    q, k, v, P, dO = inputs(2, 0, 2, 130, 64, 32, 128)
    out, lo = (torch.empty(2, 0, 130, 128, dtype=BF16, device="cuda") for _ in range(2))
    lse = torch.empty(2, 0, 130, device="cuda")
    grads = [torch.full_like(t, math.nan) for t in (q, k, v, P)]
    got = pkg.spa_attention_window_bwd(q, k, v, P, out, lo, lse, dO, window=9, sink=1, grads=grads)
    assert [t.shape for t in got] == [t.shape for t in (q, k, v, P)]
    assert not any(bool(t.any()) for t in got)  # NaN counts as true


@pytest.mark.parametrize("case", CASES)
def test_log_sum_exp_of_each_row(case):
    """Each row's log-sum-exp against a bound of its own terms."""
    B, H, Hk, N, d, m, dv, window, sink = case
    pkg = spa()
    q, k, v, P, _ = inputs(B, H, Hk, N, d, m, dv)
    lse, lo = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, dv, dtype=BF16, device="cuda")
    pkg.spa_attention_window_fwd(q, k, v, P, window=window, sink=sink, out_lo=lo, lse=lse)
    x, y, p = q.double().view(B, Hk, H // Hk, N, d), k.double()[:, :, None], P.double()[:, None]
    root, see = math.sqrt(m), seen(N, window, min(sink, N))
    dot = lambda a, b: (a @ b.transpose(-1, -2) / root).masked_fill(~see, -math.inf)  # noqa: E731
    s = dot(x @ p, y @ p)
    # A logit: both operands rounded to fp16 (or to three bf16 parts), 2^-11 of a term each; the projections' sums of
    # d products in fp32 and the logit's of m, with ten roundings of scales and exponents, 2^-24 each of the largest
    # that the magnitudes give.  The log-sum-exp is off by no more than a logit of the row; the weights in its sum are
    # rounded to bf16, half a step 2^-8 of each, and a sum of N and the logarithm add N + 8 roundings.
    terms = dot((x @ p).abs(), (y @ p).abs()).amax(-1)
    sizes = dot(x.abs() @ p.abs(), y.abs() @ p.abs()).amax(-1)
    tol = 2.0 ** -10 * terms + (2 * d + m + 10) * 2.0 ** -24 * sizes + 2.0 ** -8 + (N + 8) * 2.0 ** -24
    ref = torch.logsumexp(s, -1)
    tol = tol + 2.0 ** -23 * ref.abs()
    over = ((lse.double().view(ref.shape) - ref).abs() - tol).max()
    assert float(over) <= 0, float(over)
