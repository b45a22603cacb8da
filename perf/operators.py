"""The serving operators around the projected key cache, in plain form and as the library computes them.

Four operators that a decode loop calls one after the other:

  rope     rotary positions on the queries and keys, before they are projected (and the gradient of that)
  append   new keys projected into a ragged cache, with their value rows: K~ = K P_h as fp16 rows with one
           power-of-two multiplier per row
  decode   one query per sequence and head against a prefix that the whole batch shares and the sequence's
           own cache rows, the two joined in one softmax; on request the attention weight of every cache row
           is added to its running sum
  evict    the cache rows of smallest accumulated weight leave the cache, in place

`own` false: elementary torch operations in 32 bits or more.  `own` true: the library's calls.
"""
import math

import torch

own = False

LOG2_64 = 2.0 ** 64


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # rotary positions of one decode step: 64 sequences at their own far positions, 32 query and 8 key heads
        dict(name="rope step", op="rope", B=64, H=32, G=4, N=1, d=128, rot=128, interleaved=False, factor=1.0,
             far=131072, inverse=False, dtype="bf16"),
        # a prompt chunk as the fused q/k/v product leaves it (token-major), half of each head rotated, positions
        # interpolated by 4 for a long context
        dict(name="rope prompt", op="rope", B=2, H=16, G=4, N=8192, d=128, rot=64, interleaved=True, factor=4.0,
             far=8192, inverse=False, dtype="bf16"),
        # the gradient of the same in fp32, at an odd length and an odd head width
        dict(name="rope gradient", op="rope", B=1, H=12, G=3, N=8191, d=96, rot=96, interleaved=False, factor=1.0,
             far=262144, inverse=True, dtype="f32"),
        # the new key and value rows of one decode step, 64 sequences
        dict(name="append step", op="append", B=64, H=8, T=1, d=128, m=32, dv=128, cap=1024),
        # a ragged batch of prompts into the cache
        dict(name="append prompts", op="append", B=4, H=8, T=4095, d=128, m=32, dv=128, cap=4608),
        # the smallest call: one sequence, a few hundred keys, no prefix, no shared heads
        dict(name="decode small", op="decode", B=1, H=8, G=1, d=64, m=16, dv=64, prefix=0, lo=300, hi=300, cap=512,
             weights=False),
        # a batch on one long system prompt, with short sequences of its own
        dict(name="decode prefix", op="decode", B=32, H=32, G=4, d=128, m=32, dv=128, prefix=32768, lo=1, hi=511,
             cap=512, weights=False),
        # ragged sequences without a prefix, with the weights that the eviction goes by
        dict(name="decode weights", op="decode", B=16, H=16, G=4, d=128, m=32, dv=128, prefix=0, lo=17, hi=8191,
             cap=8192, weights=True),
        # many sequences on a very long prefix: the matrix products decide
        dict(name="decode large", op="decode", B=128, H=32, G=4, d=128, m=64, dv=128, prefix=65536, lo=0, hi=2047,
             cap=2048, weights=True),
        # a cache at its budget: one row more than it may hold, every step
        dict(name="evict step", op="evict", B=64, H=8, m=32, dv=128, lo=2049, hi=2049, cap=2304, budget=2048, sink=4,
             recent=128),
        # prompts cut down to their budget once they are read
        dict(name="evict prompts", op="evict", B=8, H=8, m=64, dv=128, lo=1000, hi=16383, cap=16384, budget=4096,
             sink=16, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    if op == "rope":
        G = rng.choice([1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([32, 64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = max(1, int(1e8) // ((H + H // G) * d * (2 if dtype == "bf16" else 4)))  # tokens
        N = _log(rng, 1, min(8192, most))
        B = _log(rng, 1, max(1, min(64, most // N)))
        return dict(op=op, B=B, H=H, G=G, N=N, d=d, rot=2 * rng.randint(1, d // 2), interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 1.0, 2.5, 8.0]), far=_log(rng, N + 1, 1 << 20),
                    inverse=rng.random() < 0.4, dtype=dtype)
    d = rng.choice([32, 64, 96, 128, 200])
    m = rng.choice([16, 32, 32, 64, 128])
    dv = rng.choice([64, 128])
    if op == "append":
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(96, 16384 // T)))
        return dict(op=op, B=B, H=rng.choice([1, 2, 3, 8]), T=T, d=d, m=m, dv=dv, cap=T + rng.randint(0, 600))
    if op == "decode":
        hi = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(128, 131072 // max(hi, 1024))))
        G = rng.choice([1, 2, 4, 5, 8])
        H = G * rng.choice([1, 2, 4, 8])
        most = min(60000, int(4e10) // (B * H * (m + dv)))  # keys
        prefix = 0 if rng.random() < 0.3 or most < 1 else _log(rng, 1, most)
        return dict(op=op, B=B, H=H, G=G, d=d, m=m, dv=dv, prefix=prefix, lo=rng.randint(0, hi), hi=hi,
                    cap=hi + rng.randint(0, 100), weights=rng.random() < 0.5)
    hi = _log(rng, 64, 16384)
    B = _log(rng, 1, max(1, min(64, 131072 // hi)))
    budget = rng.randint(32, hi)
    sink = rng.randint(0, budget // 4)
    return dict(op=op, B=B, H=rng.choice([1, 2, 3, 8]), m=m, dv=dv, lo=rng.randint(1, hi), hi=hi,
                cap=hi + rng.randint(0, 100), budget=budget, sink=sink, recent=rng.randint(0, budget // 2))


def _lengths(lo, hi, B):
    """B lengths spread evenly over lo..hi: the same ones for every seed, in an order of its own."""
    return [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)] if B > 1 else [hi]


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _rows(g, *shape):
    """Rows of norm sqrt(d), as a normalisation layer leaves them, in bf16."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * (math.sqrt(shape[-1]) / x.norm(dim=-1, keepdim=True))).to(torch.bfloat16)


def _projection(g, H, d, m):
    return (torch.randn((H, d, m), generator=g, device="cuda") / math.sqrt(m)).to(torch.bfloat16)


def _key_rows(g, *shape, d):
    """Cache rows of projected keys: entries of variance d/m, fp16 bits and one multiplier per row."""
    m = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda") * math.sqrt(d / m)
    e = torch.frexp(x.abs().amax(dim=-1))[1] - 14
    mul = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (x / mul[..., None]).to(torch.float16).view(torch.int16), mul


def _shuffled_lengths(g, c):
    n = torch.tensor(_lengths(c["lo"], c["hi"], c["B"]), device="cuda", dtype=torch.int32)
    return n[torch.randperm(c["B"], generator=g, device="cuda")].contiguous()


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, H, N, d = c["B"], c["H"], c["N"], c["d"]
        Hk = H // c["G"]
        # one token-major buffer [B][N][H + Hk][d], as the product with the stacked weights leaves it
        x = _normal(g, B, N, H + Hk, d, dtype=dt)
        s["q"] = x[:, :, :H].permute(0, 2, 1, 3)
        s["k"] = x[:, :, H:].permute(0, 2, 1, 3)
        first = torch.randint(0, max(1, c["far"] - N), (B, 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2.0 * i / c["rot"]) / c["factor"]
        # the library's table: the advance per position, in units of 2^-64 turns
        s["table"] = (s["freq"] / (2.0 * math.pi) * LOG2_64).round().to(torch.int64)
        s["q_out"] = torch.empty((B, H, N, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((B, Hk, N, d), dtype=dt, device="cuda")
    elif c["op"] == "append":
        B, H, T = c["B"], c["H"], c["T"]
        s["k"] = _rows(g, B, H, T, c["d"])
        s["v"] = _normal(g, B, H, T, c["dv"], dtype=torch.bfloat16)
        s["P"] = _projection(g, H, c["d"], c["m"])
        s["pos"] = torch.randint(0, c["cap"] - T + 1, (B,), generator=g, device="cuda").to(torch.int32)
        n = torch.tensor(_lengths((T + 1) // 2, T, B), device="cuda", dtype=torch.int32)
        s["count"] = n[torch.randperm(B, generator=g, device="cuda")].contiguous()
        s["kc"] = torch.zeros((B, H, c["cap"], c["m"]), dtype=torch.int16, device="cuda")
        s["mul"] = torch.zeros((B, H, c["cap"]), dtype=torch.float32, device="cuda")
        s["vc"] = torch.zeros((B, H, c["cap"], c["dv"]), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "decode":
        B, H, Hk, cap, d, m, dv = c["B"], c["H"], c["H"] // c["G"], c["cap"], c["d"], c["m"], c["dv"]
        s["q"] = _rows(g, B, H, d)
        s["P"] = _projection(g, Hk, d, m)
        s["kc"], s["mul"] = _key_rows(g, B, Hk, cap, m, d=d)
        s["vc"] = _normal(g, B, Hk, cap, dv, dtype=torch.bfloat16)
        s["len"] = _shuffled_lengths(g, c)
        s["prefix"] = None
        if c["prefix"]:
            kc, mul = _key_rows(g, Hk, c["prefix"], m, d=d)
            s["prefix"] = (kc, mul, _normal(g, Hk, c["prefix"], dv, dtype=torch.bfloat16))
        s["out"] = torch.empty((B, H, dv), dtype=torch.bfloat16, device="cuda")
        s["acc"] = s["acc_out"] = None
        if c["weights"]:
            # some steps' worth of weight already on every row
            s["acc"] = torch.rand((B, Hk, cap), generator=g, device="cuda") * 0.02
            s["acc_out"] = torch.zeros_like(s["acc"])
    else:
        B, H, cap = c["B"], c["H"], c["cap"]
        s["kc"], s["mul"] = _key_rows(g, B, H, cap, c["m"], d=128)
        s["vc"] = _normal(g, B, H, cap, c["dv"], dtype=torch.bfloat16)
        # accumulated weights: a few rows hold most of it, and rows of equal weight are there too
        a = torch.rand((B, H, cap), generator=g, device="cuda")
        s["acc"] = torch.floor(a ** 6 * 65536.0) / 4096.0
        s["len"] = _shuffled_lengths(g, c)
        # the rows stand in an order that earlier evictions left: positions are distinct, not sorted
        s["row_pos"] = torch.argsort(torch.rand((B, H, cap), generator=g, device="cuda"), dim=-1).to(torch.int32)
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["row_pos_out"] = torch.zeros_like(s["row_pos"])
        s["len_out"] = torch.zeros_like(s["len"])
        s["src"] = torch.zeros((B, H, c["budget"]), dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    # far positions: the angle is formed in 64 bits
    angle = s["pos"].double()[:, None, :, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        return torch.cat((r, y[..., rot:]), dim=-1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _plain_append(s):
    c = s["case"]
    # the multiplier turns on whether the row's largest value reaches a power of two: 64 bits
    x = torch.matmul(s["k"].double(), s["P"].double())
    top = x.abs().amax(dim=-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 14, torch.zeros_like(top, dtype=torch.int32))
    mul = torch.ldexp(torch.ones_like(top), e)
    rows = (x / mul[..., None]).to(torch.float16).view(torch.int16)
    t = torch.arange(c["T"], device="cuda")
    b, t = torch.nonzero(t[None, :] < s["count"][:, None], as_tuple=True)
    at = (s["pos"].long()[b] + t)
    s["kc"][b, :, at] = rows[b, :, t]
    s["mul"][b, :, at] = mul.float()[b, :, t]
    s["vc"][b, :, at] = s["v"][b, :, t]
    return s["kc"].view(torch.float16), s["mul"], s["vc"]


def _plain_decode(s):
    c = s["case"]
    B, H, G, cap, m, dv = c["B"], c["H"], c["G"], c["cap"], c["m"], c["dv"]
    Hk = H // G
    q = torch.matmul(s["q"].float().view(B, Hk, G, c["d"]), s["P"].float()) / math.sqrt(m)
    inside = torch.arange(cap, device="cuda")[None, :] < s["len"][:, None]
    k = s["kc"].view(torch.float16).float() * s["mul"][..., None]
    scores = torch.matmul(q, k.transpose(-1, -2)).masked_fill(~inside[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    if c["prefix"]:
        kp, mp, vp = s["prefix"]
        k = kp.view(torch.float16).float() * mp[..., None]
        qp = q.transpose(0, 1).reshape(Hk, B * G, m)
        shared = torch.matmul(qp, k.transpose(-1, -2))
        top = torch.maximum(top, shared.amax(dim=-1).view(Hk, B, G, 1).transpose(0, 1))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(dim=-1, keepdim=True)
    out = torch.matmul(e, s["vc"].float())
    if c["prefix"]:
        shared = torch.exp(shared - top.transpose(0, 1).reshape(Hk, B * G, 1))
        total = total + shared.sum(dim=-1).view(Hk, B, G, 1).transpose(0, 1)
        out = out + torch.matmul(shared, vp.float()).view(Hk, B, G, dv).transpose(0, 1)
    some = total > 0
    total = torch.where(some, total, torch.ones_like(total))
    out = (out / total).view(B, H, dv).to(torch.bfloat16)
    if not c["weights"]:
        return out
    weight = (e / total).sum(dim=2)
    return out, torch.where(inside[:, None], s["acc"] + weight, s["acc_out"])


def _plain_evict(s):
    c = s["case"]
    B, H, cap, budget = c["B"], c["H"], c["cap"], c["budget"]
    row = torch.arange(cap, device="cuda").expand(B, H, cap)
    n = s["len"].view(B, 1, 1)
    inside = row < n
    newest = torch.where(inside, s["row_pos"], torch.full_like(s["row_pos"], -1)).amax(dim=-1, keepdim=True)
    safe = (s["row_pos"] < c["sink"]) | (s["row_pos"] > newest - c["recent"])
    rank = torch.where(safe, torch.full_like(s["acc"], math.inf), s["acc"]).masked_fill(~inside, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1]
    left = torch.clamp(n, max=budget)
    kept = torch.zeros((B, H, cap), dtype=torch.bool, device="cuda").scatter(-1, order, (row < left))
    hole, mover = ~kept & (row < left), kept & (row >= left)
    # the i-th hole takes the i-th mover
    at = torch.where(mover, mover.cumsum(dim=-1) - 1, torch.full_like(row, cap))
    movers = torch.zeros((B, H, cap + 1), dtype=torch.int64, device="cuda").scatter(-1, at, row)
    src = torch.where(hole, movers.gather(-1, (hole.cumsum(dim=-1) - 1).clamp(min=0)), row)[..., :budget]
    have = (row < left)[..., :budget]
    for_rows = src[..., None]
    s["kc"][:, :, :budget] = s["kc"].gather(2, for_rows.expand(-1, -1, -1, c["m"]))
    s["vc"][:, :, :budget] = s["vc"].gather(2, for_rows.expand(-1, -1, -1, c["dv"]))
    s["mul"][:, :, :budget] = s["mul"].gather(2, src)
    s["acc_out"][:, :, :budget] = torch.where(have, s["acc"].gather(2, src), s["acc_out"][:, :, :budget])
    s["row_pos_out"][:, :, :budget] = torch.where(have, s["row_pos"].gather(2, src), s["row_pos_out"][:, :, :budget])
    return (s["kc"].view(torch.float16), s["mul"], s["vc"], s["acc_out"], s["row_pos_out"],
            torch.clamp(s["len"], max=budget), torch.where(have, src, torch.full_like(src, -1)).to(torch.int32))


# --------------------------------------------------------------------------- the library's calls
def _own(s):
    import projected_feature_efficient_gb300 as spa
    c = s["case"]
    if c["op"] == "rope":
        return spa.spa_rope(s["q"], s["table"], s["pos"], k=s["k"], rot=c["rot"], interleaved=c["interleaved"],
                            inverse=c["inverse"], out=s["q_out"], k_out=s["k_out"])
    if c["op"] == "append":
        spa.spa_kcache_append_ragged(s["k"], s["v"], s["P"], s["kc"], s["mul"], s["vc"], s["pos"], count=s["count"])
        return s["kc"].view(torch.float16), s["mul"], s["vc"]
    if c["op"] == "decode":
        out = spa.spa_attention_decode_shared(s["q"], s["P"], s["kc"], s["mul"], s["vc"], s["len"],
                                              prefix=s["prefix"], acc=s["acc"], acc_out=s["acc_out"], out=s["out"])
        return (out, s["acc_out"]) if c["weights"] else out
    spa.spa_kcache_evict(s["kc"], s["mul"], s["vc"], s["acc"], s["row_pos"], s["len"], c["budget"], sink=c["sink"],
                         recent=c["recent"], acc_out=s["acc_out"], row_pos_out=s["row_pos_out"],
                         lens_out=s["len_out"], src=s["src"])
    return s["kc"].view(torch.float16), s["mul"], s["vc"], s["acc_out"], s["row_pos_out"], s["len_out"], s["src"]


_PLAIN = dict(rope=_plain_rope, append=_plain_append, decode=_plain_decode, evict=_plain_evict)


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- what each cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * (c["H"] + c["H"] // c["G"]) * c["N"]
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * c["d"] * size + 4 * c["B"] * c["N"] + 4 * c["rot"], flops=3 * n * c["rot"])
    if c["op"] == "append":
        n = c["H"] * sum(_lengths((c["T"] + 1) // 2, c["T"], c["B"]))
        return dict(bytes=n * (2 * c["d"] + 2 * c["m"] + 4 + 4 * c["dv"]) + 2 * c["H"] * c["d"] * c["m"],
                    flops=2 * n * c["d"] * c["m"])
    lens = _lengths(c["lo"], c["hi"], c["B"])
    if c["op"] == "decode":
        Hk, m, dv = c["H"] // c["G"], c["m"], c["dv"]
        rows = Hk * (c["prefix"] + sum(lens))
        pairs = c["H"] * (c["B"] * c["prefix"] + sum(lens))
        size = rows * (2 * m + 4 + 2 * dv) + c["B"] * c["H"] * (2 * c["d"] + 2 * dv) + 2 * Hk * c["d"] * m
        if c["weights"]:
            size += 8 * Hk * sum(lens)
        return dict(bytes=size, flops=2 * pairs * (m + dv) + 2 * c["B"] * c["H"] * c["d"] * m)
    left = [min(n, c["budget"]) for n in lens]
    moved = [k * (n - k) / n for n, k in zip(lens, left)]  # rows of equal standing: so many are kept behind the budget
    row = 2 * c["m"] + 4 + 2 * c["dv"]
    return dict(bytes=c["H"] * (8 * sum(lens) + 12 * sum(left) + 2 * row * sum(moved)), flops=4 * c["H"] * sum(lens))


# --------------------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        turns = s["pos"].double()[..., None] * s["freq"]                       # [B][N][rot/2]
        w = torch.polar(torch.ones_like(turns), -turns if c["inverse"] else turns)[:, None]

        def spin(x):
            y = x.double().clone()
            pairs = y[..., :c["rot"]]
            pairs = pairs.unflatten(-1, (-1, 2)) if c["interleaved"] else pairs.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
            y[..., :c["rot"]] = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return y
        return spin(s["q"]), spin(s["k"])
    if c["op"] == "append":
        kc = torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda")
        mul, vc = s["mul"].double(), s["vc"].double()
        for b, (p, n) in enumerate(zip(s["pos"].tolist(), s["count"].tolist())):
            x = torch.einsum("htd,hdm->htm", s["k"][b, :, :n].double(), s["P"].double())
            top = x.abs().max(dim=-1).values
            step = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 13), torch.ones_like(top))
            # a logarithm just off a whole number: the range [2^13, 2^14) decides
            step = torch.where(top / step >= 2.0 ** 14, 2 * step, torch.where((top / step < 2.0 ** 13) & (top > 0), step / 2, step))
            kc[b, :, p:p + n], mul[b, :, p:p + n], vc[b, :, p:p + n] = x / step[..., None], step, s["v"][b, :, :n].double()
        return kc, mul, vc
    if c["op"] == "decode":
        B, H, G = c["B"], c["H"], c["G"]
        out = torch.zeros((B, H, c["dv"]), dtype=torch.float64, device="cuda")
        acc = s["acc_out"].double() if c["weights"] else None
        lens = s["len"].tolist()
        for h in range(H // G):
            q = torch.einsum("bgd,dm->bgm", s["q"][:, h * G:(h + 1) * G].double(), s["P"][h].double()) / math.sqrt(c["m"])
            if c["prefix"]:
                k0 = s["prefix"][0][h].view(torch.float16).double() * s["prefix"][1][h].double()[:, None]
                v0 = s["prefix"][2][h].double()
            for b in range(B):
                n = lens[b]
                k = s["kc"][b, h, :n].view(torch.float16).double() * s["mul"][b, h, :n].double()[:, None]
                v = s["vc"][b, h, :n].double()
                if c["prefix"]:
                    k, v = torch.cat((k0, k)), torch.cat((v0, v))
                if len(k):
                    p = torch.softmax(q[b] @ k.T, dim=-1)
                    out[b, h * G:(h + 1) * G] = p @ v
                    if c["weights"]:
                        acc[b, h, :n] = s["acc"][b, h, :n].double() + p[:, len(k) - n:].sum(dim=0)
        return (out, acc) if c["weights"] else out
    # moved rows are the inputs' own bits; which rows move, one (sequence, head) after the other
    kc, mul, vc = s["kc"].view(torch.float16).double(), s["mul"].double(), s["vc"].double()
    acc, acc_out, src = s["acc"].double().cpu(), s["acc_out"].double(), s["src"].cpu()
    at, at_out, lens = s["row_pos"].cpu(), s["row_pos_out"], s["len"].tolist()
    for b in range(c["B"]):
        n = lens[b]
        left = min(n, c["budget"])
        for h in range(c["H"]):
            a, p = acc[b, h, :n].tolist(), at[b, h, :n].tolist()
            first = max(p) - c["recent"]
            order = sorted(range(n), key=lambda i: (not (p[i] < c["sink"] or p[i] > first), -a[i], i))
            kept = set(order[:left])
            late = iter(sorted(i for i in kept if i >= left))
            rows = [i if i in kept else next(late) for i in range(left)]
            src[b, h] = -1
            src[b, h, :left] = torch.tensor(rows, dtype=torch.int32)
            r = torch.tensor(rows, device="cuda")
            for x in (kc, mul, vc):
                x[b, h, :left] = x[b, h, r]
            acc_out[b, h, :left], at_out[b, h, :left] = s["acc"][b, h, r].double(), s["row_pos"][b, h, r]
    return kc, mul, vc, acc_out, at_out, torch.clamp(s["len"], max=c["budget"]), src.cuda()
