"""Operators around the projected attention, in plain form and as the library computes them.

  norm      norms of queries and keys for each head with the rotary positions in the same pass, and the gradient
  pack      full blocks of 64 rows of the 16-bit projected cache become pages of 8-bit values with one scale per
            block and head; the rows behind them move to the front
  decode    one query per sequence and head over such pages and the open 16-bit rows behind them, all keys or a
            window of the newest ones with a few first keys that stay visible

`own` false: elementary torch operations in 32 bits or more.  `own` true: the library's calls.
"""
import math

import torch

own = False

BLOCK = 64
EPS = 1e-6
F8 = torch.float8_e4m3fn


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the queries and keys of one decode step: 64 sequences at far positions of their own, 32 query and 8 key heads
        dict(name="norm step", op="norm", B=64, H=32, G=4, N=1, d=128, rot=128, interleaved=False, far=131072,
             gradient=False, dtype="bf16"),
        # a prompt chunk as the fused q/k/v product leaves it (token-major), half of each head rotated
        dict(name="norm prompt", op="norm", B=2, H=16, G=4, N=8192, d=128, rot=64, interleaved=True, far=8192,
             gradient=False, dtype="bf16"),
        # fp32 at an odd length and an odd head width
        dict(name="norm odd", op="norm", B=1, H=12, G=3, N=8191, d=96, rot=96, interleaved=False, far=262144,
             gradient=False, dtype="f32"),
        # the gradients of a training step's queries, keys and weights
        dict(name="norm gradient", op="norm", B=4, H=16, G=4, N=8192, d=128, rot=128, interleaved=False, far=8192,
             gradient=True, dtype="bf16"),
        # the same in fp32, small and ragged, a rotated part of an odd number of pairs
        dict(name="norm gradient odd", op="norm", B=3, H=6, G=6, N=1021, d=80, rot=38, interleaved=True, far=5000,
             gradient=True, dtype="f32"),
        # a decode step's packing: 64 sequences, of which one has just filled its block
        dict(name="pack step", op="pack", B=64, H=8, m=32, dv=128, lo=1, hi=64, cap=128, blocks=32),
        # prompts that have been read into the 16-bit rows
        dict(name="pack prompts", op="pack", B=8, H=8, m=64, dv=128, lo=1000, hi=8191, cap=8192, blocks=2),
        # the smallest call: one sequence, a few hundred keys, no shared heads
        dict(name="decode small", op="decode", B=1, H=8, G=1, d=64, m=16, dv=64, lo=300, hi=300, window=0, sink=0),
        # a batch of ragged sequences
        dict(name="decode batch", op="decode", B=64, H=32, G=4, d=128, m=32, dv=128, lo=17, hi=8191, window=0, sink=0),
        # two very long sequences
        dict(name="decode long", op="decode", B=2, H=64, G=8, d=128, m=64, dv=128, lo=131071, hi=131072, window=0,
             sink=0),
        # long sequences that see their newest 4096 keys and the first few; pages in between are gone
        dict(name="decode window", op="decode", B=32, H=16, G=2, d=128, m=32, dv=128, lo=3000, hi=65536, window=4096,
             sink=4),
        # many query heads on each key head
        dict(name="decode wide", op="decode", B=16, H=64, G=16, d=128, m=32, dv=128, lo=1023, hi=16383, window=0,
             sink=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "decode", "decode"])
    if op == "norm":
        G = rng.choice([1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([32, 64, 80, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = max(1, int(1e8) // ((H + H // G) * d * (2 if dtype == "bf16" else 4)))  # tokens
        N = _log(rng, 1, min(8192, most))
        B = _log(rng, 1, max(1, min(64, most // N)))
        return dict(op=op, B=B, H=H, G=G, N=N, d=d, rot=2 * rng.randint(1, d // 2), interleaved=rng.random() < 0.5,
                    far=_log(rng, N + 1, 1 << 20), gradient=rng.random() < 0.5, dtype=dtype)
    m = rng.choice([16, 32, 32, 64, 128])
    dv = rng.choice([64, 128])
    if op == "pack":
        hi = _log(rng, 1, 8191)
        B = _log(rng, 1, max(1, min(96, 65536 // hi)))
        return dict(op=op, B=B, H=rng.choice([1, 2, 3, 8]), m=m, dv=dv, lo=rng.randint(0, hi), hi=hi,
                    cap=hi + rng.randint(0, 100), blocks=rng.randint(0, 5))
    G = rng.choice([1, 2, 4, 5, 8, 16])
    H = G * rng.choice([1, 2, 4, 8])
    hi = _log(rng, 1, 131072)
    most = int(4e8) // (H // G * (m + dv))  # keys
    B = _log(rng, 1, max(1, min(128, most // max(hi, 2048))))
    window = 0 if rng.random() < 0.5 else _log(rng, 1, hi)
    return dict(op=op, B=B, H=H, G=G, d=rng.choice([32, 64, 96, 128, 200]), m=m, dv=dv, lo=rng.randint(0, hi), hi=hi,
                window=window, sink=rng.choice([0, 1, 4, 70, 130]) if window else 0)


def _lengths(lo, hi, B):
    """B lengths spread evenly over lo..hi: the same ones for every seed, in an order of its own."""
    return [lo + (hi - lo) * i // max(1, B - 1) for i in range(B)] if B > 1 else [hi]


# --------------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _key_rows(g, *shape, d):
    """Cache rows of projected keys: entries of variance d/m, fp16 bits and one multiplier per row."""
    m = shape[-1]
    x = torch.randn(shape, generator=g, device="cuda") * math.sqrt(d / m)
    e = torch.frexp(x.abs().amax(dim=-1))[1] - 14
    mul = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (x / mul[..., None]).to(torch.float16).view(torch.int16), mul


def _shuffled(g, values):
    t = torch.tensor(values, device="cuda", dtype=torch.int32)
    return t[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _codes(g, *shape, pages):
    """8-bit values of normal rows, page by page, in the upper half of the range that their scale gives."""
    x = torch.empty((pages, *shape), dtype=F8, device="cuda")
    step = max(1, (1 << 27) // max(1, math.prod(shape)))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x[i:i + n] = (torch.randn((n, *shape), generator=g, device="cuda") * 80.0).to(F8)
    return x


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = dict(case=c)
    if c["op"] == "norm":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, H, N, d = c["B"], c["H"], c["N"], c["d"]
        Hk = H // c["G"]

        def heads():
            # one token-major buffer [B][N][H + Hk][d], as the product with the stacked weights leaves it
            x = _normal(g, B, N, H + Hk, d, dtype=dt)
            return x[:, :, :H].permute(0, 2, 1, 3), x[:, :, H:].permute(0, 2, 1, 3)
        s["q"], s["k"] = heads()
        s["wq"], s["wk"] = ((1.0 + 0.2 * _normal(g, d)).to(dt) for _ in range(2))
        first = torch.randint(0, max(1, c["far"] - N), (B, 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -2.0 * i / c["rot"])
        # the library's table: the advance per position, in units of 2^-64 turns
        s["table"] = (s["freq"] / (2.0 * math.pi) * 2.0 ** 64).round().to(torch.int64)
        if c["gradient"]:
            # the gradients that the attention's backward hands over, head-major
            s["dq_out"], s["dk_out"] = _normal(g, B, H, N, d, dtype=dt), _normal(g, B, Hk, N, d, dtype=dt)
            x = torch.empty((B, N, H + Hk, d), dtype=dt, device="cuda")  # token-major, for the product's gradient
            s["dq"], s["dk"] = x[:, :, :H].permute(0, 2, 1, 3), x[:, :, H:].permute(0, 2, 1, 3)
        else:
            s["q_out"] = torch.empty((B, H, N, d), dtype=dt, device="cuda")
            s["k_out"] = torch.empty((B, Hk, N, d), dtype=dt, device="cuda")
    elif c["op"] == "pack":
        B, H, m, dv, cap = c["B"], c["H"], c["m"], c["dv"], c["cap"]
        s["kc"], s["mul"] = _key_rows(g, B, H, cap, m, d=128)
        s["vc"] = _normal(g, B, H, cap, dv, dtype=torch.bfloat16)
        s["len"] = _shuffled(g, _lengths(c["lo"], c["hi"], B))
        s["blocks"] = torch.randint(0, c["blocks"] + 1, (B,), generator=g, device="cuda").to(torch.int32)
        width = c["blocks"] + max(1, cap // BLOCK)
        s["table"] = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
        s["kc8"] = torch.zeros((B * width, H, BLOCK, m), dtype=torch.uint8, device="cuda").view(F8)
        s["vc8"] = torch.zeros((B * width, H, dv, BLOCK), dtype=torch.uint8, device="cuda").view(F8)
        s["ks"] = torch.zeros((B * width, H), dtype=torch.float32, device="cuda")
        s["vs"] = torch.zeros((B * width, H), dtype=torch.float32, device="cuda")
        s["len_out"], s["blocks_out"] = torch.zeros_like(s["len"]), torch.zeros_like(s["blocks"])
    else:
        B, H, Hk, d, m, dv = c["B"], c["H"], c["H"] // c["G"], c["d"], c["m"], c["dv"]
        s["q"] = _normal(g, B, H, d, dtype=torch.bfloat16)
        s["P"] = (torch.randn((Hk, d, m), generator=g, device="cuda") / math.sqrt(m)).to(torch.bfloat16)
        total = _shuffled(g, _lengths(c["lo"], c["hi"], B))
        s["blocks"] = torch.div(total, BLOCK, rounding_mode="floor").to(torch.int32)
        s["len"] = total - BLOCK * s["blocks"]
        width = max(1, c["hi"] // BLOCK)
        at = torch.arange(width, device="cuda")[None]
        there = at < s["blocks"][:, None]
        if c["window"]:  # pages that no later query sees have been given back
            there &= (at >= (total[:, None] - c["window"]).clamp(min=0) // BLOCK) | (at * BLOCK < c["sink"])
        pages = max(1, B * min(width, (c["window"] + BLOCK - 1) // BLOCK + 2 + c["sink"] // BLOCK)
                    if c["window"] else sum(n // BLOCK for n in _lengths(c["lo"], c["hi"], B)))
        order = torch.randperm(pages, generator=g, device="cuda")
        rank = there.flatten().cumsum(0).view(B, width) - 1
        s["table"] = torch.where(there, order[rank.clamp(0, pages - 1)], -1).to(torch.int32).contiguous()
        s["kc8"] = _codes(g, Hk, BLOCK, m, pages=pages)
        s["vc8"] = _codes(g, Hk, dv, BLOCK, pages=pages)
        # a power of two per block and head: values of the size that the codes' own spread gives
        near = torch.randint(-1, 2, (2, pages, Hk), generator=g, device="cuda").float()
        s["ks"] = torch.exp2(near[0] + round(math.log2(math.sqrt(d / m) / 80.0)))
        s["vs"] = torch.exp2(near[1] - 6.0)
        s["kc"], s["mul"] = _key_rows(g, B, Hk, BLOCK, m, d=d)
        s["vc"] = _normal(g, B, Hk, BLOCK, dv, dtype=torch.bfloat16)
        s["out"] = torch.empty((B, H, dv), dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, interleaved):
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((r, x[..., rot:]), dim=-1)


def _plain_norm(s):
    c = s["case"]
    # far positions: the angle is formed in 64 bits
    angle = s["pos"].double()[:, None, :, None] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def forward(x, w):
        y = x.float()
        r = torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + EPS)
        return _turn(y * r * w.float(), cos, sin, c["rot"], c["interleaved"]).to(x.dtype)

    def gradient(x, w, dy):
        y = x.float()
        r = torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + EPS)
        y = y * r
        back = _turn(dy.float(), cos, -sin, c["rot"], c["interleaved"])
        g = back * w.float()
        dx = r * (g - y * (g * y).mean(dim=-1, keepdim=True))
        return dx.to(x.dtype), (back * y).sum(dim=(0, 1, 2))

    if not c["gradient"]:
        return forward(s["q"], s["wq"]), forward(s["k"], s["wk"])
    dq, dwq = gradient(s["q"], s["wq"], s["dq_out"])
    dk, dwk = gradient(s["k"], s["wk"], s["dk_out"])
    return dq, dk, dwq, dwk


def _value_order():
    """The token of a block at each of the 64 places of a value column."""
    p = torch.arange(BLOCK, device="cuda")
    return 8 * (p // 2 % 8) + 2 * (p // 16) + p % 2


def _scale_of(x):
    """The least power of two s >= 2^-100 with max|x| <= 448 s, over the last two dimensions."""
    top = x.abs().amax(dim=(-1, -2))
    f, e = torch.frexp(top)  # 448 is 0.875 x 2^9
    e = torch.where(f <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, -100).clamp(min=-100))


def _plain_pack(s):
    c = s["case"]
    B, H, cap, m, dv = c["B"], c["H"], c["cap"], c["m"], c["dv"]
    most = cap // BLOCK
    n = torch.div(s["len"], BLOCK, rounding_mode="floor")
    b, i = torch.nonzero(torch.arange(most, device="cuda")[None] < n[:, None], as_tuple=True)
    page = s["table"].long()[b, s["blocks"].long()[b] + i]
    k = s["kc"].view(torch.float16)[:, :, :most * BLOCK].float() * s["mul"][:, :, :most * BLOCK, None]
    k = k.view(B, H, most, BLOCK, m)[b, :, i]
    v = s["vc"][:, :, :most * BLOCK].view(B, H, most, BLOCK, dv)[b, :, i].float()
    ks, vs = _scale_of(k), _scale_of(v)
    s["ks"][page], s["vs"][page] = ks, vs
    # an index into 8-bit values goes by their bytes
    s["kc8"].view(torch.uint8)[page] = (k / ks[..., None, None]).to(F8).view(torch.uint8)
    v = (v / vs[..., None, None])[:, :, _value_order()].transpose(-1, -2)
    s["vc8"].view(torch.uint8)[page] = v.contiguous().to(F8).view(torch.uint8)
    # what is left moves to the front
    left = s["len"] - BLOCK * n
    row = torch.arange(min(BLOCK, cap), device="cuda")
    src = torch.where(row[None] < left[:, None], row[None] + BLOCK * n[:, None], row[None]).long()[:, None].expand(B, H, -1)
    head = len(row)
    s["kc"][:, :, :head] = s["kc"].gather(2, src[..., None].expand(-1, -1, -1, m))
    s["vc"][:, :, :head] = s["vc"].gather(2, src[..., None].expand(-1, -1, -1, dv))
    s["mul"][:, :, :head] = s["mul"].gather(2, src)
    return (s["kc8"], s["ks"], s["vc8"], s["vs"], s["kc"].view(torch.float16), s["mul"], s["vc"], left,
            s["blocks"] + n)


def _plain_decode(s):
    c = s["case"]
    B, H, G, m, dv = c["B"], c["H"], c["G"], c["m"], c["dv"]
    Hk, width = H // G, s["table"].shape[1]
    q = torch.matmul(s["q"].float().view(B, Hk, G, c["d"]), s["P"].float()) / math.sqrt(m)
    total = BLOCK * s["blocks"] + s["len"]
    first = (total - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(total)
    # the blocks to look at: all, or those of the first keys and of the window
    if c["window"]:
        sinks = min(width, (c["sink"] + BLOCK - 1) // BLOCK)
        some = min(width, (c["window"] + BLOCK - 1) // BLOCK + 1)
        begin = torch.div(first, BLOCK, rounding_mode="floor").clamp(min=sinks)
        at = torch.cat((torch.arange(sinks, device="cuda").expand(B, sinks),
                        begin[:, None] + torch.arange(some, device="cuda")), dim=1)
    else:
        at = torch.arange(width, device="cuda").expand(B, width)
    inside = at < s["blocks"][:, None]
    page = s["table"].long().gather(1, at.clamp(max=width - 1)).clamp(min=0)
    j = BLOCK * at[..., None] + torch.arange(BLOCK, device="cuda")
    seen = inside[..., None] & ((j >= first[:, None, None]) | (j < c["sink"]))
    k = s["kc8"].view(torch.uint8)[page].view(F8).float() * s["ks"][page][..., None, None]  # [B][blocks][Hk][64][m]
    k = k.transpose(1, 2).reshape(B, Hk, -1, m)
    v = s["vc8"].view(torch.uint8)[page].view(F8).float() * s["vs"][page][..., None, None]  # [B][blocks][Hk][dv][64]
    v = v[..., torch.argsort(_value_order())].permute(0, 2, 1, 4, 3).reshape(B, Hk, -1, dv)
    # the open rows behind the blocks
    row = torch.arange(BLOCK, device="cuda")
    j = BLOCK * s["blocks"][:, None] + row
    seen = torch.cat((seen.flatten(1), (row < s["len"][:, None]) & ((j >= first[:, None]) | (j < c["sink"]))), dim=1)
    k = torch.cat((k, s["kc"].view(torch.float16).float() * s["mul"][..., None]), dim=2)
    v = torch.cat((v, s["vc"].float()), dim=2)
    scores = torch.matmul(q, k.transpose(-1, -2)).masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    sum_ = e.sum(dim=-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(sum_ > 0, sum_, 1.0)
    return out.view(B, H, dv).to(torch.bfloat16)


# --------------------------------------------------------------------------- the library's calls
def _own(s):
    import projected_feature_efficient_gb300 as spa
    c = s["case"]
    if c["op"] == "norm" and c["gradient"]:
        return spa.spa_norm_rope_bwd(s["dq_out"], s["q"], s["wq"], s["table"], s["pos"], dk_out=s["dk_out"], k=s["k"],
                                     wk=s["wk"], eps=EPS, interleaved=c["interleaved"], dq=s["dq"], dk=s["dk"])
    if c["op"] == "norm":
        return spa.spa_norm_rope(s["q"], s["wq"], s["table"], s["pos"], k=s["k"], wk=s["wk"], eps=EPS,
                                 interleaved=c["interleaved"], out=s["q_out"], k_out=s["k_out"])
    if c["op"] == "pack":
        spa.spa_kcache8_pack(s["kc"], s["mul"], s["vc"], s["len"], (s["kc8"], s["ks"], s["vc8"], s["vs"]), s["table"],
                             s["blocks"], lens_out=s["len_out"], blocks_out=s["blocks_out"])
        return (s["kc8"], s["ks"], s["vc8"], s["vs"], s["kc"].view(torch.float16), s["mul"], s["vc"], s["len_out"],
                s["blocks_out"])
    return spa.spa_attention_decode8(s["q"], s["P"], (s["kc8"], s["ks"], s["vc8"], s["vs"]), s["table"], s["blocks"],
                                     s["kc"], s["mul"], s["vc"], s["len"], window=c["window"], sink=c["sink"],
                                     out=s["out"])


_PLAIN = dict(norm=_plain_norm, pack=_plain_pack, decode=_plain_decode)


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------- what each cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        heads = c["H"] + c["H"] // c["G"]
        n = c["B"] * heads * c["N"]
        size = 2 if c["dtype"] == "bf16" else 4
        moved = (3 if c["gradient"] else 2) * n * c["d"] * size
        return dict(bytes=moved + 4 * c["B"] * c["N"] + 4 * c["rot"] + 2 * size * c["d"] + (8 * c["d"] if c["gradient"] else 0),
                    flops=n * ((11 if c["gradient"] else 4) * c["d"] + 3 * c["rot"]))
    lens = _lengths(c["lo"], c["hi"], c["B"])
    if c["op"] == "pack":
        rows = c["H"] * sum(BLOCK * (n // BLOCK) for n in lens)
        left = c["H"] * sum(n % BLOCK for n in lens if n >= BLOCK)
        row = 2 * c["m"] + 4 + 2 * c["dv"]
        size = rows * (row + c["m"] + c["dv"]) + rows // BLOCK * 8 + 2 * left * row + 16 * c["B"]
        return dict(bytes=size, flops=3 * rows * (c["m"] + c["dv"]))
    Hk, m, dv, w = c["H"] // c["G"], c["m"], c["dv"], c["window"]
    seen = closed = 0
    for n in lens:
        begin = max(0, n - w) if w else 0
        gone = max(0, begin - c["sink"])  # keys that are masked
        seen += n - gone
        full = BLOCK * (n // BLOCK)
        closed += max(0, full - max(0, min(gone, full - c["sink"])))
    opened = seen - closed
    size = Hk * (closed * (m + dv) + closed // BLOCK * 8 + opened * (2 * m + 4 + 2 * dv))
    size += c["B"] * c["H"] * (2 * c["d"] + 2 * dv) + 2 * Hk * c["d"] * m + 8 * c["B"] + closed // BLOCK * 4
    return dict(bytes=size, flops=2 * c["H"] * seen * (m + dv) + 2 * c["B"] * c["H"] * c["d"] * m)


# --------------------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        turns = s["pos"].double()[..., None] * s["freq"]
        w = torch.polar(torch.ones_like(turns), turns)[:, None]

        def apply(x, weight):
            y = x * (weight / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / c["d"] + EPS))
            pairs = y[..., :c["rot"]]
            pairs = pairs.unflatten(-1, (-1, 2)) if c["interleaved"] else pairs.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat((z, y[..., c["rot"]:]), dim=-1)

        if not c["gradient"]:
            return apply(s["q"].double(), s["wq"].double()), apply(s["k"].double(), s["wk"].double())
        found = []
        for name in "qk":
            x = s[name].double().requires_grad_()
            weight = s["w" + name].double().requires_grad_()
            found.append(torch.autograd.grad(apply(x, weight), (x, weight), s["d%s_out" % name].double()))
        return found[0][0], found[1][0], found[0][1], found[1][1]
    if c["op"] == "pack":
        kc8, vc8 = torch.zeros(s["kc8"].shape, dtype=torch.float64, device="cuda"), torch.zeros(
            s["vc8"].shape, dtype=torch.float64, device="cuda")
        ks, vs = s["ks"].double(), s["vs"].double()
        kc, mul, vc = s["kc"].view(torch.float16).double(), s["mul"].double(), s["vc"].double()
        new = [t.clone() for t in (kc, mul, vc)]
        place = [16 * ((t % 8) // 2) + 2 * (t // 8) + t % 2 for t in range(BLOCK)]
        lens, blocks, table = s["len"].tolist(), s["blocks"].tolist(), s["table"].tolist()

        def scale(x):
            top = x.abs().amax(dim=(1, 2))
            e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
            # a logarithm just off a whole number: the comparison decides
            e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e))
            return torch.exp2(e.clamp(min=-100.0))

        for b, n in enumerate(lens):
            for i in range(n // BLOCK):
                p, rows = table[b][blocks[b] + i], slice(BLOCK * i, BLOCK * (i + 1))
                x, y = kc[b, :, rows] * mul[b, :, rows, None], vc[b, :, rows]
                ks[p], vs[p] = scale(x), scale(y)
                kc8[p] = x / ks[p][:, None, None]
                vc8[p][:, :, place] = (y / vs[p][:, None, None]).transpose(1, 2)
            r = n % BLOCK
            if n >= BLOCK and r:
                for t, old in zip(new, (kc, mul, vc)):
                    t[b, :, :r] = old[b, :, n - r:n]
        left = torch.tensor([n % BLOCK for n in lens], dtype=torch.int32, device="cuda")
        return (kc8, ks, vc8, vs, *new, left, s["blocks"] + torch.tensor([n // BLOCK for n in lens], device="cuda").int())
    B, H, G = c["B"], c["H"], c["G"]
    out = torch.zeros((B, H, c["dv"]), dtype=torch.float64, device="cuda")
    at = torch.tensor([16 * ((t % 8) // 2) + 2 * (t // 8) + t % 2 for t in range(BLOCK)], device="cuda")
    q = torch.einsum("bkgd,kdm->bkgm", s["q"].double().view(B, H // G, G, -1), s["P"].double()) / math.sqrt(c["m"])
    for b in range(B):
        nb, r = int(s["blocks"][b]), int(s["len"][b])
        n = BLOCK * nb + r
        seen = [j for j in range(n) if not c["window"] or j >= n - c["window"] or j < c["sink"]]
        if not seen:
            continue
        cut = torch.tensor(seen, device="cuda")
        closed = cut[cut < BLOCK * nb]
        which, place = torch.unique(closed // BLOCK, return_inverse=True)
        page = s["table"][b].long()[which]
        # 8-bit values by their bytes, for the index
        k8 = s["kc8"].view(torch.uint8)[page].view(F8)
        v8 = s["vc8"].view(torch.uint8)[page].view(F8)
        for h in range(H // G):
            k = (k8[:, h].double() * s["ks"][page, h].double()[:, None, None])[place, closed % BLOCK]
            v = (v8[:, h].double() * s["vs"][page, h].double()[:, None, None])[place, :, at[closed % BLOCK]]
            tail = cut[len(closed):] - BLOCK * nb
            k = torch.cat((k, s["kc"][b, h].view(torch.float16).double()[tail] * s["mul"][b, h].double()[tail, None]))
            v = torch.cat((v, s["vc"][b, h].double()[tail]))
            out[b, h * G:(h + 1) * G] = torch.softmax(q[b, h] @ k.T, dim=-1) @ v
    return out
