"""The 8-bit operators' workloads: e4m3 codes with one float32 scale per block of 128.

Four operators of one format: ``fp8_quantize`` (rows of activations, or 128 x 128 blocks of a
weight), ``fp8_linear`` (the product of two quantized operands, with the linear layers' bias and
activation), ``fp8_cache_write`` (keys and values quantized into a paged cache as they are
produced) and ``fp8_cache_read`` (a batch of sequences decoded back from the pages).

``run`` computes each either in its plain form (elementary torch operations in float32, rounded
once) or, where ``own`` is true, through the package.

The format. A block's largest finite magnitude m (at least 2^-64) gives scale = m / 448; a value x
is stored as the e4m3 number nearest 448 x / m, ties to even; infinities are stored as +-448 and a
NaN as NaN. A stored code c stands for c * scale.
"""
import math

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token's activations in front of the fused QKV projection: the smallest call, latency
        dict(name="quantize token", op="quantize", rows=1, k=3840, block_rows=1, dtype="bf16"),
        # the activations between the feed-forward layers of the transformer block: streaming
        dict(name="quantize activations", op="quantize", rows=4096, k=10240, block_rows=1, dtype="bf16"),
        # a feed-forward weight, quantized once when a model is loaded
        dict(name="quantize weight", op="quantize", rows=10240, k=3840, block_rows=128, dtype="bf16"),
        # one token through the fused QKV projection: streams the weight
        dict(name="linear token", op="linear", m=1, n=11520, k=3840, bias=False, act="none", dtype="bf16"),
        # a ragged batch of single tokens through the feed-forward down projection
        dict(name="linear batch", op="linear", m=37, n=3840, k=10240, bias=True, act="none", dtype="bf16"),
        # a short prompt through the up projection with its activation, float16 outputs
        dict(name="linear prompt", op="linear", m=333, n=10240, k=3840, bias=True, act="silu", dtype="fp16"),
        # a text-and-image sequence through an attention projection: few tiles for the whole chip
        dict(name="linear projection", op="linear", m=1089, n=3840, k=3840, bias=False, act="none", dtype="bf16"),
        # the up projection of the transformer block at its full token count: tensor-bound
        dict(name="linear up", op="linear", m=4096, n=10240, k=3840, bias=True, act="gelu_tanh", dtype="bf16"),
        # one step of a decoding batch: a token per sequence, three padded rows
        dict(name="write step", op="write", tokens=48, pad=3, heads=8, dim=128, page=16, pages=512, dtype="bf16"),
        # a long prompt into the cache
        dict(name="write prompt", op="write", tokens=16383, pad=0, heads=8, dim=128, page=64, pages=320, dtype="bf16"),
        # the cached prefixes of a few short sequences, a narrow head, float16
        dict(name="read short", op="read", lens="1 17 0 130 64", heads=8, dim=64, page=16, pages=64, dtype="fp16"),
        # the prefixes of a batch of long conversations
        dict(name="read long", op="read", lens="4096 3001 517 2048 1 3777 2500 4000 1234 999 3300 63",
             heads=8, dim=128, page=64, pages=512, dtype="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = (v + step - 1) // step * step
    return max(step, min(v, hi))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "write", "read"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "quantize":
        k = _log(rng, 32, 12288, 32)
        rows = min(_log(rng, 1, 16384), 4096 * 10240 // k)
        return dict(op=op, rows=rows, k=k, block_rows=rng.choice([1, 1, 128]), dtype=dtype)
    if op == "linear":
        m, n, k = _log(rng, 1, 4096), _log(rng, 1, 11520), _log(rng, 32, 10240, 32)
        m = max(1, min(m, 4096 * 10240 * 3840 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu_tanh"]),
                    dtype=dtype)
    heads, dim, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([32, 64, 80, 96, 128, 192, 256]), rng.choice([8, 16, 24, 64, 128])
    most = 16384 * 1024 // (heads * dim)
    if op == "write":
        tokens = min(_log(rng, 1, 16384), most)
        pages = -(-tokens // page) + rng.randint(1, 16)
        return dict(op=op, tokens=tokens, pad=min(rng.choice([0, 0, 1, 5]), tokens - 1), heads=heads, dim=dim, page=page,
                    pages=pages, dtype=dtype)
    seqs = rng.randint(1, 24)
    lens = [0 if rng.random() < 0.05 else _log(rng, 1, 4096) for _ in range(seqs)]
    while sum(lens) > min(most, 25000):
        lens[lens.index(max(lens))] //= 2
    lens[0] = max(lens[0], 1)
    pages = sum(-(-n // page) for n in lens) + rng.randint(1, 16)
    return dict(op=op, lens=" ".join(map(str, lens)), heads=heads, dim=dim, page=page, pages=pages, dtype=dtype)


# ------------------------------------------------------------------ inputs --
def _lens(case):
    """The cached lengths of a batch, written as one text."""
    return [int(n) for n in case["lens"].split()]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, std, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _weights(shape, std, g):
    """Student-t with four degrees of freedom: the heavy tails of trained weights."""
    z = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    u = 1.0 - torch.rand((2,) + tuple(shape), generator=g, device="cuda", dtype=torch.float32)
    return z / torch.sqrt(-0.5 * torch.log(u[0] * u[1])) * (std / math.sqrt(2.0))


def _activations(shape, g):
    """Normal activations with a few channels that are an order of magnitude larger."""
    x = _normal(shape, 1.0, g)
    loud = torch.rand(shape[-1:], generator=g, device="cuda") < 0.004
    return torch.where(loud, x * 20.0, x)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "quantize":
        shape = (case["rows"], case["k"])
        x = _activations(shape, g) if case["block_rows"] == 1 else _weights(shape, 0.02, g)
        return dict(op=op, x=x.to(dt), block_rows=case["block_rows"])
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        xc, xs = _encode(_activations((m, k), g).to(torch.bfloat16), 1)
        wc, ws = _encode(_weights((n, k), 0.02, g).to(torch.bfloat16), BLOCK)
        bias = _normal((n,), 0.5, g).to(dt) if case["bias"] else None
        return dict(op=op, xc=xc, xs=xs, wc=wc, ws=ws, bias=bias, act=case["act"], dt=dt)
    heads, dim, page, pages = case["heads"], case["dim"], case["page"], case["pages"]
    nb = -(-dim // BLOCK)
    shape = (pages, page, heads, dim)

    def filled():
        return _normal(shape, 60.0, g).clamp(-448, 448).to(F8), _normal((pages, page, heads, nb), 1.0, g).abs() * 1e-2 + 1e-4

    kc, ks = filled()
    vc, vs = filled()
    cache = (kc, ks, vc, vs)
    if op == "write":
        tokens = case["tokens"]
        # keys and values are slices of the fused projection's output (two query heads per key head)
        qkv = _activations((tokens, 4 * heads * dim), g).to(dt)
        k = qkv[:, 2 * heads * dim:3 * heads * dim].view(tokens, heads, dim)
        v = qkv[:, 3 * heads * dim:].view(tokens, heads, dim)
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
        if case["pad"]:
            slots[tokens - case["pad"]:] = -1
        return dict(op=op, k=k, v=v, cache=cache, slots=slots)
    lens = _lens(case)
    width = max(-(-n // page) for n in lens)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        p = -(-n // page)
        table[b, :p] = order[at:at + p]
        at += p
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return dict(op=op, cache=cache, table=table, cu=cu, rows=sum(lens), dt=dt)


# -------------------------------------------------------------- plain forms --
def _encode(x, block_rows):
    """codes [R, K] and scales [ceil(K / 128), ceil(R / block_rows)] of x [R, K]."""
    R, K = x.shape
    rb, kb = -(-R // block_rows), -(-K // BLOCK)
    v = torch.zeros((rb * block_rows, kb * BLOCK), dtype=torch.float32, device=x.device)
    v[:R, :K] = x
    v = v.view(rb, block_rows, kb, BLOCK)
    mag = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    m = mag.amax(dim=(1, 3), keepdim=True).clamp_min(FLOOR)
    # 448 x / m as (7/8 x) / (m / 512): neither side leaves float32's range
    q = (torch.minimum(torch.maximum(v, -m), m) * 0.875) / (m * 2.0 ** -9)
    codes = q.to(F8).view(rb * block_rows, kb * BLOCK)[:R, :K].contiguous()
    return codes, (m / 448.0).view(rb, kb).t().contiguous()


def _decode(codes, scales, block_rows):
    R, K = codes.shape
    s = scales.t().repeat_interleave(block_rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :K]
    return codes.float() * s


def _activation(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain(s):
    op = s["op"]
    if op == "quantize":
        return _encode(s["x"], s["block_rows"])
    if op == "linear":
        y = _decode(s["xc"], s["xs"], 1) @ _decode(s["wc"], s["ws"], BLOCK).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return _activation(y, s["act"]).to(s["dt"])
    kc, ks, vc, vs = s["cache"]
    if op == "write":
        keep = s["slots"] >= 0
        slots = s["slots"][keep]
        for x, codes, scales in ((s["k"], kc, ks), (s["v"], vc, vs)):
            T, H, D = x.shape
            c, sc = _encode(x.reshape(T * H, D), 1)
            codes.view(torch.uint8).view(-1, H, D)[slots] = c.view(torch.uint8).view(T, H, D)[keep]
            scales.view(-1, H, scales.shape[-1])[slots] = sc.t().reshape(T, H, -1)[keep]
        return kc, ks, vc, vs
    page = kc.shape[1]
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
    pos = row - s["cu"].long()[seq]
    slot = s["table"].long()[seq, pos // page] * page + pos % page
    outs = []
    for codes, scales in ((kc, ks), (vc, vs)):
        H, D = codes.shape[2:]
        c = codes.view(torch.uint8).view(-1, H, D)[slot].view(F8).float()
        outs.append((c * scales.view(-1, H, scales.shape[-1])[slot].repeat_interleave(BLOCK, 2)[..., :D]).to(s["dt"]))
    return tuple(outs)


def run(state):
    if not own:
        return _plain(state)
    import bit_diffusion_transformer_b200 as opq
    s, op = state, state["op"]
    if op == "quantize":
        return opq.fp8_quantize(s["x"], s["block_rows"])
    if op == "linear":
        return opq.fp8_linear(s["xc"], s["xs"], s["wc"], s["ws"], bias=s["bias"], act=s["act"], dtype=s["dt"])
    if op == "write":
        opq.fp8_cache_write(s["k"], s["v"], s["cache"], s["slots"])
        return s["cache"]
    return opq.fp8_cache_read(s["cache"], s["table"], s["cu"], s["rows"], dtype=s["dt"])


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["k"]
        nb = -(-case["rows"] // case["block_rows"]) * -(-case["k"] // BLOCK)
        return {"bytes": 3 * n + 4 * nb, "flops": 4 * n}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // BLOCK)) + 2 * m * n + (2 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    row = 2 * case["heads"] * case["dim"]
    scales = 2 * 4 * case["heads"] * -(-case["dim"] // BLOCK)
    if op == "write":
        t = case["tokens"] - case["pad"]
        return {"bytes": t * (3 * row + scales) + 8 * case["tokens"], "flops": 4 * t * row}
    lens = _lens(case)
    t = sum(lens)
    return {"bytes": t * (3 * row + scales) + 4 * sum(-(-n // case["page"]) for n in lens) + 4 * len(lens) + 4,
            "flops": t * row}


# ------------------------------------------------- the definition in 64 bits --
def _e4m3_nearest(v):
    """The e4m3 number nearest v (float64), ties to even: 3 mantissa bits, exponents from -6, at most 448."""
    _, e = torch.frexp(v.abs())
    steps = torch.tensor([2.0 ** (b - 3) for b in range(-6, 9)], dtype=torch.float64, device=v.device)
    step = steps[(e.long() - 1).clamp(-6, 8) + 6]
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _blocks_exact(x):
    """(values the codes stand for, scale) of x [..., n] float64, one block along the last axis."""
    m = x.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    return _e4m3_nearest(448.0 * x / m), (m / 448.0).squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        x, br = s["x"].double(), s["block_rows"]
        R, K = x.shape
        codes = torch.empty_like(x)
        scales = torch.empty((-(-K // BLOCK), -(-R // br)), dtype=torch.float64, device="cuda")
        if br == 1:
            for j in range(scales.shape[0]):
                codes[:, j * BLOCK:(j + 1) * BLOCK], scales[j] = _blocks_exact(x[:, j * BLOCK:(j + 1) * BLOCK])
        else:
            full, tail = R // br, R % br
            for j in range(scales.shape[0]):
                part = x[:, j * BLOCK:(j + 1) * BLOCK]
                w = part.shape[1]
                if full:
                    c, scales[j, :full] = _blocks_exact(part[:full * br].reshape(full, br * w))
                    codes[:full * br, j * BLOCK:j * BLOCK + w] = c.view(full * br, w)
                if tail:
                    c, sc = _blocks_exact(part[full * br:].reshape(1, tail * w))
                    scales[j, full:] = sc
                    codes[full * br:, j * BLOCK:j * BLOCK + w] = c.view(tail, w)
        return codes, scales
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        y = torch.zeros((m, n), dtype=torch.float64, device="cuda")
        for j in range(s["xs"].shape[0]):
            a = s["xc"][:, j * BLOCK:(j + 1) * BLOCK].double() * s["xs"][j].double()[:, None]
            per_row = s["ws"][j].double()[torch.arange(n, device="cuda") // BLOCK]
            y.addmm_(a, (s["wc"][:, j * BLOCK:(j + 1) * BLOCK].double() * per_row[:, None]).t())
        if s["bias"] is not None:
            y += s["bias"].double()
        if s["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif s["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        return y
    if op == "write":
        out = []
        slots = s["slots"].tolist()
        live = [t for t, a in enumerate(slots) if a >= 0]
        where = s["slots"][live]
        for x, codes, scales in ((s["k"], s["cache"][0], s["cache"][1]), (s["v"], s["cache"][2], s["cache"][3])):
            H, D = x.shape[1:]
            c, sc = codes.double().view(-1, H, D), scales.double().view(-1, H, scales.shape[-1])
            for j in range(scales.shape[-1]):
                cj, sj = _blocks_exact(x[live, :, j * BLOCK:(j + 1) * BLOCK].double())
                c[where, :, j * BLOCK:(j + 1) * BLOCK] = cj
                sc[where, :, j] = sj
            out += [c.view(codes.shape), sc.view(scales.shape)]
        return tuple(out)
    page = s["cache"][0].shape[1]
    out = []
    for codes, scales in ((s["cache"][0], s["cache"][1]), (s["cache"][2], s["cache"][3])):
        rows = []
        for b, n in enumerate(_lens(case)):
            ids = s["table"][b, :-(-n // page)].long()
            c = codes.view(torch.uint8)[ids].view(F8).double().flatten(0, 1)[:n]
            sc = scales[ids].double().flatten(0, 1)[:n]
            rows.append(torch.cat([c[..., j * BLOCK:(j + 1) * BLOCK] * sc[..., j:j + 1]
                                   for j in range(scales.shape[-1])], dim=-1))
        out.append(torch.cat(rows))
    return tuple(out)
