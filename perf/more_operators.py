"""The operators around the paged cache in a decode layer, as they are timed: the
norm with the residual's addition and the gated activation, both with 8-bit
outputs and a scale for each 128 of a row; the 8-bit matrix product that takes
them; rotary positions, alone and on the way into the cache.

``run`` computes them in elementary torch operations, or with ``own`` set
through the library's entry points."""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
BLOCK = 128             # elements of a row that share a scale
LEAST = 2.0 ** -64      # a block's largest element counts as this at least
EPS = 1e-6


def listed():
    return [
        # one frame of 32 streams, hidden size 1024: the residual's sum and the next product's 8-bit input
        norm("norm_frame", rows=32, dim=1024, kind="bf16", out="e4m3", residual=True),
        # prompts admitted together, wide hidden state
        norm("norm_prompts", rows=32768, dim=4096, kind="bf16", out="e4m3", residual=True),
        # 32 bits, an odd width, no residual
        norm("norm_f32_odd", rows=5000, dim=1001, kind="f32", out="bf16", residual=False),
        # one frame of 128 streams, the middle of a feed-forward block
        gate("gate_frame", rows=128, dim=2816, kind="bf16", out="e4m3", act="silu"),
        # prompts, a wide feed-forward block
        gate("gate_prompts", rows=16384, dim=11008, kind="bf16", out="e4m3", act="gelu"),
        # one frame of 32 streams: 16 query and 2 x 8 key and value heads of 128 from hidden size 1024
        linear("linear_frame", m=32, n=4096, k=1024, out="bf16"),
        # one frame of 128 streams through a wide feed-forward block
        linear("linear_128_streams", m=128, n=11008, k=4096, out="bf16"),
        # prompts: as much arithmetic as the tensor cores can take
        linear("linear_prompts", m=8192, n=8192, k=4096, out="bf16"),
        # odd sizes, 32-bit outputs
        linear("linear_f32_odd", m=777, n=2001, k=1040, out="f32"),
        # one frame of 128 streams: queries and keys turned, keys and values into the cache, a few rows unused
        rotary("rotary_frame", tokens=128, heads=16, kv_heads=8, dim=128, rot=128, layout="half", kind="bf16", cache="bf16",
               block=16, far=2000, skipped=3),
        # prompts into an 8-bit cache, neighbours as pairs, half of the head turned
        rotary("rotary_prompts_e4m3", tokens=32768, heads=32, kv_heads=8, dim=128, rot=64, layout="pairs", kind="bf16", cache="e4m3",
               block=32, far=32768, skipped=100),
        # 32 bits, no cache, an odd head and far positions, slowed for a long context
        rotary("rotary_f32_far", tokens=6001, heads=5, kv_heads=0, dim=80, rot=40, layout="half", kind="f32", cache="f32",
               block=16, far=1000000, skipped=7, slower=32.0),
    ]


def norm(name, *, rows, dim, kind, out, residual):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "kind": kind, "out": out, "residual": residual}


def gate(name, *, rows, dim, kind, out, act):
    return {"name": name, "op": "gate", "rows": rows, "dim": dim, "kind": kind, "out": out, "act": act}


def linear(name, *, m, n, k, out):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "out": out}


def rotary(name, *, tokens, heads, kv_heads, dim, rot, layout, kind, cache, block, far, skipped, slower=1.0):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "layout": layout, "kind": kind, "cache": cache, "block": block, "far": far, "skipped": skipped, "slower": slower}


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("norm", "gate", "linear", "linear", "rotary"))
    kind, out = rng.choice((("bf16", "e4m3"), ("bf16", "e4m3"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "e4m3")))
    if op in ("norm", "gate"):
        dim = rng.choice((log(64, 16384), 8 * log(8, 2048), 128 * log(1, 128)))
        rows = log(1, max(2, min(65536, (1 << 26) // dim)))
        if op == "norm":
            c = norm("", rows=rows, dim=dim, kind=kind, out=out, residual=rng.random() < 0.7)
        else:
            c = gate("", rows=rows, dim=dim, kind=kind, out=out, act=rng.choice(("silu", "gelu", "gelu_tanh", "none")))
    elif op == "linear":
        k = rng.choice((16 * log(4, 1024), 128 * log(1, 128)))
        n = rng.choice((log(64, 16384), 64 * log(1, 256)))
        m = log(1, max(2, min(16384, (1 << 37) // (n * k))))
        c = linear("", m=m, n=n, k=k, out=rng.choice(("bf16", "bf16", "f32")))
    else:
        kind, cache = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")))
        kv_heads = rng.choice((0, 1, 2, 3, 5, 8, 12))
        heads = max(1, kv_heads) * rng.choice((1, 2, 4, 5))
        dim = rng.choice((48, 64, 80, 96, 128, 128, 192, 256))
        tokens = log(1, max(2, min(65536, (1 << 26) // ((heads + 2 * kv_heads) * dim))))
        c = rotary("", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rng.choice((dim, dim, dim // 2, 16)),
                   layout=rng.choice(("half", "pairs")), kind=kind, cache=cache, block=rng.choice((8, 16, 16, 24, 32, 64, 128)),
                   far=log(2, 1 << 20), skipped=rng.randrange(tokens // 8 + 1), slower=rng.choice((1.0, 1.0, 8.0)))
    c.pop("name")
    return c


def blocks_of(x, block):
    return -(-x // block)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
_sampler = None


def library():
    """The package, and the one handle that a program keeps."""
    global _sampler
    import codebook_token_sampling_gb300 as ts
    if _sampler is None:
        _sampler = ts.Sampler(0)
    return ts, _sampler.handle


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"norm": prepare_norm, "gate": prepare_gate, "linear": prepare_linear, "rotary": prepare_rotary}[case["op"]](s, case, gen)
    return s


def normal(shape, gen, dtype=torch.float32):
    return torch.randn(shape, device=DEVICE, generator=gen, dtype=dtype)


def outputs(case, rows, dim):
    """A program's buffers: the output, and its scales where it has 8 bits."""
    out = torch.empty((rows, dim), device=DEVICE, dtype=TYPES[case["out"]])
    return out, torch.empty((rows, blocks_of(dim, BLOCK)), device=DEVICE) if case["out"] == "e4m3" else None


def prepare_norm(s, case, gen):
    rows, dim, dtype = case["rows"], case["dim"], TYPES[case["kind"]]
    # a hidden state has a few channels that are much larger than the others
    big = 1 + 15 * (torch.rand(dim, device=DEVICE, generator=gen) < 0.01)
    s["x"] = normal((rows, dim), gen, dtype) * big.to(dtype)
    s["residual"] = normal((rows, dim), gen, dtype) * (3 * big).to(dtype) if case["residual"] else None
    s["weight"] = 1 + 0.2 * normal((dim,), gen)
    if own:
        ts, _ = library()
        s["out"], s["scale"] = outputs(case, rows, dim)
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["plan"] = ts.RmsNorm(s["x"], s["out"], s["weight"], residual=s["residual"], residual_out=s["sum"], out_scale=s["scale"], eps=EPS)


def prepare_gate(s, case, gen):
    rows, dim, dtype = case["rows"], case["dim"], TYPES[case["kind"]]
    both = 2 * normal((rows, 2 * dim), gen, dtype)  # as one projection leaves them
    s["gate"] = both[:, :dim] if case["act"] != "none" else None
    s["up"] = both[:, dim:]
    if own:
        ts, _ = library()
        s["out"], s["scale"] = outputs(case, rows, dim)
        s["plan"] = ts.Gate(s["up"], s["out"], s["gate"], activation=case["act"], out_scale=s["scale"])


def prepare_linear(s, case, gen):
    m, n, k = case["m"], case["n"], case["k"]
    # as ts_rms_norm leaves its rows: blocks that reach 448, scales about what a normalised row has
    x = normal((m, k), gen, torch.bfloat16) * 120
    s["x"] = x.clamp(-E4M3_MAX, E4M3_MAX).to(TYPES["e4m3"])
    s["x_scale"] = 0.008 * torch.exp(0.5 * normal((m, blocks_of(k, BLOCK)), gen))
    w = normal((n, k), gen, torch.bfloat16) * 110
    s["w"] = w.clamp(-E4M3_MAX, E4M3_MAX).to(TYPES["e4m3"])
    s["w_scale"] = 0.009 / math.sqrt(k) * torch.exp(0.2 * normal((blocks_of(n, BLOCK), blocks_of(k, BLOCK)), gen))
    if own:
        ts, _ = library()
        s["out"] = torch.empty((m, n), device=DEVICE, dtype=TYPES[case["out"]])
        s["plan"] = ts.LinearE4m3(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"])


def prepare_rotary(s, case, gen):
    t, h, kv, d, bs = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    rows = normal((t, h + 2 * kv, d), gen, TYPES[case["kind"]]) * 3  # as one projection leaves them
    s["q"], s["k_new"], s["v_new"] = rows[:, :h], rows[:, h:h + kv], rows[:, h + kv:]
    positions = torch.randint(0, case["far"], (t,), device=DEVICE, generator=gen, dtype=torch.int32)
    unused = torch.randperm(t, device=DEVICE, generator=gen)[:case["skipped"]]
    positions[unused] = -1
    s["positions"] = positions
    i = torch.arange(case["rot"] // 2, device=DEVICE, dtype=torch.float64)
    s["freqs"] = 10000.0 ** (-2 * i / case["rot"]) / case["slower"]
    s["out"] = torch.zeros((t, h, d), device=DEVICE, dtype=TYPES[case["kind"]])  # unused rows stay as they are
    if kv:
        n_blocks = blocks_of(t, bs) + 2
        slots = torch.randperm(n_blocks, device=DEVICE, generator=gen)[:, None] * bs + torch.arange(bs, device=DEVICE)
        s["slots"] = slots.reshape(-1)[:t].clone()
        s["slots"][unused] = -1
        s["n_blocks"] = n_blocks
        # one block more than the pool: the plain form's place for unused tokens
        s["k"], s["v"] = (torch.zeros((n_blocks + 1, bs, kv, d), device=DEVICE, dtype=TYPES[case["cache"]]) for _ in range(2))
        s["k_scale"], s["v_scale"] = (size * (0.8 + 0.4 * torch.rand(kv, device=DEVICE, generator=gen)) if case["cache"] == "e4m3" else None
                                      for size in (0.03, 0.02))
    if own:
        ts, _ = library()
        s["plan"] = ts.Rotary(s["q"], s["out"], positions, s["freqs"], interleaved=case["layout"] == "pairs")
        if kv:
            s["cache"] = ts.KvCache(s["k"][:n_blocks], s["v"][:n_blocks], s["k_scale"], s["v_scale"])
            s["tokens"] = ts.KvTokens(s["k_new"], s["v_new"], s["slots"])


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"norm": run_norm, "gate": run_gate, "linear": run_linear, "rotary": run_rotary}[s["op"]](s)


def in_blocks(y):
    """[rows, dim] as [rows, blocks, 128], the last block filled up with zeros."""
    rows, dim = y.shape
    return torch.nn.functional.pad(y, (0, -dim % BLOCK)).view(rows, -1, BLOCK)


def stored(y, dtype):
    """`y` in the output's type: for 8 bits, each block of 128 over its scale."""
    if dtype != TYPES["e4m3"]:
        return {"out": y.to(dtype)}
    b = in_blocks(y)
    scale = b.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    q = (b / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)
    return {"out": q.view(y.shape[0], -1)[:, :y.shape[1]].contiguous(), "scale": scale}


def run_norm(s):
    if own:
        ts, handle = library()
        ts.ts_rms_norm(handle, s["plan"])
        return {"out": s["out"], "scale": s["scale"], "sum": s["sum"]}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    return {"scale": None, **stored(y, TYPES[s["case"]["out"]]), "sum": h.to(s["x"].dtype) if s["residual"] is not None else None}


def activated(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return g * 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def run_gate(s):
    if own:
        ts, handle = library()
        ts.ts_gate(handle, s["plan"])
        return {"out": s["out"], "scale": s["scale"]}
    y = s["up"].float()
    if s["gate"] is not None:
        y = activated(s["gate"].float(), s["case"]["act"]) * y
    return {"scale": None, **stored(y, TYPES[s["case"]["out"]])}


def values(x, scale, rows, dtype):
    """What 8-bit codes stand for: a scale for each `rows` rows and 128 columns."""
    n, k = x.shape
    scale = scale.to(dtype).repeat_interleave(rows, 0)[:n]
    return x.to(dtype) * scale.repeat_interleave(BLOCK, 1)[:, :k]


def run_linear(s):
    if own:
        ts, handle = library()
        ts.ts_linear_e4m3(handle, s["plan"])
        return {"out": s["out"]}
    x, w = values(s["x"], s["x_scale"], 1, torch.float32), values(s["w"], s["w_scale"], BLOCK, torch.float32)
    return {"out": torch.matmul(x, w.t()).to(TYPES[s["case"]["out"]])}


def turned(x, cos, sin, layout):
    """Rows [tokens, heads, dim] with their first elements turned in pairs."""
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def run_rotary(s):
    c = s["case"]
    if own:
        ts, handle = library()
        if c["kv_heads"] == 0:
            ts.ts_rotary(handle, s["plan"])
            return {"out": s["out"]}
        ts.ts_kv_append_rotary(handle, s["cache"], s["tokens"], s["plan"])
        return {"out": s["out"], "k": s["k"][:s["n_blocks"]], "v": s["v"][:s["n_blocks"]]}
    # far positions: angles in 64 bits
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    used = (s["positions"] >= 0)[:, None, None]
    got = {"out": torch.where(used, turned(s["q"].float(), cos, sin, c["layout"]).to(s["q"].dtype), s["out"])}
    if c["kv_heads"]:
        n_blocks, bs = s["n_blocks"], c["block"]
        slot = torch.where(s["slots"] >= 0, s["slots"], n_blocks * bs)
        where = (slot // bs, slot % bs)
        for name, x in (("k", turned(s["k_new"].float(), cos, sin, c["layout"])), ("v", s["v_new"].float())):
            bits_of(s[name])[where] = bits_of(in_cache(x, s[name + "_scale"], s[name].dtype))
            got[name] = s[name][:n_blocks]
    return got


def bits_of(x):
    return x.view(torch.uint8) if x.dtype == TYPES["e4m3"] else x


def in_cache(x, scale, dtype):
    return x.to(dtype) if scale is None else (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "gate"):
        rows, dim, es = case["rows"], case["dim"], SIZE[case["kind"]]
        moved = rows * dim * (es + SIZE[case["out"]]) + (4 * rows * blocks_of(dim, BLOCK) if case["out"] == "e4m3" else 0)
        if op == "norm":
            return {"bytes": moved + (2 * rows * dim * es if case["residual"] else 0) + 4 * dim, "flops": 5 * rows * dim}
        return {"bytes": moved + (rows * dim * es if case["act"] != "none" else 0), "flops": 8 * rows * dim}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * (m + blocks_of(n, BLOCK)) * blocks_of(k, BLOCK)
        return {"bytes": (m + n) * k + scales + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    t, es = case["tokens"] - case["skipped"], SIZE[case["kind"]]
    q, kv = t * case["heads"] * case["dim"], 2 * t * case["kv_heads"] * case["dim"]
    return {"bytes": 2 * q * es + kv * (es + SIZE[case["cache"]]) + (12 if kv else 4) * case["tokens"], "flops": 3 * (q + kv // 2)}


# --------------------------------------------------------------------------
# the definitions, in 64 bits, before the rounding to the outputs' types (what is
# beyond an 8-bit cache's largest value counts as that)
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "gate": exact_gate, "linear": exact_linear, "rotary": exact_rotary}[case["op"]](s, case)


def exact_stored(y, case):
    if case["out"] != "e4m3":
        return {"out": y}
    rows, dim = y.shape
    wide = torch.zeros((rows, blocks_of(dim, BLOCK) * BLOCK), dtype=torch.float64, device=DEVICE)
    wide[:, :dim] = y
    scale = torch.stack([b.abs().max(1).values for b in wide.split(BLOCK, 1)], 1)
    scale = torch.where(scale < LEAST, LEAST, scale) / E4M3_MAX
    return {"out": y / scale[:, torch.arange(dim, device=DEVICE) // BLOCK], "scale": scale}


def exact_norm(s, case):
    h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    y = h * torch.rsqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["dim"] + EPS) * s["weight"].double()
    return {**exact_stored(y, case), "sum": None if s["residual"] is None else h}


def exact_gate(s, case):
    y = s["up"].double()
    if s["gate"] is not None:
        g = s["gate"].double()
        if case["act"] == "silu":
            g = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            g = g * 0.5 * torch.erfc(-g / math.sqrt(2.0))
        else:  # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
            g = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        y = y * g
    return exact_stored(y, case)


def exact_linear(s, case):
    m, n, k = case["m"], case["n"], case["k"]
    x, w = s["x"].double(), s["w"].double()
    out = torch.zeros((m, n), dtype=torch.float64, device=DEVICE)
    of_row = torch.arange(n, device=DEVICE) // BLOCK
    for b, k0 in enumerate(range(0, k, BLOCK)):
        wb = w[:, k0:k0 + BLOCK] * s["w_scale"][of_row, b].double()[:, None]
        out.addmm_(x[:, k0:k0 + BLOCK] * s["x_scale"][:, b].double()[:, None], wb.t())
    return {"out": out}


def exact_rotary(s, case):
    """Pairs as complex numbers."""
    rot, half = case["rot"], case["rot"] // 2
    used = s["positions"] >= 0
    angle = s["positions"].double()[:, None] * s["freqs"]
    by = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(half, device=DEVICE) * (2 if case["layout"] == "pairs" else 1)
    second = first + (1 if case["layout"] == "pairs" else half)

    def turn(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y
    got = {"out": torch.where(used[:, None, None], turn(s["q"]), 0.0)}
    if case["kv_heads"]:
        for name, x in (("k", turn(s["k_new"])), ("v", s["v_new"].double())):
            if s[name + "_scale"] is not None:
                x = (x / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            cache = torch.zeros((s["n_blocks"] * case["block"], case["kv_heads"], case["dim"]), dtype=torch.float64, device=DEVICE)
            cache[s["slots"][used]] = x[used]
            got[name] = cache.view(s["n_blocks"], case["block"], case["kv_heads"], case["dim"])
    return got
