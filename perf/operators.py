"""The paged key-value cache's operators, as they are timed: block tables and
slot maps built on the GPU, new tokens' keys and values written to the cache,
and the attention of one new token per request over it.

``run`` computes them in elementary torch operations, or with ``own`` set
through the library's entry points."""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # one frame of 128 streams: each has one new token, a few have just stopped
        tables("tables_frame", n=128, len_lo=1, len_hi=2000, new_lo=1, new_hi=1, stopped=6, block=16),
        # prompts admitted together, the pool a little short of what they ask for
        tables("tables_prompts", n=1024, len_lo=0, len_hi=0, new_lo=1, new_hi=1500, stopped=0, block=16, short=40),
        # one frame of 32 streams, a layer with 8 key heads of 128
        append("append_frame", t=32, heads=8, dim=128, block=16, layout="nhd", kind="bf16", cache="bf16", skipped=2),
        # prompts into an 8-bit cache
        append("append_prompts_e4m3", t=65536, heads=8, dim=128, block=32, layout="hnd", kind="bf16", cache="e4m3", skipped=100),
        # odd sizes in 32 bits
        append("append_f32_odd", t=11111, heads=3, dim=80, block=24, layout="nhd", kind="f32", cache="f32", skipped=11),
        # the first frames of four streams: latency
        attention("attn_first_frames", n=4, len_lo=1, len_hi=40, heads=8, group=2, dim=128, block=16, layout="nhd", kind="bf16", cache="bf16"),
        # 32 streams of up to two minutes of frames, hidden size 1024
        attention("attn_32_streams", n=32, len_lo=100, len_hi=1500, heads=8, group=2, dim=128, block=16, layout="nhd", kind="bf16", cache="bf16"),
        # a full batch of 128 long requests, grouped heads
        attention("attn_128_long", n=128, len_lo=200, len_hi=8000, heads=8, group=4, dim=128, block=16, layout="hnd", kind="bf16", cache="bf16"),
        # one request with a very long context
        attention("attn_one_131071", n=1, len_lo=131071, len_hi=131071, heads=4, group=8, dim=128, block=64, layout="hnd", kind="bf16", cache="bf16"),
        # an 8-bit cache, long requests
        attention("attn_e4m3_64", n=64, len_lo=500, len_hi=16000, heads=8, group=8, dim=128, block=32, layout="nhd", kind="bf16", cache="e4m3"),
        # 32 bits, one query head per key head, odd sizes, evicted tokens masked out
        attention("attn_f32_masked", n=24, len_lo=1, len_hi=3001, heads=12, group=1, dim=80, block=24, layout="nhd", kind="f32", cache="f32", kept=0.75),
        # wide heads, a sliding window and capped scores
        attention("attn_window_256", n=48, len_lo=10, len_hi=6000, heads=2, group=8, dim=256, block=32, layout="hnd", kind="bf16", cache="bf16", window=1024, softcap=30.0),
    ]


def tables(name, *, n, len_lo, len_hi, new_lo, new_hi, stopped, block, short=0):
    return {"name": name, "op": "tables", "n": n, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "stopped": stopped, "block": block, "short": short}


def append(name, *, t, heads, dim, block, layout, kind, cache, skipped):
    return {"name": name, "op": "append", "t": t, "heads": heads, "dim": dim, "block": block, "layout": layout,
            "kind": kind, "cache": cache, "skipped": skipped}


def attention(name, *, n, len_lo, len_hi, heads, group, dim, block, layout, kind, cache, window=0, softcap=0.0, kept=1.0):
    return {"name": name, "op": "attention", "n": n, "len_lo": len_lo, "len_hi": len_hi, "heads": heads,
            "group": group, "dim": dim, "block": block, "layout": layout, "kind": kind, "cache": cache,
            "window": window, "softcap": softcap, "kept": kept}


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("tables", "append", "append", "attention", "attention", "attention"))
    block = rng.choice((8, 16, 16, 24, 32, 64, 128))
    layout = rng.choice(("nhd", "hnd"))
    kind, cache = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")))
    if op == "tables":
        n = log(1, 4000)
        hi = log(1, max(1, min(1500, 760000 // n)))
        len_hi = rng.choice((0, log(1, 4000)))
        c = tables("", n=n, len_lo=min(len_hi, rng.randrange(3)), len_hi=len_hi, new_lo=rng.choice((0, 1, hi)), new_hi=hi,
                   stopped=rng.randrange(n // 8 + 1), block=block, short=rng.choice((0, 0, rng.randrange(60))))
    elif op == "append":
        heads, dim = rng.choice((1, 2, 3, 5, 8, 12, 16)), rng.choice((48, 64, 80, 96, 128, 192, 256))
        t = log(1, max(2, min(65536, (1 << 26) // (heads * dim))))
        c = append("", t=t, heads=heads, dim=dim, block=block, layout=layout, kind=kind, cache=cache,
                   skipped=rng.randrange(t // 8 + 1))
    else:
        heads, group = rng.choice((1, 2, 3, 4, 8, 12)), rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
        dim = rng.choice((48, 64, 80, 96, 128, 128, 192, 256))
        n = log(1, 256)
        hi = log(1, max(2, min(131072, (1 << 28) // (n * heads * dim))))
        c = attention("", n=n, len_lo=rng.randrange(hi // 2 + 1), len_hi=hi, heads=heads, group=group, dim=dim, block=block,
                      layout=layout, kind=kind, cache=cache, window=rng.choice((0, 0, 0, log(1, 4096))),
                      softcap=rng.choice((0.0, 0.0, 20.0)), kept=rng.choice((1.0, 1.0, 1.0, 0.6)))
    c.pop("name")
    return c


def spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread: the same ones for every seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


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
        ts.ts_reserve_kv(_sampler.handle, 8192)
    return ts, _sampler.handle


def shuffled(values, gen):
    order = torch.randperm(len(values), generator=gen)
    return torch.tensor(values, dtype=torch.int32)[order]


def pool(case, n_blocks, gen, fill):
    """One half of a cache, seen as [block, token, head, dim] whatever its layout in memory."""
    b, h, d = case["block"], case["heads"], case["dim"]
    shape = (n_blocks, b, h, d) if case["layout"] == "nhd" else (n_blocks, h, b, d)
    if fill:
        x = torch.randn(shape, device=DEVICE, dtype=torch.bfloat16 if case["cache"] != "f32" else torch.float32, generator=gen)
        x = (x * 100).to(TYPES["e4m3"]) if case["cache"] == "e4m3" else x
    else:
        x = torch.zeros(shape, device=DEVICE, dtype=TYPES[case["cache"]])
    return x if case["layout"] == "nhd" else x.permute(0, 2, 1, 3)


def scales(case, gen, size):
    """One scale per key head of an 8-bit cache: about `size`, None for the wider types."""
    if case["cache"] != "e4m3":
        return None
    return size * (0.8 + 0.4 * torch.rand(case["heads"], device=DEVICE, generator=gen))


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"tables": prepare_tables, "append": prepare_append, "attention": prepare_attention}[case["op"]](s, case, host, gen)
    return s


def prepare_tables(s, case, host, gen):
    n, bs = case["n"], case["block"]
    lens = shuffled(spread(case["len_lo"], case["len_hi"], n), host)
    new = shuffled(spread(case["new_lo"], case["new_hi"], n), host)
    finished = shuffled([1] * case["stopped"] + [0] * (n - case["stopped"]), host).to(torch.uint8)
    wide = max(1, blocks_of(case["len_hi"] + case["new_hi"], bs))
    held = -(-lens // bs)
    need = torch.where(finished > 0, 0, -(-(lens + new) // bs) - held)
    used, free = int(held.sum()), int(need.sum())
    most_blocks = sum(blocks_of(x, bs) + 1 for x in spread(case["new_lo"], case["new_hi"], n))
    released = int(torch.where(finished > 0, held, 0).sum())
    n_free = max(0, free - released - case["short"])
    n_blocks = used + most_blocks + 8
    ids = torch.randperm(n_blocks, generator=host).to(torch.int32)
    table = torch.full((n, wide), -1, dtype=torch.int32)
    table[torch.arange(wide)[None, :] < held[:, None]] = ids[:used]
    stack = torch.full((n_blocks,), -1, dtype=torch.int32)
    stack[:n_free] = ids[used:used + n_free]
    most = sum(spread(case["new_lo"], case["new_hi"], n)) + 37
    s.update(lens=lens.to(DEVICE), new=new.to(DEVICE), finished=finished.to(DEVICE), table=table.to(DEVICE), stack=stack.to(DEVICE),
             n_free=torch.tensor([n_free], dtype=torch.int32, device=DEVICE), n_blocks=n_blocks, most=most)
    if own:
        ts, _ = library()
        s["plan"] = ts.KvTables(n, wide, n_blocks, bs, max_tokens=most, lens=s["lens"], n_new=s["new"], finished=s["finished"],
                                block_table=s["table"], free_blocks=s["stack"], n_free=s["n_free"], double=True)


def prepare_append(s, case, host, gen):
    t, h, d, bs = case["t"], case["heads"], case["dim"], case["block"]
    n_blocks = blocks_of(t, bs) + 2
    slots = torch.randperm(n_blocks, generator=host)[:, None] * bs + torch.arange(bs)
    slots = slots.reshape(-1)[:t].clone()
    slots[torch.randperm(t, generator=host)[:case["skipped"]]] = -1
    # one block more than the pool: the plain form's place for skipped tokens
    k, v = (pool(case, n_blocks + 1, gen, False) for _ in range(2))
    new = torch.randn((t, 2, h, d), device=DEVICE, generator=gen, dtype=TYPES[case["kind"]]) * 3  # as one projection leaves them
    s.update(k=k, v=v, k_new=new[:, 0], v_new=new[:, 1], slots=slots.to(DEVICE), n_blocks=n_blocks,
             k_scale=scales(case, gen, 0.03), v_scale=scales(case, gen, 0.02))
    if own:
        ts, _ = library()
        s["plan"] = (ts.KvCache(k[:n_blocks], v[:n_blocks], s["k_scale"], s["v_scale"]), ts.KvTokens(s["k_new"], s["v_new"], s["slots"]))


def prepare_attention(s, case, host, gen):
    n, h, g, d, bs = case["n"], case["heads"], case["group"], case["dim"], case["block"]
    lens = shuffled(spread(case["len_lo"], case["len_hi"], n), host)
    held, wide = -(-lens // bs), max(1, blocks_of(case["len_hi"], bs))
    used = int(held.sum())
    n_blocks = used + 5
    table = torch.full((n, wide), -1, dtype=torch.int32)
    table[torch.arange(wide)[None, :] < held[:, None]] = torch.randperm(n_blocks, generator=host)[:used].to(torch.int32)
    k, v = (pool(case, n_blocks, gen, True) for _ in range(2))
    # scores of a few units, as trained heads have them
    q = 2 * torch.randn((n, h * g, d), device=DEVICE, generator=gen, dtype=TYPES[case["kind"]])
    mask = (torch.rand((n, wide * bs), device=DEVICE, generator=gen) < case["kept"]).to(torch.uint8) if case["kept"] < 1 else None
    s.update(k=k, v=v, q=q, table=table.to(DEVICE), lens=lens.to(DEVICE), mask=mask, scale=1 / math.sqrt(d),
             k_scale=scales(case, gen, 0.01), v_scale=scales(case, gen, 0.01))
    if own:
        ts, _ = library()
        s["out"], s["lse"] = torch.empty_like(q), torch.empty((n, h * g), device=DEVICE)
        s["plan"] = (ts.KvCache(k, v, s["k_scale"], s["v_scale"]),
                     ts.PagedQuery(q, s["out"], s["table"], s["lens"], scale=s["scale"], lse=s["lse"], key_mask=mask,
                                   window=case["window"], softcap=case["softcap"]))


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"tables": run_tables, "append": run_append, "attention": run_attention}[s["op"]](s)


def run_tables(s):
    if own:
        ts, handle = library()
        p = s["plan"]
        ts.ts_kv_tables(handle, p)
        return {"lens": p.lens_out, "n_free": p.n_free_out, "table": p.block_table, "stack": p.free_blocks, "starts": p.token_starts,
                "slots": p.slots, "positions": p.positions, "requests": p.requests}
    bs, most, lens, table = s["case"]["block"], s["most"], s["lens"].long(), s["table"]
    n, wide = table.shape
    cols = torch.arange(wide, device=DEVICE)
    stop = s["finished"] > 0
    new = torch.where(stop, 0, s["new"].long())
    held = (lens + bs - 1) // bs
    freed = torch.where(stop, held, 0)
    need = torch.where(stop, 0, (lens + new + bs - 1) // bs - held)
    # released blocks go on the stack, in request and table order
    at = s["n_free"] + freed.cumsum(0) - freed
    spare = s["stack"].numel()
    stack = torch.cat([s["stack"], s["stack"][:1]])
    place = torch.where(cols < freed[:, None], at[:, None] + cols, spare)
    stack = stack.scatter(0, place.reshape(-1), table.reshape(-1))[:spare]
    top = s["n_free"] + freed.sum()
    # who gets what it asks for
    blocks, tokens = need.cumsum(0), new.cumsum(0)
    given = ~stop & ((new == 0) | (((need == 0) | (blocks <= top)) & (tokens <= most)))
    new, need_given = torch.where(given, new, 0), torch.where(given, need, 0)
    j = cols - held[:, None]
    source = (top - 1 - (blocks - need)[:, None] - j).clamp(0, spare - 1)
    table = torch.where((j >= 0) & (j < need_given[:, None]), stack[source], table)
    # the new tokens, packed in request order
    ends = new.cumsum(0)
    token = torch.arange(most, device=DEVICE)
    r = torch.searchsorted(ends, token, right=True)
    real = r < n
    r = r.clamp(max=n - 1)
    pos = lens[r] + token - (ends - new)[r]
    slot = table[r, (pos // bs).clamp(0, wide - 1)].long() * bs + pos % bs
    return {"lens": torch.where(stop, 0, lens + new).int(), "n_free": (top - need_given.sum()).int(), "table": table, "stack": stack,
            "starts": torch.cat([ends.new_zeros(1), ends]).int(), "slots": torch.where(real, slot, -1),
            "positions": torch.where(real, pos, -1).int(), "requests": torch.where(real, r, -1).int()}


def run_append(s):
    k, v, n_blocks, bs = s["k"], s["v"], s["n_blocks"], s["case"]["block"]
    if own:
        ts, handle = library()
        ts.ts_kv_append(handle, *s["plan"])
        return {"k": k[:n_blocks], "v": v[:n_blocks]}
    slot = torch.where(s["slots"] >= 0, s["slots"], n_blocks * bs)
    where = (slot // bs, slot % bs)
    for_cache(k)[where] = stored(s["k_new"], s["k_scale"], k.dtype)
    for_cache(v)[where] = stored(s["v_new"], s["v_scale"], v.dtype)
    return {"k": k[:n_blocks], "v": v[:n_blocks]}


def for_cache(x):
    return x.view(torch.uint8) if x.dtype == TYPES["e4m3"] else x


def stored(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)


def run_attention(s):
    if own:
        ts, handle = library()
        ts.ts_paged_attention(handle, *s["plan"])
        return {"out": s["out"], "lse": s["lse"]}
    c = s["case"]
    n, wide = s["table"].shape
    h, g, d, length = c["heads"], c["group"], c["dim"], wide * c["block"]
    pos = torch.arange(length, device=DEVICE)
    seen = pos < s["lens"][:, None]
    if c["window"]:
        seen = seen & (pos >= s["lens"][:, None] - c["window"])
    if s["mask"] is not None:
        seen = seen & (s["mask"][:, :length] > 0)
    rows = s["table"].clamp(min=0).long()

    def rows_of(x, scale):
        x = for_cache(x)[rows].view(x.dtype).float().reshape(n, length, h, d)
        return x if scale is None else x * scale[:, None]

    k = rows_of(s["k"], s["k_scale"])
    score = torch.einsum("nhgd,nlhd->nhgl", s["q"].float().view(n, h, g, d), k) * s["scale"]
    del k
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = rows_of(s["v"], s["v_scale"]).masked_fill(~seen[:, :, None, None], 0.0)
    out = torch.einsum("nhgl,nlhd->nhgd", p, v) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).view(n, h * g)
    return {"out": out.reshape(n, h * g, d).to(s["q"].dtype), "lse": lse}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        n, bs = case["n"], case["block"]
        lens, new = spread(case["len_lo"], case["len_hi"], n), spread(case["new_lo"], case["new_hi"], n)
        grown = blocks_of(sum(new), bs)  # about: blocks taken off the stack and put into tables
        most = sum(new) + 37
        return {"bytes": 9 * n + 8 * n + 8 * grown + 16 * most + 8 * blocks_of(sum(lens), bs) * case["stopped"] // max(n, 1), "flops": 0}
    h, d = case["heads"], case["dim"]
    if case["op"] == "append":
        t = case["t"] - case["skipped"]
        return {"bytes": 2 * t * h * d * (SIZE[case["kind"]] + SIZE[case["cache"]]) + 8 * case["t"], "flops": 0}
    lens = spread(case["len_lo"], case["len_hi"], case["n"])
    keys = sum(min(x, case["window"]) if case["window"] else x for x in lens)
    hq = h * case["group"]
    mask = keys if case["kept"] < 1 else 0
    keys *= case["kept"]
    return {"bytes": int(2 * keys * h * d * SIZE[case["cache"]]) + mask + 2 * case["n"] * hq * d * SIZE[case["kind"]] + 4 * case["n"] * hq
            + 4 * blocks_of(int(sum(lens)), case["block"]),
            "flops": int(4 * keys * hq * d)}


# --------------------------------------------------------------------------
# the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": exact_tables, "append": exact_append, "attention": exact_attention}[case["op"]](s, case)


def exact_tables(s, case):
    """One request after the other, one block after the other."""
    bs, most = case["block"], s["most"]
    lens, new, stop = s["lens"].tolist(), s["new"].tolist(), s["finished"].tolist()
    table, stack = s["table"].tolist(), s["stack"].tolist()
    top = s["n_free"].item()
    lens_out, starts, slots, positions, requests = [], [0], [], [], []
    for r, length in enumerate(lens):
        if stop[r]:
            for b in table[r][:blocks_of(length, bs)]:
                stack[top] = b
                top += 1
    left, asked, room = top, 0, True
    for r, length in enumerate(lens):
        want = 0 if stop[r] else new[r]
        need = 0 if stop[r] else blocks_of(length + want, bs) - blocks_of(length, bs)
        asked += want
        room = room and left >= need
        if want and ((need and not room) or asked > most):
            want = need = 0
        for j in range(need):
            left -= 1
            table[r][blocks_of(length, bs) + j] = stack[left]
        for p in range(length, length + want):
            slots.append(table[r][p // bs] * bs + p % bs)
            positions.append(p)
            requests.append(r)
        starts.append(len(slots))
        lens_out.append(0 if stop[r] else length + want)
    fill = [-1] * (most - len(slots))
    return {"lens": torch.tensor(lens_out, dtype=torch.int32), "n_free": torch.tensor([left], dtype=torch.int32),
            "table": torch.tensor(table, dtype=torch.int32), "stack": torch.tensor(stack, dtype=torch.int32),
            "starts": torch.tensor(starts, dtype=torch.int32), "slots": torch.tensor(slots + fill, dtype=torch.int64),
            "positions": torch.tensor(positions + fill, dtype=torch.int32), "requests": torch.tensor(requests + fill, dtype=torch.int32)}


def exact_append(s, case):
    bs, kept = case["block"], (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][kept]
    got = {}
    for name in ("k", "v"):
        x, scale = s[name + "_new"][kept].double(), s[name + "_scale"]
        if scale is not None:  # the nearest of the type's values, an even code where two are as near
            codes = torch.arange(127, dtype=torch.uint8, device=DEVICE).view(TYPES["e4m3"]).double()
            size = (x / scale.double()[:, None]).abs()
            above = torch.searchsorted(codes, size).clamp(1, 126)
            low, high = size - codes[above - 1], codes[above] - size
            code = torch.where((high < low) | ((high == low) & (above % 2 == 0)), above, above - 1)
            x = codes[code] * torch.sign(x)
        cache = torch.zeros((s["n_blocks"], bs, case["heads"], case["dim"]), dtype=torch.float64, device=DEVICE)
        cache[slot // bs, slot % bs] = x
        got[name] = cache
    return got


def exact_attention(s, case):
    n, h, g, d, bs = case["n"], case["heads"], case["group"], case["dim"], case["block"]
    out = torch.zeros((n, h, g, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((n, h, g), -math.inf, dtype=torch.float64, device=DEVICE)
    lens = s["lens"].tolist()
    for r in range(n):
        first = max(0, lens[r] - case["window"]) if case["window"] else 0
        keys = torch.arange(first, lens[r], device=DEVICE)
        if s["mask"] is not None:
            keys = keys[s["mask"][r, first:lens[r]] > 0]
        if not keys.numel():
            continue
        block, token = s["table"][r].long()[keys // bs], keys % bs
        k, v = (for_cache(s[x])[block, token].view(s[x].dtype).to(torch.float64) for x in ("k", "v"))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        z = torch.matmul(s["q"][r].double().view(h, g, d), k.permute(1, 2, 0)) * s["scale"]
        if case["softcap"]:
            z = case["softcap"] * torch.tanh(z / case["softcap"])
        lse[r] = torch.logsumexp(z, -1)
        out[r] = torch.matmul(torch.exp(z - lse[r][..., None]), v.transpose(0, 1))
    return {"out": out.reshape(n, h * g, d), "lse": lse.reshape(n, h * g)}
