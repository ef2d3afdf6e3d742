"""The paged cache's operators against their plain 64-bit versions: block
tables and slot maps, cache writes, and the attention of one new token."""
import numpy as np
import pytest

from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ts():
    import codebook_token_sampling_gb300 as mod
    return mod


@pytest.fixture(scope="module")
def sampler(ts):
    s = ts.Sampler(0)
    s.reserve_kv(8192)
    yield s
    s.close()


# --------------------------------------------------------------------------
# Block tables and slot maps (whole numbers: equal)
# --------------------------------------------------------------------------
def tables_state(rng, n, *, block_size, len_hi, new_hi, finished=0.0, short=0, wide=None, spare=4):
    lens = rng.integers(0, len_hi + 1, n).astype(np.int32)
    new = rng.integers(0, new_hi + 1, n).astype(np.int32)
    fin = (rng.random(n) < finished).astype(np.uint8)
    wide = max(1, -(-(len_hi + new_hi) // block_size)) if wide is None else wide
    held = -(-lens // block_size)
    need = np.where(fin > 0, 0, -(-(lens + new) // block_size) - held)
    free = max(0, int(need.sum() - held[fin > 0].sum()) - short)
    used = int(held.sum())
    n_blocks = used + max(free, int(need.sum())) + spare
    ids = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((n, wide), -7, np.int32)
    table[np.arange(wide)[None, :] < held[:, None]] = ids[:used]
    stack = np.full(n_blocks, -9, np.int32)
    stack[:free] = ids[used:used + free]
    return {"block_table": table, "lens": lens, "n_new": new, "finished": fin, "free_blocks": stack,
            "n_free": free, "block_size": block_size, "n_blocks": n_blocks,
            "max_tokens": int(new.sum()) + 5}


def run_tables(ts, sampler, st, *, double, pad=0, stream=None):
    import torch
    dev = "cuda"
    n, wide = st["block_table"].shape
    table = torch.full((n, wide + pad), -3, dtype=torch.int32, device=dev)
    table[:, :wide] = torch.from_numpy(st["block_table"]).to(dev)

    def put(x):
        return None if x is None else torch.from_numpy(np.array(x)).to(dev)
    t = ts.KvTables(n, wide, st["n_blocks"], st["block_size"], max_tokens=st["max_tokens"],
                    lens=put(st["lens"]), n_new=put(st["n_new"]), finished=put(st["finished"]),
                    block_table=table[:, :wide], free_blocks=put(st["free_blocks"]),
                    n_free=put(np.array([st["n_free"]], np.int32)), double=double)
    sampler.read_status()
    ts.ts_kv_tables(sampler.handle, t, stream)
    torch.cuda.synchronize()
    got = {"block_table": t.block_table, "free_blocks": t.free_blocks, "lens": t.lens_out,
           "token_starts": t.token_starts, "slots": t.slots, "positions": t.positions,
           "requests": t.requests}
    got = {k: v.cpu().numpy() for k, v in got.items()}
    got["n_free"] = int(t.n_free_out.item())
    got["status"] = sampler.read_status()
    assert pad == 0 or bool((table[:, wide:] == -3).all())
    return got


def check_tables(ts, sampler, st, **how):
    want = okv.tables(st["block_table"], st["lens"], st["n_new"], st["finished"], st["free_blocks"],
                      st["n_free"], block_size=st["block_size"], n_blocks=st["n_blocks"],
                      max_tokens=st["max_tokens"])
    got = run_tables(ts, sampler, st, **how)
    for key, w in want.items():
        assert np.array_equal(got[key], w), (key, got[key], w)
    return want


@pytest.mark.parametrize("double", [False, True])
@pytest.mark.parametrize("n,block_size,len_hi,new_hi,finished,short", [
    (1, 16, 0, 1, 0.0, 0), (1, 1, 3, 2, 0.0, 0), (5, 16, 40, 1, 0.3, 0), (37, 7, 100, 30, 0.2, 0),
    (128, 16, 2000, 1, 0.1, 0), (257, 24, 50, 9, 0.3, 40), (1000, 16, 0, 60, 0.0, 90),
    (1025, 128, 300, 3, 0.5, 3), (64, 16, 64, 300, 0.1, 25), (3000, 8, 20, 12, 0.1, 0),
    (150, 16, 30, 700, 0.1, 60), (40, 6, 30, 2500, 0.0, 7),
    (8192, 16, 40, 2, 0.2, 11)])
def test_tables(ts, sampler, n, block_size, len_hi, new_hi, finished, short, double):
    rng = np.random.default_rng([n, block_size, len_hi, new_hi, short])
    st = tables_state(rng, n, block_size=block_size, len_hi=len_hi, new_hi=new_hi, finished=finished,
                      short=short)
    want = check_tables(ts, sampler, st, double=double, pad=3 if n > 1 else 0)
    held = -(-st["lens"] // block_size)
    ends = st["finished"] > 0
    need = np.where(ends, 0, -(-(st["lens"] + st["n_new"]) // block_size) - held).sum()
    assert bool(want["status"] & okv.NO_BLOCKS) == bool(need > st["n_free"] + held[ends].sum())


def test_tables_sums_past_32_bits(ts, sampler):
    """Table rows that could hold more than 2^31 tokens together (64-bit sums)."""
    rng = np.random.default_rng(9)
    st = tables_state(rng, 40, block_size=65536, len_hi=300000, new_hi=4000, finished=0.2, wide=1024)
    for double in (False, True):
        check_tables(ts, sampler, st, double=double)


def test_tables_one_token_each_and_a_short_map(ts, sampler):
    rng = np.random.default_rng(5)
    st = tables_state(rng, 60, block_size=16, len_hi=100, new_hi=1)
    st.update(n_new=None, finished=None)
    held = -(-st["lens"] // 16)
    need = int((-(-(st["lens"] + 1) // 16) - held).sum())
    used = int(held.sum())
    st["n_blocks"] = st["free_blocks"].size + 60
    st["free_blocks"] = np.full(st["n_blocks"], -1, np.int32)
    rest = np.setdiff1d(np.arange(st["n_blocks"]), st["block_table"][st["block_table"] >= 0])
    st["free_blocks"][:need] = rest[:need]
    st["n_free"] = need
    for most in (60, 33, 1, 0):
        st["max_tokens"] = most
        want = check_tables(ts, sampler, st, double=True)
        assert want["token_starts"][-1] == most
    assert used > 0


def test_tables_everything_ends(ts, sampler):
    rng = np.random.default_rng(6)
    st = tables_state(rng, 70, block_size=16, len_hi=200, new_hi=1)
    st["finished"] = np.ones(70, np.uint8)
    want = check_tables(ts, sampler, st, double=False)
    assert want["token_starts"][-1] == 0 and not want["lens"].any()


def test_tables_errors(ts, sampler):
    """Lengths, counts, blocks and a stack that are out of range."""
    rng = np.random.default_rng(7)
    st = tables_state(rng, 40, block_size=16, len_hi=100, new_hi=20, finished=0.2)
    st["finished"][[3, 5, 9]] = 0
    st["lens"][3], st["n_new"][5] = -4, -1
    st["lens"][9] = st["block_table"].shape[1] * 16 + 1
    assert check_tables(ts, sampler, st, double=True)["status"] & okv.BAD_SHAPE
    st = tables_state(rng, 40, block_size=16, len_hi=100, new_hi=20)
    st["lens"][0], st["n_new"][0] = 15, 2
    st["block_table"][0, 0] = st["n_blocks"]
    st["free_blocks"][st["n_free"] - 1] = -1
    st["max_tokens"] += 100
    assert check_tables(ts, sampler, st, double=True)["status"] & okv.BAD_BLOCK
    st = tables_state(rng, 40, block_size=16, len_hi=100, new_hi=2, finished=0.5)
    for n_free in (-3, st["free_blocks"].size + 2, st["free_blocks"].size - 1):
        st["n_free"] = n_free
        st["free_blocks"][:] = np.arange(st["free_blocks"].size)
        assert check_tables(ts, sampler, st, double=False)["status"] & okv.BAD_SHAPE


def test_the_longest_token_maps(ts, sampler):
    """Maps of 2^31 - 1 entries: the tokens there are in front, then -1; and a cache
    write of as many tokens, all but those skipped."""
    import torch
    most, block = 2 ** 31 - 1, 6
    st = tables_state(np.random.default_rng(11), 50, block_size=block, len_hi=40, new_hi=90)
    want = okv.tables(st["block_table"], st["lens"], st["n_new"], None, st["free_blocks"], st["n_free"],
                      block_size=block, n_blocks=st["n_blocks"], max_tokens=st["max_tokens"])
    put = {k: torch.from_numpy(st[k]).cuda() for k in ("lens", "n_new", "block_table", "free_blocks")}
    slots = torch.zeros(most, dtype=torch.int64, device="cuda")
    t = ts.KvTables(50, st["block_table"].shape[1], st["n_blocks"], block, max_tokens=1, double=True,
                    n_free=torch.tensor([st["n_free"]], dtype=torch.int32, device="cuda"), **put)
    t.c.max_tokens, t.c.slots, t.c.positions, t.c.requests = most, slots.data_ptr(), None, None
    sampler.read_status()
    ts.ts_kv_tables(sampler.handle, t)
    n = int(want["token_starts"][-1])
    assert 1000 < n < st["max_tokens"]
    assert np.array_equal(slots[:n].cpu().numpy(), want["slots"][:n])
    assert int(slots[n:].max()) == int(slots[n:].min()) == -1
    assert np.array_equal(t.token_starts.cpu().numpy(), want["token_starts"])
    assert np.array_equal(t.lens_out.cpu().numpy(), want["lens"]) and int(t.n_free_out) == want["n_free"]
    assert np.array_equal(t.block_table.cpu().numpy(), want["block_table"])
    k, v = cache_pair(torch, st["n_blocks"], block, 1, 8, torch.bfloat16, "nhd")
    new = torch.arange(8, device="cuda").bfloat16().view(1, 1, 8).expand(most, 1, 8)
    ts.ts_kv_append(sampler.handle, ts.KvCache(k, v), ts.KvTokens(new, new, slots))
    torch.cuda.synchronize()
    assert sampler.read_status() == want["status"] == 0
    there = np.zeros(st["n_blocks"] * block, bool)
    there[want["slots"][:n]] = True
    before = raw(torch, cache_pair(torch, 1, 1, 1, 8, torch.bfloat16, "nhd")[0])[0, 0, 0]
    for x in (k, v):
        got = raw(torch, x).reshape(-1, 8)
        assert np.array_equal(got[there], np.broadcast_to(raw(torch, new[0, 0]), (n, 8)))
        assert np.array_equal(got[~there], np.broadcast_to(before, (there.size - n, 8)))


def test_tables_refusals(ts, sampler):
    import torch
    st = tables_state(np.random.default_rng(8), 6, block_size=16, len_hi=50, new_hi=1)

    def make():
        t = ts.KvTables(6, st["block_table"].shape[1], st["n_blocks"], 16, max_tokens=6)
        return t
    bad = [("n_requests", -1, ts.TS_ERR_INVALID_ARG), ("block_size", 0, ts.TS_ERR_INVALID_ARG),
           ("block_size", 65537, ts.TS_ERR_UNSUPPORTED), ("max_tokens", -1, ts.TS_ERR_INVALID_ARG),
           ("table_stride", 0, ts.TS_ERR_INVALID_ARG), ("lens", None, ts.TS_ERR_INVALID_ARG),
           ("slots", None, ts.TS_ERR_INVALID_ARG), ("token_starts", None, ts.TS_ERR_INVALID_ARG),
           ("n_requests", 8193, ts.TS_ERR_UNSUPPORTED)]
    for field, value, status in bad:
        t = make()
        setattr(t.c, field, value)
        with pytest.raises(ts.SamplerError) as e:
            ts.ts_kv_tables(sampler.handle, t)
        assert e.value.status == status, field
    t = make()
    t.c.max_blocks = t.c.table_stride = 1 << 28
    with pytest.raises(ts.SamplerError) as e:
        ts.ts_kv_tables(sampler.handle, t)
    assert e.value.status == ts.TS_ERR_UNSUPPORTED
    t = make()
    t.c.lens_out = t.c.lens + 4
    with pytest.raises(ts.SamplerError):
        ts.ts_kv_tables(sampler.handle, t)
    fresh = ts.Sampler(0)  # no workspace
    with pytest.raises(ts.SamplerError):
        ts.ts_kv_tables(fresh.handle, make())
    fresh.close()
    t = make()
    t.c.n_requests = 0
    ts.ts_kv_tables(sampler.handle, t)
    with pytest.raises(ValueError):
        t.set_requests(n_new=torch.zeros(6, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert sampler.read_status() == 0


def test_tables_overlapping_arrays(ts, sampler):
    """An output that shares memory with an input or another output is refused;
    arrays side by side, and lengths and free count in place, are not."""
    import torch
    n, most = 6, 8

    def make(**at):
        t = ts.KvTables(n, 3, 18, 16, max_tokens=most, double=True, n_new=torch.ones(n, dtype=torch.int32, device="cuda"),
                        finished=torch.zeros(n, dtype=torch.uint8, device="cuda"))
        for name, value in at.items():
            setattr(t.c, name, value(t))
        return t
    outs = {"lens_out": 4 * n, "n_free_out": 4, "token_starts": 4 * (n + 1), "slots": 8 * most, "positions": 4 * most,
            "requests": 4 * most, "free_blocks": 4 * 18}
    ins = {"lens": 4 * n, "n_new": 4 * n, "finished": n, "n_free": 4}
    sampler.read_status()
    for out in outs:
        for other, size in {**ins, **outs}.items():
            if other == out:
                continue
            inside = [0, size - 1 & ~7] if out == "slots" else [0, size - 1 & ~3]
            for by in inside:
                if by == 0 and (out, other) in (("lens_out", "lens"), ("n_free_out", "n_free")):
                    continue
                with pytest.raises(ts.SamplerError) as e:
                    ts.ts_kv_tables(sampler.handle, make(**{out: lambda t, b=by: getattr(t.c, other) + b}))
                assert e.value.status == ts.TS_ERR_INVALID_ARG, (out, other, by)
    whole = torch.zeros(64, dtype=torch.int32, device="cuda")  # one array after the other
    at = whole.data_ptr()
    for t in (make(lens_out=lambda t: t.c.lens, n_free_out=lambda t: t.c.n_free),
              make(lens_out=lambda t: at, token_starts=lambda t: at + 4 * n, positions=lambda t: at + 4 * (2 * n + 1),
                   requests=lambda t: at + 4 * (2 * n + 1 + most), n_free_out=lambda t: at + 4 * (2 * n + 1 + 2 * most))):
        ts.ts_kv_tables(sampler.handle, t)
    torch.cuda.synchronize()
    want = [1] * n + list(range(n + 1)) + [0] * n + [-1] * 2 + list(range(n)) + [-1] * 2 + [12]
    assert whole.tolist()[:len(want)] == want and not whole[len(want):].any()
    assert sampler.read_status() == 0


# --------------------------------------------------------------------------
# Cache writes (bits: equal)
# --------------------------------------------------------------------------
def cache_pair(torch, n_blocks, block, heads, dim, dtype, layout, fill=0x55):
    """K and V bytes set to a pattern, seen as [block, token, head, dim]."""
    size = {torch.float32: 4, torch.bfloat16: 2, torch.float8_e4m3fn: 1}[dtype]
    pair = []
    for _ in range(2):
        shape = (n_blocks, block, heads, dim * size) if layout == "nhd" else (n_blocks, heads, block, dim * size)
        x = torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(dtype)
        pair.append(x if layout == "nhd" else x.permute(0, 2, 1, 3))
    return pair


def raw(torch, x):
    """The bits of a tensor as a numpy array."""
    kind = {4: torch.int32, 2: torch.int16, 1: torch.uint8}[x.element_size()]
    return x.contiguous().view(kind).cpu().numpy()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("t,heads,dim,block,layout,offset", [
    (1, 1, 16, 16, "nhd", 0), (7, 3, 80, 5, "hnd", 0), (33, 8, 128, 16, "nhd", 1), (129, 2, 256, 64, "hnd", 0),
    (300, 5, 48, 1, "nhd", 0), (2000, 12, 96, 24, "hnd", 3), (40, 100, 256, 16, "nhd", 0)])
def test_append(ts, sampler, kind, cache, t, heads, dim, block, layout, offset):
    import torch
    types = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
    gen = torch.Generator(device="cuda").manual_seed(t * heads + dim)
    n_blocks = -(-t // block) + 3
    k, v = cache_pair(torch, n_blocks, block, heads, dim, types[cache], layout)
    # rows of one projection, at an offset that may break 16-byte alignment
    wide = torch.randn((t, 2 * heads * dim + offset + 4), device="cuda", generator=gen) * 30
    wide[0, offset] = 1e9
    wide = wide.to(types[kind])
    kn = wide[:, offset:offset + heads * dim].view(t, heads, dim)
    vn = wide[:, offset + heads * dim:offset + 2 * heads * dim].view(t, heads, dim)
    rng = np.random.default_rng(t)
    slots = rng.permutation(n_blocks * block)[:t].astype(np.int64)
    slots[::5] = -1
    if t > 3:
        slots[3] = n_blocks * block  # past the cache
        slots[1] = n_blocks * block - 1 if n_blocks * block - 1 not in slots else slots[1]
    scales = [None, None]
    if cache == "e4m3":
        scales = [(torch.rand(heads, device="cuda", generator=gen) + 0.1) * s for s in (0.07, 1.0)]
    want = []
    for x, new, scale in ((k, kn, scales[0]), (v, vn, scales[1])):
        w = raw(torch, x).copy()
        for i, s in enumerate(slots):
            if 0 <= s < n_blocks * block:
                if cache == "e4m3":
                    y = new[i].float().cpu().numpy() / scale.cpu().numpy()[:, None]
                    w[s // block, s % block] = okv.to_e4m3(y)
                else:
                    w[s // block, s % block] = raw(torch, new[i])
        want.append(w)
    sampler.read_status()
    c = ts.KvCache(k, v, *scales)
    ts.ts_kv_append(sampler.handle, c, ts.KvTokens(kn, vn, torch.from_numpy(slots).cuda()))
    torch.cuda.synchronize()
    assert sampler.read_status() == (ts.TS_ROW_BAD_SLOT if t > 3 else 0)
    for x, w in zip((k, v), want):
        assert np.array_equal(raw(torch, x), w)


def test_append_e4m3_rounding(ts, sampler):
    """Every tie between two e4m3 values, values beyond 448, infinities, NaN,
    zeros and subnormals, with a scale of 1."""
    import torch
    vals = okv.e4m3_values()
    mid = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 1e9),
                        [448.1, 464.0, 480.0, 1e30, np.inf, np.nan, 1e-30, 2.0 ** -10, 2.0 ** -11]]).astype(np.float32)
    x = np.concatenate([x, -x])
    x = np.concatenate([x, np.zeros(-x.size % 16, np.float32)])
    k, v = cache_pair(torch, x.size // 16, 1, 1, 16, torch.float8_e4m3fn, "nhd")
    new = torch.from_numpy(x).cuda().view(-1, 1, 16)
    ts.ts_kv_append(sampler.handle, ts.KvCache(k, v), ts.KvTokens(new, new, torch.arange(new.shape[0], device="cuda")))
    got, want = raw(torch, k).reshape(-1), okv.to_e4m3(x)
    nan = np.isnan(x)
    assert np.array_equal(got[~nan], want[~nan])
    assert np.all(got[nan] & 0x7F == 0x7F)
    assert np.array_equal(raw(torch, v).reshape(-1), got)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_rows(ts, sampler, cache):
    """Tokens in other rows than their own: a row twice, rows out of range (bit
    set, skipped), a skipped token's row not looked at."""
    import torch
    types = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
    k, v = cache_pair(torch, 3, 8, 2, 64, types[cache], "nhd")
    before = raw(torch, k).copy()
    new = torch.randn((5, 2, 2, 64), device="cuda").bfloat16()
    rows = torch.tensor([4, 0, 4, 2, 9, -1, 5, 1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 20, 7, -1, -1, 11, 12, 23], device="cuda")
    sampler.read_status()
    ts.ts_kv_append(sampler.handle, ts.KvCache(k, v), ts.KvTokens(new[:, 0], new[:, 1], slots, rows))
    torch.cuda.synchronize()
    assert sampler.read_status() == ts.TS_ROW_BAD_SLOT
    for x, i in ((k, 0), (v, 1)):
        want = before.copy()
        for s, r in ((3, 4), (20, 0), (7, 4), (23, 1)):
            y = new[r, i]
            want[s // 8, s % 8] = okv.to_e4m3(y.float().cpu().numpy()) if cache == "e4m3" else raw(torch, y)
        assert np.array_equal(raw(torch, x), want)


@pytest.mark.parametrize("scale", [0.03, 1.0 / 3.0, 7.3e-5, 448.0, 1e-30, 3e30, 2.0 ** -100])
def test_append_e4m3_scales(ts, sampler, scale):
    """Values around every tie times the scale, at scales from tiny to huge: the
    fp32 quotient, rounded once more."""
    import torch
    scale = np.float32(scale)
    vals = okv.e4m3_values()
    mid = np.concatenate([(vals[1:] + vals[:-1]) / 2, vals])
    rng = np.random.default_rng(3)
    with np.errstate(over="ignore"):
        at = (mid * float(scale)).astype(np.float32)
        x = np.concatenate([at] + [np.nextafter(at, np.float32(s), dtype=np.float32) for s in (0, 3e38)]
                           + [(rng.normal(0, 100, 20000) * float(scale)).astype(np.float32)])
        x = np.concatenate([x, -x, np.array([np.inf, -np.inf, 3e38, -3e38, 0.0, -0.0], np.float32)])
        x = np.concatenate([x, np.zeros(-x.size % 16, np.float32)])
        want = okv.to_e4m3(x / scale)
    k, v = cache_pair(torch, x.size // 16, 1, 1, 16, torch.float8_e4m3fn, "nhd")
    new = torch.from_numpy(x).cuda().view(-1, 1, 16)
    sc = torch.tensor([float(scale)], device="cuda")
    ts.ts_kv_append(sampler.handle, ts.KvCache(k, v, sc, sc), ts.KvTokens(new, new, torch.arange(new.shape[0], device="cuda")))
    assert np.array_equal(raw(torch, k).reshape(-1), want)
    assert np.array_equal(raw(torch, v).reshape(-1), want)


def test_append_refusals(ts, sampler):
    import torch
    k, v = cache_pair(torch, 4, 16, 2, 64, torch.bfloat16, "nhd")
    new = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")

    def go(field=None, value=None, cfield=None, cvalue=None, tokens=new):
        c, t = ts.KvCache(k, v), ts.KvTokens(tokens, tokens, slots)
        if field:
            setattr(t.c, field, value)
        if cfield:
            setattr(c.c, cfield, cvalue)
        with pytest.raises(ts.SamplerError) as e:
            ts.ts_kv_append(sampler.handle, c, t)
        return e.value.status
    inv, uns = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    assert go("n_tokens", -1) == inv and go("slots", None) == inv and go("dtype", 2) == inv
    assert go("k_token_stride", -1) == inv and go("k", new.data_ptr() + 1) == inv
    assert go(cfield="head_dim", cvalue=60) == inv and go(cfield="head_dim", cvalue=264) == uns
    assert go(cfield="k", cvalue=k.data_ptr() + 2) == inv and go(cfield="v_head_stride", cvalue=63) == inv
    assert go(cfield="k_scale", cvalue=slots.data_ptr()) == inv and go(cfield="n_blocks", cvalue=0) == inv
    assert go(cfield="dtype", cvalue=7) == inv and go(cfield="v_block_stride", cvalue=1 << 30) == uns
    assert go(cfield="block_size", cvalue=65537) == uns
    assert go(tokens=new.float()) == uns  # fp32 tokens for a bf16 cache
    with pytest.raises(ValueError):
        ts.KvTokens(new, new, slots.int())
    with pytest.raises(ValueError):
        ts.KvCache(k.half(), v.half())
    t = ts.KvTokens(new[:0], new[:0], slots[:0])
    ts.ts_kv_append(sampler.handle, ts.KvCache(k, v), t)
    torch.cuda.synchronize()
    assert bool((k.view(torch.uint8) == 0x55).all()) and sampler.read_status() == 0


# --------------------------------------------------------------------------
# Attention
# --------------------------------------------------------------------------
def attention_case(torch, seed, lens, *, heads, group, dim, block, layout, kind, window=0, softcap=0.0,
                   masked=None, spread=2.0, stale=True, q_pad=0):
    """Inputs on the GPU; whatever a call may not read holds NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    n = lens.size
    wide = max(1, int(-(-lens.max(initial=1) // block)) + 1)
    held = -(-lens // block)
    n_blocks = int(held.sum()) + 3
    table = rng.integers(-2**31, 2**31, (n, wide)).astype(np.int32)  # unused entries are anything
    table[np.arange(wide)[None, :] < held[:, None]] = rng.permutation(n_blocks)[:held.sum()]
    qtype = torch.float32 if kind == "f32" else torch.bfloat16
    pair, scales = [], [None, None]
    for i in range(2):
        shape = (n_blocks, block, heads, dim) if layout == "nhd" else (n_blocks, heads, block, dim)
        x = torch.randn(shape, device="cuda", generator=gen)
        if kind == "e4m3":
            x = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            scales[i] = (0.5 + torch.rand(heads, device="cuda", generator=gen)) / 60
        else:
            x = x.to(qtype)
        pair.append(x if layout == "nhd" else x.permute(0, 2, 1, 3))
    k, v = pair
    mask = None
    if masked is not None:
        mask = (rng.random((n, wide * block)) >= masked).astype(np.uint8) * 3
        mask[n // 2] = 0
    if stale:  # places outside every attended set
        seen = np.zeros((n_blocks, block), bool)
        for r in range(n):
            t = np.arange(lens[r])
            t = t[t >= lens[r] - window] if window else t
            t = t[mask[r, t] != 0] if mask is not None else t
            seen[table[r, t // block], t % block] = True
        gone = torch.from_numpy(~seen).cuda()
        for x in pair:
            if kind == "e4m3":
                x.view(torch.uint8)[gone] = 0x7F
            else:
                x[gone] = float("nan")
                x[gone.nonzero()[:1, 0], gone.nonzero()[:1, 1]] = float("inf")
    q = (spread * torch.randn((n, heads * group * dim + q_pad), device="cuda", generator=gen)).to(qtype)
    q = q[:, q_pad:].view(n, heads * group, dim)
    return {"q": q, "k": k, "v": v, "k_scale": scales[0], "v_scale": scales[1], "lens": lens, "table": table,
            "mask": mask, "window": window, "softcap": softcap, "scale": float(np.float32(dim ** -0.5)),
            "n_blocks": n_blocks, "kind": kind}


def run_attention(ts, sampler, c, stream=None):
    import torch
    q = c["q"]
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    mask = torch.from_numpy(c["mask"]).cuda() if c["mask"] is not None else None
    query = ts.PagedQuery(q, out, torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda(),
                          scale=c["scale"], lse=lse, key_mask=mask, window=c["window"], softcap=c["softcap"])
    cache = ts.KvCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    sampler.read_status()
    ts.ts_paged_attention(sampler.handle, cache, query, stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy(), sampler.read_status()


def want_attention(torch, c):
    def host(x):
        if x.dtype == torch.float8_e4m3fn:
            return okv.from_e4m3(x.contiguous().view(torch.uint8).cpu().numpy())
        return x.float().cpu().numpy()
    return okv.attention(host(c["q"]), host(c["k"]), host(c["v"]), c["table"], c["lens"], scale=c["scale"],
                         n_blocks=c["n_blocks"], window=c["window"], softcap=c["softcap"], key_mask=c["mask"],
                         k_scale=None if c["k_scale"] is None else c["k_scale"].cpu().numpy(),
                         v_scale=None if c["v_scale"] is None else c["v_scale"].cpu().numpy())


def assert_attention(c, want, got, lse):
    """The bounds.  A score is a sum of dim products in fp32 (one unit of 2^-23
    per product of the sum of their sizes), scaled, perhaps capped (a few units
    of the cap), and its weight an exp2 of it; the weights' and outputs' sums add
    2^-24 per key.  On the way into the tensor cores a weight keeps 2^-16 of
    itself (two bf16 numbers) or 2^-11 and at least 2^-25 (f16, of a largest
    weight of 1), a query row next to an e4m3 cache 2^-24 of its largest element.
    The output is rounded once to bf16 (2^-8 of it covers that) or fp32."""
    dim = c["q"].shape[2]
    n = want["keys"][:, None]
    size = np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0))
    err = dim * 2.0 ** -23 * want["dot"] + 2.0 ** -21 * (size + want["dot"]) + 2.0 ** -20 * c["softcap"]
    if c["kind"] == "e4m3":
        err = err + dim * 2.0 ** -24 * want["dot"]
    weight = {"bf16": 2.0 ** -15, "e4m3": 2.0 ** -10, "f32": 2.0 ** -21}[c["kind"]]
    last = 2.0 ** -22 if c["kind"] == "f32" else 2.0 ** -8
    bound = want["abs_v"] * (4 * err + n * 2.0 ** -23 + weight)[..., None] + last * np.abs(want["out"])
    if c["kind"] == "e4m3":
        bound = bound + (n * 2.0 ** -24 * want["max_v"])[..., None]
    assert np.array_equal(np.isnan(got), np.isnan(want["out"]))
    off = np.abs(got - want["out"]) - bound - 1e-37
    assert np.nanmax(off, initial=-1) <= 0, (np.nanmax(off), np.unravel_index(np.nanargmax(off), off.shape))
    assert np.array_equal(np.isneginf(lse), np.isneginf(want["lse"]))
    fine = np.isfinite(want["lse"])
    assert np.array_equal(fine, np.isfinite(lse))
    lim = (2 * err + n * 2.0 ** -23 + 2.0 ** -20) * np.ones_like(lse)
    assert np.all(np.abs(lse[fine] - want["lse"][fine]) <= lim[fine])


def check_attention(ts, sampler, c, **how):
    import torch
    want = want_attention(torch, c)
    got, lse, status = run_attention(ts, sampler, c, **how)
    assert status == want["status"]
    assert_attention(c, want, got, lse)
    return got, lse


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 0, 128, 200, 255, 257, 511]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 144, 192, 256])
@pytest.mark.parametrize("group,block,layout", [(1, 16, "nhd"), (2, 24, "hnd"), (5, 7, "nhd"), (16, 64, "hnd"),
                                                (20, 1, "nhd")])
def test_attention_shapes(ts, sampler, kind, dim, group, block, layout):
    import torch
    heads = 1 if group == 20 else 3
    c = attention_case(torch, dim + group, EDGES, heads=heads, group=group, dim=dim, block=block, layout=layout, kind=kind)
    check_attention(ts, sampler, c)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("window,softcap,masked", [(1, 0.0, None), (16, 0.0, 0.5), (100, 5.0, None), (0, 30.0, 0.3),
                                                   (0, 0.0, 0.97), (1000, 0.0, 0.1)])
@pytest.mark.parametrize("block", [16, 10])
def test_attention_masks(ts, sampler, kind, window, softcap, masked, block):
    """Windows, key masks (one request's leaves nothing) and capped scores; what
    is not attended to holds NaN and infinities."""
    import torch
    c = attention_case(torch, 3, EDGES, heads=2, group=4, dim=64, block=block, layout="nhd", kind=kind, window=window,
                       softcap=softcap, masked=masked)
    got, lse = check_attention(ts, sampler, c)
    if masked is not None:
        assert not got[len(EDGES) // 2].any() and np.isneginf(lse[len(EDGES) // 2]).all()


@pytest.mark.parametrize("kind,group", [("bf16", 4), ("e4m3", 8), ("f32", 2), ("f32", 11)])
@pytest.mark.parametrize("join", [1, 2])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40, 0])
def test_attention_cuts(ts, sampler, kind, group, ctas, join):
    """The same answers however the tiles are dealt to the CTAs."""
    import torch
    c = attention_case(torch, 11, [1000, 3, 0, 700, 64, 1, 2000], heads=2, group=group, dim=128, block=16, layout="hnd",
                       kind=kind)
    sampler.set_option(ts.TS_OPT_KV_CTAS, ctas)
    sampler.set_option(ts.TS_OPT_KV_JOIN, join)
    try:
        one = check_attention(ts, sampler, c)
        two = run_attention(ts, sampler, c)
    finally:
        sampler.set_option(ts.TS_OPT_KV_JOIN, 0)
        sampler.set_option(ts.TS_OPT_KV_CTAS, 0)
    assert np.array_equal(one[0], two[0]) and np.array_equal(one[1], two[1])  # the same in every run


def test_attention_sums_past_32_bits(ts, sampler):
    """Table rows that could hold more than 2^31 tiles of work together, and a
    context that crosses one of its 65,536-token blocks."""
    import torch
    c = attention_case(torch, 20, [100, 0, 65540], heads=32, group=1, dim=16, block=65536, layout="nhd", kind="bf16",
                       stale=False)
    wide = np.random.default_rng(0).integers(-2**31, 2**31, (3, 32000)).astype(np.int32)
    wide[:, :2] = c["table"][:, :2]
    c["table"] = wide
    check_attention(ts, sampler, c)


def test_attention_nothing_to_do(ts, sampler):
    """No requests, and requests whose tables have no entries."""
    import torch
    c = attention_case(torch, 21, [0, 0], heads=1, group=2, dim=64, block=16, layout="nhd", kind="bf16", stale=False)
    c["table"] = c["table"][:, :0]
    got, lse, status = run_attention(ts, sampler, c)
    assert not got.any() and np.isneginf(lse).all() and status == 0
    c["lens"] = np.array([0, 1], np.int32)  # longer than its table
    got, lse, status = run_attention(ts, sampler, c)
    assert not got[0].any() and np.isnan(got[1]).all() and np.isnan(lse[1]).all() and status == okv.BAD_SHAPE
    q = c["q"][:0]
    query = ts.PagedQuery(q, torch.empty_like(q), torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                          torch.zeros(0, dtype=torch.int32, device="cuda"))
    ts.ts_paged_attention(sampler.handle, ts.KvCache(c["k"], c["v"]), query)


def test_attention_many_requests(ts, sampler):
    """More requests than a CTA has threads, most of them empty."""
    import torch
    lens = np.zeros(1000, np.int32)
    lens[[0, 127, 128, 129, 500, 999]] = [5, 300, 1, 64, 90, 33]
    c = attention_case(torch, 12, lens, heads=2, group=2, dim=64, block=16, layout="nhd", kind="bf16")
    check_attention(ts, sampler, c)
    c["lens"] = np.zeros(1000, np.int32)
    got, lse, status = run_attention(ts, sampler, c)
    assert not got.any() and np.isneginf(lse).all() and status == 0


@pytest.mark.parametrize("join", [0, 2])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_attention_long(ts, sampler, kind, join):
    """One long context, peaked scores (the running maximum moves late)."""
    import torch
    c = attention_case(torch, 13, [20011], heads=1, group=8, dim=128, block=32, layout="hnd", kind=kind, spread=6.0)
    c["k"].view(torch.uint8)[0] = c["k"].view(torch.uint8)[1]
    sampler.set_option(ts.TS_OPT_KV_JOIN, join)
    try:
        check_attention(ts, sampler, c)
    finally:
        sampler.set_option(ts.TS_OPT_KV_JOIN, 0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attention_values(ts, sampler, kind):
    """Attended infinities and NaN come out as the arithmetic has them; scores
    of -inf weigh nothing, and a head with no others attends to nothing."""
    import torch
    c = attention_case(torch, 14, [40, 40, 40, 40], heads=1, group=2, dim=64, block=16, layout="nhd", kind=kind, stale=False)
    q, t = c["q"], c["table"]
    q[1:3] = q[1:3].abs() + 0.1
    c["k"][t[0, 1], 3] = float("nan")
    c["k"][t[1, 0], 2] = float("-inf")        # one score of -inf
    for b in range(3):
        c["k"][t[2, b]] = float("-inf")       # all of them
    c["v"][t[3, 0], 5, 0, 7] = float("inf")
    got, lse, status = run_attention(ts, sampler, c)
    want = want_attention(torch, c)
    assert status == 0
    assert np.isnan(got[0]).all() and np.isnan(lse[0]).all()
    assert np.allclose(got[1], want["out"][1], rtol=2 ** -7, atol=1e-2) and np.isfinite(lse[1]).all()
    assert not got[2].any() and np.isneginf(lse[2]).all()
    assert np.isposinf(got[3, :, 7]).all() and np.isfinite(np.delete(got[3], 7, 1)).all()


@pytest.mark.parametrize("gap", [12.0, 16.0, 18.0, 20.0, 24.0])
@pytest.mark.parametrize("n,group,dim,ctas", [(1500, 2, 64, 0), (1500, 16, 128, 1), (16000, 8, 128, 1), (16000, 1, 256, 0),
                                              (16000, 3, 192, 40)])
def test_attention_small_weights_on_e4m3(ts, sampler, gap, n, group, dim, ctas):
    """One key far above all others in score, with a value of zeros: what comes
    out is the others', whose weights are 2^-17 to 2^-35 of the largest.  Bounds
    as in assert_attention, but a weight in f16 counts from 2^15, so what it
    loses at least is 2^-40 of the largest weight."""
    import torch
    c = attention_case(torch, 22, [n, 300], heads=1, group=group, dim=dim, block=16, layout="nhd", kind="e4m3", stale=False)
    c.update(k_scale=None, v_scale=None, scale=1.0)
    c["q"][:] = 0
    c["q"][:, :, 0] = 1
    c["k"].view(torch.uint8)[:] = 0
    c["v"].copy_(c["v"].float().abs().to(c["v"].dtype))
    for r, t in ((0, n // 3), (1, 299)):
        at = int(c["table"][r, t // 16]), t % 16
        c["k"].view(torch.uint8)[at[0], at[1], 0, 0] = int(okv.to_e4m3([gap])[0])
        c["v"].view(torch.uint8)[at] = 0
    want = want_attention(torch, c)
    assert np.allclose(want["lse"][0], np.logaddexp(gap, np.log(n - 1)), rtol=1e-12)
    sampler.set_option(ts.TS_OPT_KV_CTAS, ctas)
    try:
        got, lse, status = run_attention(ts, sampler, c)
    finally:
        sampler.set_option(ts.TS_OPT_KV_CTAS, 0)
    assert status == 0
    keys = want["keys"][:, None]
    err = dim * 2.0 ** -22 * want["dot"] + 2.0 ** -21 * (np.abs(want["lse"]) + want["dot"])
    bound = want["abs_v"] * (4 * err + keys * 2.0 ** -23 + 2.0 ** -10)[..., None] + 2.0 ** -8 * want["out"]
    bound = bound + (keys * 2.0 ** -40 * want["max_v"])[..., None]
    assert np.all(np.abs(got - want["out"]) <= bound), np.max((np.abs(got - want["out"]) / want["out"]))
    assert np.all(np.abs(lse - want["lse"]) <= 2 * err + keys * 2.0 ** -23 + 2.0 ** -20)


def test_attention_large_queries_on_e4m3(ts, sampler):
    """Query rows far outside f16's range, and one of zeros."""
    import torch
    c = attention_case(torch, 15, [100, 37, 64], heads=1, group=8, dim=64, block=16, layout="nhd", kind="e4m3")
    powers = torch.tensor([2.0 ** e for e in (60, -60, 20, -20, 3, 0, 100, -100)], device="cuda").bfloat16()
    c["q"] *= powers[None, :, None]
    c["q"][0, 3] = 0
    c["k_scale"] = c["k_scale"] * 0 + 2.0 ** -6
    c["scale"] = 2.0 ** -3
    want = want_attention(torch, c)
    got, lse, _ = run_attention(ts, sampler, c)
    calm = [1, 3, 4, 5, 7]  # the others pick one key, within rounding of the scores
    part = {k: (v if k in ("keys", "status") else v[:, calm]) for k, v in want.items()}
    assert_attention(c, part, got[:, calm], lse[:, calm])
    assert np.isfinite(got).all()


def test_attention_strided_queries(ts, sampler):
    """Queries and outputs inside wider rows, an output of other strides, no lse."""
    import torch
    c = attention_case(torch, 16, EDGES, heads=2, group=3, dim=64, block=16, layout="nhd", kind="bf16", q_pad=40)
    want = want_attention(torch, c)
    n = len(EDGES)
    out = torch.full((6, n + 2, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, 1:n + 1, :64].permute(1, 0, 2)
    query = ts.PagedQuery(c["q"], view, torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda())
    ts.ts_paged_attention(sampler.handle, ts.KvCache(c["k"], c["v"]), query)
    torch.cuda.synchronize()
    assert_attention(c, want, view.float().cpu().numpy(), want["lse"].astype(np.float32))
    out[:, 1:n + 1, :64] = 3.0
    assert bool((out == 3.0).all())  # nothing outside was written


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attention_offsets_past_32_bits(ts, sampler, kind):
    """Blocks whose byte and element offsets pass 2^31 and 2^32."""
    import torch
    c = attention_case(torch, 17, [33, 70], heads=1, group=2, dim=64, block=16, layout="nhd", kind=kind, stale=False)
    used = c["n_blocks"]
    apart = (1 << 32) // (used - 1) // 64 * 64 + 64  # elements between blocks
    far = []
    for x in (c["k"], c["v"]):
        y = torch.empty(apart * (used - 1) + 16 * 64, dtype=x.dtype, device="cuda")
        view = y.as_strided((used, 16, 1, 64), (apart, 64, 64, 1))
        view.copy_(x)
        far.append(view)
    want = want_attention(torch, c)
    c["k"], c["v"] = far
    got, lse, status = run_attention(ts, sampler, c)
    assert status == 0
    assert_attention(c, want, got, lse)
    k2 = torch.randn((4, 1, 64), device="cuda").to(far[0].dtype)
    slots = torch.tensor([(used - 1) * 16 + 3, 0, 17, (used - 2) * 16], device="cuda")
    ts.ts_kv_append(sampler.handle, ts.KvCache(*far), ts.KvTokens(k2, -k2, slots))
    torch.cuda.synchronize()
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(far[0][s // 16, s % 16], k2[i]) and torch.equal(far[1][s // 16, s % 16], -k2[i])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("block", [16, 10])
def test_attention_errors(ts, sampler, kind, block):
    """Lengths and blocks out of range: NaN there, the others untouched."""
    import torch
    c = attention_case(torch, 18, [40, 50, 60, 70, 80], heads=2, group=2, dim=64, block=block, layout="nhd", kind=kind)
    wide = c["table"].shape[1]
    c["lens"][1] = -1
    c["lens"][2] = wide * block + 1
    c["table"][3, 2] = c["n_blocks"]
    c["table"][4, -1] = -1  # past its length: not looked at
    want = want_attention(torch, c)
    assert want["status"] == okv.BAD_SHAPE | okv.BAD_BLOCK
    check_attention(ts, sampler, c)
    sampler.set_option(ts.TS_OPT_KV_CTAS, 1)
    try:
        check_attention(ts, sampler, c)
    finally:
        sampler.set_option(ts.TS_OPT_KV_CTAS, 0)


def test_attention_refusals(ts, sampler):
    import torch
    c = attention_case(torch, 19, [40, 50], heads=2, group=2, dim=64, block=16, layout="nhd", kind="bf16")
    out = torch.full_like(c["q"], 7.0)
    mask = torch.ones((2, c["table"].shape[1] * 16), dtype=torch.uint8, device="cuda")

    def go(field=None, value=None, cfield=None, cvalue=None, handle=None):
        query = ts.PagedQuery(c["q"], out, torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda(),
                              key_mask=mask)
        cache = ts.KvCache(c["k"], c["v"])
        if field:
            setattr(query.c, field, value)
        if cfield:
            setattr(cache.c, cfield, cvalue)
        with pytest.raises(ts.SamplerError) as e:
            ts.ts_paged_attention(handle or sampler.handle, cache, query)
        return e.value.status
    inv, uns = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    for field in ("q", "out", "lens", "block_table"):
        assert go(field, None) == inv, field
    assert go("n_heads", 3) == inv and go("n_heads", 0) == inv and go("n_requests", -1) == inv
    assert go("window", -1) == inv and go("softcap", -1.0) == inv and go("scale", float("nan")) == inv
    assert go("mask_stride", 15) == inv and go("table_stride", 1) == inv
    assert go("q", c["q"].data_ptr() + 2) == inv and go("q_head_stride", 63) == inv
    assert go("out_request_stride", -64) == inv and go("dtype", 2) == inv and go("dtype", 0) == uns
    assert go("max_blocks", 1 << 28) == inv  # the stride is below it
    assert go("n_heads", 1 << 17) == uns
    assert go(cfield="dtype", cvalue=0) == uns and go(cfield="block_size", cvalue=0) == inv
    assert go(cfield="head_dim", cvalue=264) == uns and go(cfield="v", cvalue=None) == inv
    fresh = ts.Sampler(0)
    assert go(handle=fresh.handle) == inv  # no workspace
    fresh.close()
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and sampler.read_status() == 0


def test_attention_on_another_stream_and_in_a_graph(ts, sampler):
    """Tables, append and attention of three steps captured once and replayed;
    the same as the calls on a stream of their own."""
    import torch
    n, heads, group, dim, block, wide = 5, 2, 2, 64, 16, 4
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((12, n, heads * (group + 2), dim), device="cuda", generator=gen).bfloat16()

    def program(stream_of):
        k, v = (torch.zeros((n * wide, block, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        t = ts.KvTables(n, wide, n * wide, block, max_tokens=n)
        x = torch.zeros_like(rows[0])
        out = torch.zeros((n, heads * group, dim), dtype=torch.bfloat16, device="cuda")
        cache = ts.KvCache(k, v)
        tok = ts.KvTokens(x[:, heads * group:heads * (group + 1)], x[:, heads * (group + 1):], t.slots)
        query = ts.PagedQuery(x[:, :heads * group], out, t.block_table, t.lens)

        def step(stream=None):
            ts.ts_kv_tables(sampler.handle, t, stream)
            ts.ts_kv_append(sampler.handle, cache, tok, stream)
            ts.ts_paged_attention(sampler.handle, cache, query, stream)
        got = []
        if stream_of == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        else:
            side = torch.cuda.Stream()
        for i in range(rows.shape[0]):
            x.copy_(rows[i])
            if stream_of == "graph":
                g.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                step(side)
                torch.cuda.current_stream().wait_stream(side)
            got.append(out.clone())
        torch.cuda.synchronize()
        assert t.lens.tolist() == [rows.shape[0]] * n
        return got
    for a, b in zip(program("graph"), program("side")):
        assert torch.equal(a, b)
    # the last step against the definition: all keys so far
    x = rows.double()
    q = x[-1, :, :heads * group].view(n, heads, group, dim)
    k, v = x[:, :, heads * group:heads * (group + 1)], x[:, :, heads * (group + 1):]
    p = torch.softmax(torch.einsum("nhgd,tnhd->nhgt", q, k) * dim ** -0.5, -1)
    want = torch.einsum("nhgt,tnhd->nhgd", p, v).reshape(n, heads * group, dim)
    assert float((a.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 2.0 ** -12


def test_options_and_reserve(ts):
    s = ts.Sampler(0)
    with pytest.raises(ts.SamplerError):
        s.set_option(ts.TS_OPT_KV_CTAS, -1)
    with pytest.raises(ts.SamplerError):
        s.reserve_kv(-1)
    s.reserve_kv(4)
    s.reserve_kv(2)
    s.reserve_kv(100)
    s.reserve_kv(0)
    s.close()


def test_a_larger_reserve_keeps_captured_graphs(ts):
    """Tables updated in place by several blocks and a joined attention, captured
    with room for four requests: the same results when they are replayed after the
    workspace has been asked for more."""
    import torch
    s = ts.Sampler(0)
    s.reserve_kv(4)
    c = attention_case(torch, 31, [3000, 2000, 5, 900], heads=2, group=4, dim=64, block=16, layout="nhd", kind="bf16", stale=False)
    want = want_attention(torch, c)
    out, lse = torch.zeros_like(c["q"]), torch.zeros(c["q"].shape[:2], device="cuda")
    cache = ts.KvCache(c["k"], c["v"])
    query = ts.PagedQuery(c["q"], out, torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda(),
                          scale=c["scale"], lse=lse)
    n_new = torch.tensor([3000, 1, 0, 2500], dtype=torch.int32, device="cuda")
    t = ts.KvTables(4, 600, 2400, 16, max_tokens=9000, n_new=n_new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.ts_kv_tables(s.handle, t)
        ts.ts_paged_attention(s.handle, cache, query)
    s.reserve_kv(8192)
    s.reserve_kv(3)
    for i in range(1, 4):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert t.lens.tolist() == [3000 * i, i, 0, 2500 * i]
        assert int(t.n_free) == 2400 - sum(-(-x // 16) for x in t.lens.tolist())
        assert_attention(c, want, out.float().cpu().numpy(), lse.cpu().numpy())
    assert s.read_status() == 0
    many = ts.KvTables(8192, 1, 8192, 16, max_tokens=8192)  # the larger number is served
    ts.ts_kv_tables(s.handle, many)
    torch.cuda.synchronize()
    assert bool((many.lens == 1).all()) and sorted(many.block_table[:, 0].tolist()) == list(range(8192))
    s.close()


def test_reserved_requests_bound_the_tables(ts):
    """Tables of more requests than were asked for are refused, as before."""
    s = ts.Sampler(0)
    s.reserve_kv(4)
    with pytest.raises(ts.SamplerError) as e:
        ts.ts_kv_tables(s.handle, ts.KvTables(5, 2, 10, 16, max_tokens=5))
    assert e.value.status == ts.TS_ERR_INVALID_ARG
    s.reserve_kv(5)
    ts.ts_kv_tables(s.handle, ts.KvTables(5, 2, 10, 16, max_tokens=5))
    assert s.read_status() == 0
    s.close()


@pytest.mark.parametrize("kind,group", [("bf16", 4), ("e4m3", 16), ("f32", 2)])
def test_attention_after_a_call_that_lost_parts(ts, sampler, kind, group):
    """Counters left behind by a call that lost parts do not reach the next ones,
    whatever number of CTAs these and the calls between have."""
    import torch
    c = attention_case(torch, 41, [1000, 3, 0, 700, 64, 1, 2000], heads=2, group=group, dim=128, block=16, layout="hnd",
                       kind=kind)
    other = attention_case(torch, 42, [900, 350], heads=1, group=1, dim=256, block=16, layout="nhd", kind="f32")
    want = want_attention(torch, c)
    sampler.set_option(ts.TS_OPT_KV_JOIN, 2)
    try:
        for ctas in (7, 40, 3, 0, 41):
            sampler.set_option(ts.TS_OPT_KV_CTAS, ctas)
            first = run_attention(ts, sampler, c)
            for lost in (1, 2, 5, 1000, 0):
                ts.ts_kv_debug_lose_parts(sampler.handle, lost)
                got = run_attention(ts, sampler, c)
                assert got[2] == 0
                assert_attention(c, want, got[0], got[1])
                again = run_attention(ts, sampler, c)
                for x, y, z in zip(first, got, again):
                    assert np.array_equal(x, y) and np.array_equal(x, z)
                check_attention(ts, sampler, other)
    finally:
        sampler.set_option(ts.TS_OPT_KV_JOIN, 0)
        sampler.set_option(ts.TS_OPT_KV_CTAS, 0)
    fresh = ts.Sampler(0)
    with pytest.raises(ts.SamplerError):
        ts.ts_kv_debug_lose_parts(fresh.handle, 1)  # no workspace
    fresh.close()
    with pytest.raises(ts.SamplerError):
        ts.ts_kv_debug_lose_parts(sampler.handle, 1001)
