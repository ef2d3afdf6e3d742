"""Calls of the layer operators that the header allows: where outputs may lie, and calls at
once."""
import numpy as np
import pytest

from oracle import layer as olayer
from test_gpu_layer import check_rows, close, get, HALF, norm_error, put, run_norm, sampler, TINY, ts  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# Rotary outputs beside what they come from
# --------------------------------------------------------------------------
def rotary_inputs(seed, tokens, heads, dim):
    import torch
    rng = np.random.default_rng(seed)
    return (put(rng.normal(0, 3, (tokens, heads, dim)), "bf16"), torch.from_numpy(rng.integers(0, 5000, tokens).astype(np.int32)).cuda(),
            torch.from_numpy(10000.0 ** (-np.arange(0, dim, 2) / dim)).cuda())


@pytest.mark.parametrize("layout", ["columns of a product", "every other head", "heads before rows", "heads before rows, in place", "one row of any stride",
                                    "one head of any stride"])
def test_rotary_outputs_beside_their_inputs(ts, sampler, layout):
    """Outputs in the inputs' buffer that share nothing with them: the bits of a call with
    buffers of its own, and what is around them stays."""
    import torch
    tokens, heads = (1 if layout.startswith("one row") else 37), (1 if layout.startswith("one head") else 6)
    x, pos, f = rotary_inputs(1, tokens, heads, 64)
    want = torch.empty_like(x)
    ts.ts_rotary(sampler.handle, ts.Rotary(x, want, pos, f))
    if layout == "columns of a product":
        buf = torch.full((tokens, 3 * heads + 1, 64), 7.0, device="cuda").bfloat16()
        a, b = buf[:, :heads], buf[:, heads + 1:2 * heads + 1]
    elif layout == "every other head":
        buf = torch.full((tokens, 2 * heads, 64), 7.0, device="cuda").bfloat16()
        a, b = buf[:, ::2], buf[:, 1::2]
    elif layout.startswith("heads before rows"):
        buf = torch.full((2 * heads, tokens, 64), 7.0, device="cuda").bfloat16()
        a, b = buf[:heads].transpose(0, 1), buf[heads:].transpose(0, 1)
        b = a if layout.endswith("in place") else b
    else:
        strides = ((16, 64, 1), (0, 64, 1)) if tokens == 1 else ((64, 16, 1), (64, 0, 1))
        buf = torch.full((2 * x.numel() + 64,), 7.0, device="cuda").bfloat16()
        a, b = (torch.as_strided(buf, x.shape, s, at) for s, at in zip(strides, (0, x.numel())))
    a.copy_(x)
    ts.ts_rotary(sampler.handle, ts.Rotary(a, b, pos, f))
    assert torch.equal(b, want)
    if b is not a:
        assert torch.equal(a, x) and int((buf == 7).sum()) >= buf.numel() - 2 * x.numel()


@pytest.mark.parametrize("layout", ["queries, keys, values", "a head's query, key and value", "outputs over queries"])
def test_append_rotary_within_one_product(ts, sampler, layout):
    """Queries, keys and values side by side in one product's rows, turned where they stand."""
    import torch
    tokens, heads, dim = 37, 4, 64
    rows, pos, f = rotary_inputs(2, tokens, 3 * heads, dim)
    if layout == "a head's query, key and value":
        parts = [rows.view(tokens, heads, 3, dim)[:, :, i] for i in range(3)]
    else:
        parts = [rows[:, i * heads:(i + 1) * heads] for i in range(3)]
    slots = torch.arange(tokens, device="cuda")
    kept = rows.clone()
    results = []
    for own in (True, False):
        k, v = (torch.zeros((3, 16, heads, dim), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        q, k_new, v_new = [p.contiguous() if own else p for p in parts]
        out = torch.empty_like(q) if own else q
        ts.ts_kv_append_rotary(sampler.handle, ts.KvCache(k, v), ts.KvTokens(k_new, v_new, slots), ts.Rotary(q, out, pos, f))
        results.append((out.clone(), k, v))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    parts[0].copy_(kept.view(tokens, heads, 3, dim)[:, :, 0] if layout.startswith("a head's") else kept[:, :heads])
    assert torch.equal(rows, kept)


# --------------------------------------------------------------------------
# Calls at once
# --------------------------------------------------------------------------
def test_two_graphs_of_finite_products(ts, sampler):
    """Two captured norms and products of one sampler, replayed on two streams, with weights
    that are all numbers: the bits of plain calls."""
    import torch
    rng = np.random.default_rng(6)
    runs = []
    for i in range(2):
        x = put(rng.normal(0, 1, (64 + 100 * i, 1024)), "bf16")
        e, s = put(np.zeros(x.shape), "e4m3"), put(np.zeros((x.shape[0], 8)))
        w, ws = put(np.clip(rng.normal(0, 100, (640, 1024)), -448, 448), "e4m3"), put(rng.uniform(0.5, 1, (5, 8)))
        out = put(np.zeros((x.shape[0], 640)))
        calls = [(ts.ts_rms_norm, ts.RmsNorm(x, e, out_scale=s)), (ts.ts_linear_e4m3, ts.LinearE4m3(e, s, w, ws, out))]
        for fn, c in calls:
            fn(sampler.handle, c)
        torch.cuda.synchronize()
        want = out.clone()
        assert bool(torch.isfinite(want).all()) and bool((want != 0).any())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for fn, c in calls:
                fn(sampler.handle, c)
        runs.append((graph, out, want, calls))
    for _, out, _, _ in runs:
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (graph, *_), st in zip(runs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in runs:
        assert torch.equal(out, want)


# --------------------------------------------------------------------------
# A copy that does not come
# --------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,k,path,split", [(3, 300, 1100, 1, 1), (30, 300, 1100, 1, 2), (60, 260, 2048, 1, 4), (64, 400, 300, 1, 1),
                                              (100, 300, 1100, 2, 1), (200, 260, 1500, 2, 2), (300, 700, 130, 2, 1)])
def test_a_lost_copy_ends_the_waits(ts, sampler, m, n, k, path, split):
    """The copies of one block never come to the first tile: the kernel's waits run out, the
    status says so, that tile's outputs stay as they were, the other tiles' are right, and so
    is the next call."""
    import torch
    rng = np.random.default_rng([m, n, k])
    blocks, wide = -(-k // 128), -(-k // 16) * 16
    x, w = (put(rng.integers(-8, 9, (r, wide)), "e4m3")[:, :k] for r in (m, n))
    xs, ws = put(rng.uniform(0.5, 1, (m, blocks))), put(rng.uniform(0.5, 1, (-(-n // 128), blocks)))
    out = torch.empty((m, n), device="cuda")
    call = ts.LinearE4m3(x, xs, w, ws, out)
    sampler.read_status()
    try:
        sampler.set_option(ts.TS_OPT_LINEAR_PATH, path)
        sampler.set_option(ts.TS_OPT_LINEAR_SPLIT, split)
        ts.ts_linear_e4m3(sampler.handle, call)
        want = out.clone()
        assert sampler.read_status() == 0 and not bool((want == 7).any())
        for block in sorted({0, blocks // 2, blocks - 1}):
            sampler.set_option(ts.TS_OPT_LINEAR_LOSE, block + 1)
            out.fill_(7)
            ts.ts_linear_e4m3(sampler.handle, call)
            assert sampler.read_status() == ts.TS_ROW_STALLED, block
            kept = out == 7
            assert bool(kept[:min(m, 16), :32].all()) and bool((kept | (out == want)).all())
            assert bool((~kept[:, -1:]).all())  # of the last tile's columns
            sampler.set_option(ts.TS_OPT_LINEAR_LOSE, 0)
            ts.ts_linear_e4m3(sampler.handle, call)
            assert sampler.read_status() == 0 and torch.equal(out, want)
        sampler.set_option(ts.TS_OPT_LINEAR_PATH, 3)
        sampler.set_option(ts.TS_OPT_LINEAR_LOSE, 1)
        with pytest.raises(ts.SamplerError) as e:  # pairs wait for one another
            ts.ts_linear_e4m3(sampler.handle, call)
        assert e.value.status == ts.TS_ERR_UNSUPPORTED
    finally:
        for option in (ts.TS_OPT_LINEAR_LOSE, ts.TS_OPT_LINEAR_PATH, ts.TS_OPT_LINEAR_SPLIT):
            sampler.set_option(option, 0)


def test_handles_made_at_once(ts):
    """Handles made by several threads, each of which multiplies: the same bits from all."""
    import threading
    import torch
    rng = np.random.default_rng(3)
    x, w = (put(rng.integers(-8, 9, (r, 256)), "e4m3") for r in (70, 300))
    xs, ws = put(rng.uniform(0.5, 1, (70, 2))), put(rng.uniform(0.5, 1, (3, 2)))
    outs, made, failed = [torch.zeros((70, 300), device="cuda") for _ in range(8)], [], []
    torch.cuda.synchronize()

    def work(out):
        try:
            torch.cuda.set_device(0)
            handle = ts.Sampler(0)
            made.append(handle)
            stream = torch.cuda.Stream()
            ts.ts_linear_e4m3(handle.handle, ts.LinearE4m3(x, xs, w, ws, out), stream)
            stream.synchronize()
        except Exception as e:  # the thread's own
            failed.append(e)
    threads = [threading.Thread(target=work, args=(out,)) for out in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for handle in made:
        handle.close()
    assert not failed and bool((outs[0] != 0).any()) and all(torch.equal(out, outs[0]) for out in outs)


# --------------------------------------------------------------------------
# Norms at the borders of their variants
# --------------------------------------------------------------------------
@pytest.mark.parametrize("rows,dim", [(609, 2064), (700, 3584), (640, 4080), (611, 4096), (608, 4096), (609, 4112), (700, 512), (700, 504)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm_with_residual_to_8_bits_at_the_borders(ts, sampler, rows, dim, kind):
    """Wide rows with a residual on both sides of 608 rows (four to an SM), of 512 and of
    4096 elements."""
    rng = np.random.default_rng([rows, dim])
    x, w, r = rng.normal(0, 3, (rows, dim)), rng.normal(1, 0.3, dim), rng.normal(0, 5, (rows, dim))
    got = run_norm(ts, sampler, x, w, r, kind, "e4m3", eps=1e-5)
    h, y = olayer.rms_norm(got["x"], got["weight"], got["residual"], eps=1e-5)
    check_rows(got["out"], got["scale"], y, norm_error(dim), 0.0, "e4m3")
    close(get(got["sum"]), h, (2.0 ** -24 + HALF[kind]) * np.abs(h) + TINY[kind], "sum")


def test_norm_of_many_elements_in_rows_of_4096(ts, sampler):
    """2^26 elements and more take another variant than fewer: a large call and its halves
    are within their roundings of the 64-bit norm, sums bit for bit the same.  (Without a
    weight a code is 448 h over the block's largest h, numbers of few bits whose quotient is
    often a tie: the variants' codes differ there, by the last bit of their scales.)"""
    import torch
    x, r = (torch.randn((16384, 4096), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    total = torch.empty_like(x)
    h = x.double() + r.double()
    y = (h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)).view(16384, 32, 128)
    del h

    def call(part, sums):
        o, s = torch.empty(x[part].shape, device="cuda", dtype=torch.float8_e4m3fn), torch.empty((x[part].shape[0], 32), device="cuda")
        ts.ts_rms_norm(sampler.handle, ts.RmsNorm(x[part], o, residual=r[part], residual_out=sums, out_scale=s))
        off = norm_error(4096) * y[part].abs()
        blocks = y[part].abs().amax(-1) / 448
        assert bool(((s - blocks).abs() <= (norm_error(4096) + 2.0 ** -23) * blocks).all())
        step = HALF["e4m3"] * (y[part].abs() + off) + TINY["e4m3"] * s[..., None]
        assert bool(((o.double().view(-1, 32, 128) * s[..., None] - y[part]).abs() <= off + step * (1 + 2.0 ** -20)).all())
    call(slice(0, 16384), total)
    for part in (slice(0, 8192), slice(8192, 16384)):
        sums = torch.empty_like(x[part])
        call(part, sums)
        assert torch.equal(sums, total[part])
