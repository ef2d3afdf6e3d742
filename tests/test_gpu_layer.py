"""The layer operators around the paged cache against their plain 64-bit versions: the
norm, the gated activation, the 8-bit product, rotary positions, and a run of them."""
import numpy as np
import pytest

from oracle import kv as okv
from oracle import layer as olayer

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}  # half a step, of the value
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "e4m3": 2.0 ** -10}  # half the smallest step or more


@pytest.fixture(scope="module")
def ts():
    import codebook_token_sampling_gb300 as mod
    return mod


@pytest.fixture(scope="module")
def sampler(ts):
    s = ts.Sampler(0)
    s.reserve_kv(64)
    yield s
    s.close()


def kind_of(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def put(x, kind="f32"):
    """A numpy array as a device tensor of a type (rounded)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(kind_of(kind))


def get(t):
    """A device tensor as 64-bit values; 8-bit ones as the codes' values."""
    import torch
    if t.dtype == torch.float8_e4m3fn:
        return okv.from_e4m3(t.contiguous().view(torch.uint8).cpu().numpy())
    return t.double().cpu().numpy()


def codes(t):
    import torch
    return t.contiguous().view(torch.uint8).cpu().numpy()


def strided(rows, dim, kind, pad, fill=0):
    """Rows of a wider buffer, and the buffer (rows start at `pad` elements, or with pad 0
    at the buffer's start and without gaps)."""
    import torch
    buf = torch.full((rows, dim + 2 * pad), fill, dtype=torch.float32, device="cuda").to(kind_of(kind))
    return buf[:, pad:pad + dim], buf


def close(got, want, bound, what=""):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], np.broadcast_to(bound, got.shape)[bad][:3])


def check_rows(out, scale, want, rel, absolute, kind):
    """Rows of `kind` for the values `want`, which may be off by rel of them and by
    `absolute` before they are rounded.  8-bit ones: their scales, and the codes' values."""
    off = rel * np.abs(want) + absolute
    if kind != "e4m3":
        close(get(out), want, off + HALF[kind] * (np.abs(want) + off) + TINY[kind], "out")
        return
    blocks = olayer.block_scales(want)
    room = np.full((want.shape[0], blocks.shape[1] * 128), 0.0)
    room[:, :want.shape[1]] = off
    # the scale's own rounding, and what its block's largest may be off by
    s_off = room.reshape(want.shape[0], -1, 128).max(2) / 448 + 2.0 ** -23 * blocks
    close(get(scale), blocks, s_off, "scale")
    s = olayer.of_columns(get(scale), want.shape[1])
    # half a step of the code at the value's size, or the smallest step; two roundings of the quotient
    close(get(out) * s, want, off + HALF["e4m3"] * (np.abs(want) + off) * (1 + 2.0 ** -20) + TINY["e4m3"] * s * (1 + 2.0 ** -20), "out")


# --------------------------------------------------------------------------
# Norm
# --------------------------------------------------------------------------
def run_norm(ts, sampler, x, weight, residual, kind, out_kind, *, w_kind="f32", pad=0, in_place=False, **kw):
    rows, dim = x.shape
    tx, bx = strided(rows, dim, kind, pad)
    tx.copy_(put(x, kind))
    tr = br = None
    if residual is not None:
        tr, br = strided(rows, dim, kind, pad)
        tr.copy_(put(residual, kind))
    out, bo = strided(rows, dim, out_kind, pad, fill=7)
    sums, bs = (None, None) if residual is None else (tr, br) if in_place else strided(rows, dim, kind, pad, fill=7)
    scale = strided(rows, -(-dim // 128), "f32", pad, fill=7)[0] if out_kind == "e4m3" else None
    w = None if weight is None else put(weight, w_kind)
    call = ts.RmsNorm(tx, out, w, residual=tr, residual_out=sums, out_scale=scale, **kw)
    before = [get(t) if t is not None else None for t in (tx, tr)]
    ts.ts_rms_norm(sampler.handle, call)
    for buf in (bo, bs):
        if buf is not None and pad and not in_place:
            assert bool((buf[:, :pad].float() == 7).all()) and bool((buf[:, pad + dim:].float() == 7).all())
    return {"x": before[0], "residual": before[1], "out": out, "scale": scale, "sum": sums, "weight": None if w is None else get(w)}


def norm_error(dim):
    """Relative error of y before its rounding: squares of sums rounded to 2^-24 (2 of
    those), added in chains of at most 32 and a tree of ten; their mean, plus eps, its
    root (half of all of that) and that root's rounding, the two products; the sum h."""
    return (0.5 * (2 + 32 + 10 + 2) + 1 + 2 + 1 + 1) * 2.0 ** -24


@pytest.mark.parametrize("kind,out_kind,w_kind", [("bf16", "e4m3", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f32", "f32"),
                                                  ("f32", "bf16", "bf16"), ("f32", "e4m3", "f32")])
@pytest.mark.parametrize("rows,dim,pad", [(1, 1, 0), (3, 7, 0), (1, 128, 0), (5, 127, 3), (9, 129, 0), (33, 256, 8), (17, 1000, 16), (2, 1024, 0),
                                          (7, 2049, 1), (4, 4096, 0), (3, 5000, 8), (2, 8200, 0), (2, 11111, 5), (1, 32768, 0), (2, 32767, 0),
                                          (2, 16384, 4), (700, 200, 0), (700, 1025, 0), (650, 1032, 3), (620, 2500, 8), (611, 4100, 1)])
def test_norm(ts, sampler, rows, dim, pad, kind, out_kind, w_kind):
    rng = np.random.default_rng([rows, dim])
    x, w = rng.normal(0, 3, (rows, dim)), rng.normal(1, 0.3, dim)
    res = rng.normal(0, 5, (rows, dim)) if (rows + dim) % 2 else None
    got = run_norm(ts, sampler, x, w, res, kind, out_kind, w_kind=w_kind, pad=pad, eps=1e-5)
    h, y = olayer.rms_norm(got["x"], got["weight"], got["residual"], eps=1e-5)
    check_rows(got["out"], got["scale"], y, norm_error(dim), 0.0, out_kind)
    if res is not None:
        close(get(got["sum"]), h, (2.0 ** -24 + HALF[kind]) * np.abs(h) + TINY[kind], "sum")
    assert sampler.read_status() == 0


def test_norm_in_place(ts, sampler):
    """The residual updated where it stands, the output over x, and a weight that counts
    from one: the same bits as with arrays of their own."""
    import torch
    rng = np.random.default_rng(3)
    x, res, w = put(rng.normal(0, 1, (37, 640)), "bf16"), put(rng.normal(0, 4, (37, 640)), "bf16"), put(rng.normal(0, 0.1, 640))
    out, total = torch.empty_like(x), torch.empty_like(x)
    ts.ts_rms_norm(sampler.handle, ts.RmsNorm(x, out, w, residual=res, residual_out=total, weight_offset=1.0))
    h, y = olayer.rms_norm(get(x), get(w), get(res), eps=1e-6, weight_offset=1.0)
    close(get(out), y, (norm_error(640) + 2.0 ** -24 + HALF["bf16"]) * np.abs(y))
    x2, res2 = x.clone(), res.clone()
    ts.ts_rms_norm(sampler.handle, ts.RmsNorm(x2, x2, w, residual=res2, residual_out=res2, weight_offset=1.0))
    assert torch.equal(x2, out) and torch.equal(res2, total)
    x3, res3 = x.clone(), res.clone()
    ts.ts_rms_norm(sampler.handle, ts.RmsNorm(x3, torch.empty_like(x3), w, residual=res3, residual_out=x3, weight_offset=1.0))
    assert torch.equal(x3, total) and torch.equal(res3, res)


@pytest.mark.parametrize("size", [1e-45, 3e-39, 1e-25, 1e-19, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-38])
@pytest.mark.parametrize("dim", [96, 1024, 3001])
def test_norm_of_extreme_rows(ts, sampler, size, eps, dim):
    """Squares that leave fp32's range: the norm is that of the definition.  (Subnormal
    elements are whole multiples of 2^-149.)"""
    rng = np.random.default_rng(1)
    x = (rng.uniform(0.2, 1.0, (4, dim)) * rng.choice([-1, 1], (4, dim)) * size).astype(np.float32)
    x[0, 0] = size
    got = run_norm(ts, sampler, x, None, None, "f32", "f32", eps=eps)
    eps = float(np.float32(eps))
    _, y = olayer.rms_norm(got["x"], None, None, eps=eps)
    # elements scaled by a power of two into the normal range; eps beside them may round to a subnormal's half step
    close(get(got["out"]), y, 2 * norm_error(dim) * np.abs(y) + TINY["f32"])


def test_norm_rows_that_are_not_finite(ts, sampler):
    """A NaN fills its row, an infinity is a NaN among zeros; rows beside them and rows of
    zeros are what they are alone; 8-bit blocks of them have NaN scales and codes."""
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (6, 384)).astype(np.float32)
    x[1, 5], x[2, 300], x[3], x[4, 0] = np.nan, np.inf, 0.0, -np.inf
    for kind in ("f32", "bf16"):
        got = run_norm(ts, sampler, x, None, None, kind, kind, eps=1e-6)
        _, y = olayer.rms_norm(got["x"], None, None, eps=1e-6)
        out = get(got["out"])
        assert np.array_equal(np.isnan(out), np.isnan(y)) and np.isnan(out[1]).all() and np.isnan(out[2]).sum() == 1
        fine = ~np.isnan(y)
        close(out[fine], y[fine], (norm_error(384) + HALF[kind]) * np.abs(y[fine]))
        got = run_norm(ts, sampler, x, None, None, kind, "e4m3", eps=1e-6)
        scale = get(got["scale"])
        assert np.array_equal(np.isnan(scale), [[0, 0, 0], [1, 1, 1], [0, 0, 1], [0, 0, 0], [1, 0, 0], [0, 0, 0]])
        nan = olayer.of_columns(scale, 384)
        assert np.array_equal((codes(got["out"]) & 0x7F) == 0x7F, np.isnan(nan))
        assert np.all(codes(got["out"])[3] == 0) and np.all(scale[3] == np.float32(2.0 ** -64) / np.float32(448))


# --------------------------------------------------------------------------
# Gate
# --------------------------------------------------------------------------
def gate_error(g, up, act):
    """(relative, absolute) error before the output's rounding.  silu: the exponential's
    argument rounded twice (|g| 2^-23 in all, relative), the exponential, the sum, the
    reciprocal and two products within 2^-22 each; results below 2^-126 / |up| may be lost
    to a reciprocal that is subnormal.  gelu: erf and tanh within 2^-22 of 1, tanh's
    argument to 2^-22 of it (|z| (1 - tanh^2 z) < 1/2)."""
    if act == "none":
        return 0.0, 0.0
    if act == "silu":
        return (np.abs(g) * 2.0 ** -23 + 6 * 2.0 ** -22), np.abs(up) * (np.abs(g) + 1) * 2.0 ** -126
    return 2.0 ** -21, np.abs(g * up) * 2.0 ** -21


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "none"])
@pytest.mark.parametrize("kind,out_kind", [("bf16", "e4m3"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "e4m3"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,dim,pad", [(1, 1, 0), (5, 100, 0), (3, 128, 8), (40, 129, 1), (130, 64, 0), (9, 2816, 0), (2, 5001, 2),
                                          (6, 11008, 16)])
def test_gate(ts, sampler, rows, dim, pad, kind, out_kind, act):
    rng = np.random.default_rng([rows, dim])
    both, _ = strided(rows, 2 * dim, kind, pad)
    both.copy_(put(rng.normal(0, 3, (rows, 2 * dim)), kind))
    g, up = both[:, :dim], both[:, dim:]
    out, bo = strided(rows, dim, out_kind, pad, fill=7)
    scale = strided(rows, -(-dim // 128), "f32", pad, fill=7)[0] if out_kind == "e4m3" else None
    ts.ts_gate(sampler.handle, ts.Gate(up, out, None if act == "none" else g, activation=act, out_scale=scale))
    want = olayer.activation(get(g), act) * get(up)
    check_rows(out, scale, want, *gate_error(get(g), get(up), act), out_kind)
    if pad:
        assert bool((bo[:, :pad].float() == 7).all()) and bool((bo[:, pad + dim:].float() == 7).all())


@pytest.mark.parametrize("rows,dim", [(64, 640), (31, 333)])
def test_quantised_rows_are_exact(ts, sampler, rows, dim):
    """Codes and scales of rows that are only rounded follow from fp32 arithmetic alone:
    equal, over sizes from 1e-30 to 1e38, ties, zeros and blocks that are not finite."""
    rng = np.random.default_rng(rows)
    y = (rng.normal(0, 1, (rows, dim)) * 10.0 ** rng.integers(-30, 38, (rows, 1))).astype(np.float32)
    y[0, :128], y[1, 3], y[2, 200], y[3] = 0.0, np.nan, -np.inf, 1.0625
    y[3, 0] = 448.0  # scale 1: ties
    y[3, 1:17] = np.arange(16) * 0.0625 + 1
    out, scale = put(np.zeros((rows, dim)), "e4m3"), put(np.zeros((rows, -(-dim // 128))))
    ts.ts_gate(sampler.handle, ts.Gate(put(y), out, activation="none", out_scale=scale))
    want, s = olayer.quantised_f32(y)
    assert np.array_equal(get(scale), s.astype(np.float64), equal_nan=True)
    nan = np.isnan(olayer.of_columns(s, dim))
    assert np.array_equal(codes(out)[~nan], want[~nan]) and np.all(codes(out)[nan] & 0x7F == 0x7F)
    b = put(np.where(np.isfinite(y) & (np.abs(y) < 1e38), y, 0), "bf16")  # and over itself, unrounded
    kept = b.clone()
    ts.ts_gate(sampler.handle, ts.Gate(b, b, activation="none"))
    assert bool((b == kept).all())


def test_gate_extremes(ts, sampler):
    """Gates far from zero: nothing overflows that the definition keeps finite."""
    g = np.array([[-1e30, -200.0, -89.0, -88.0, -20.0, -0.0, 0.0, 20.0, 89.0, 200.0, 1e19, 3e38]], np.float32)
    up = np.full_like(g, 0.5)
    for act in ("silu", "gelu", "gelu_tanh"):
        out = put(np.zeros_like(g))
        ts.ts_gate(sampler.handle, ts.Gate(put(up), out, put(g), activation=act))
        want = olayer.activation(g, act) * up
        rel, absolute = gate_error(np.minimum(np.abs(g), 100), up, act)
        close(get(out), want, rel * np.abs(want) + absolute + TINY["f32"], act)


@pytest.mark.parametrize("dim", [16, 21])
@pytest.mark.parametrize("kind,out_kind", [("bf16", "bf16"), ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gate_values_that_are_not_finite(ts, sampler, act, kind, out_kind, dim):
    """NaN and infinite gates and factors come out as the definition has them: NaN where it
    is inf times zero, the infinity where it is the gate itself."""
    inf, nan = np.inf, np.nan
    g = np.array([nan, inf, -inf, 2, 0, 3, -nan, 1] + [0.5] * (dim - 8), np.float32)
    up = np.array([2, 3, 4, nan, inf, -inf, 0, 1] + [-2.0] * (dim - 8), np.float32)
    rows = np.stack([np.roll(np.arange(dim), r) for r in range(dim)])
    gate, factor = put(g[rows], kind), put(up[rows], kind)
    with np.errstate(all="ignore"):
        want = olayer.activation(get(gate), act) * get(factor)
    out = put(np.zeros((dim, dim)), out_kind)
    scale = put(np.zeros((dim, 1))) if out_kind == "e4m3" else None
    ts.ts_gate(sampler.handle, ts.Gate(factor, out, gate, activation=act, out_scale=scale))
    if out_kind == "e4m3":  # one block a row
        assert bool(scale.isnan().all()) and np.all(codes(out) & 0x7F == 0x7F)
        return
    got, there = get(out), np.isfinite(want)
    assert np.array_equal(np.where(there, 0, got), np.where(there, 0, want), equal_nan=True)
    assert np.all(np.abs(got[there] - want[there]) <= 2.0 ** -6 * np.abs(want[there]))


@pytest.mark.parametrize("rows,dim,pad,res", [(700, 512, 0, True), (611, 528, 16, True), (900, 1040, 16, False), (640, 2048, 32, True),
                                              (1300, 4096, 0, False), (620, 4080, 8, False), (1000, 496, 0, True)])
@pytest.mark.parametrize("w_kind", ["bf16", "f32", None])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm_of_many_rows_to_8_bits(ts, sampler, rows, dim, pad, res, kind, w_kind):
    """Where a lane takes sixteen elements, and beside those sizes: rows that are large,
    small, zero and not finite among the others."""
    rng = np.random.default_rng([rows, dim])
    x, w = rng.normal(0, 3, (rows, dim)), rng.normal(1, 0.3, dim)
    x[7] *= 1e30
    x[rows - 2] *= 1e-30
    x[rows // 2] = 0
    x[rows // 3, dim - 1] = np.nan
    r = rng.normal(0, 5, (rows, dim)) * (np.abs(x).max(1, keepdims=True) > 1e-20) if res else None
    got = run_norm(ts, sampler, x, w if w_kind else None, r, kind, "e4m3", w_kind=w_kind or "f32", pad=pad, eps=1e-5, weight_offset=0.25 if w_kind else 0.0)
    weight = got["weight"] + 0.25 if w_kind else None
    h, y = olayer.rms_norm(got["x"], weight, got["residual"], eps=1e-5)
    there = np.arange(rows) != rows // 3
    assert bool(got["scale"][rows // 3].isnan().all())
    check_rows(got["out"][there], got["scale"][there], y[there], norm_error(dim) + 2.0 ** -24, 0.0, "e4m3")
    if res:
        close(get(got["sum"])[there], h[there], (2.0 ** -24 + HALF[kind]) * np.abs(h[there]) + TINY[kind], "sum")


@pytest.mark.parametrize("rows,dim,pad", [(1000, 2512, 16), (5000, 512, 0), (20000, 16, 0), (1500, 1680, 8)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "none"])
def test_gate_of_many_rows_to_8_bits(ts, sampler, rows, dim, pad, act):
    """The same of the gate: whole and broken blocks, halves of one product's rows."""
    rng = np.random.default_rng([rows, dim])
    both, _ = strided(rows, 2 * dim, "bf16", pad)
    values = rng.normal(0, 3, (rows, 2 * dim))
    values[3] *= 1e15
    values[rows - 1, dim + 5] = np.nan
    both.copy_(put(values, "bf16"))
    g, up = both[:, :dim], both[:, dim:]
    out, bo = strided(rows, dim, "e4m3", pad, fill=7)
    scale = strided(rows, -(-dim // 128), "f32", pad, fill=7)[0]
    ts.ts_gate(sampler.handle, ts.Gate(up, out, None if act == "none" else g, activation=act, out_scale=scale))
    assert bool(scale[rows - 1, 0].isnan())
    there = slice(0, rows - 1)
    gate, factor = get(g)[there], get(up)[there]
    want = olayer.activation(gate, act) * factor
    check_rows(out[there], scale[there], want, *gate_error(np.minimum(np.abs(gate), 100) if act == "silu" else gate, factor, act), "e4m3")
    if pad:
        assert bool((bo[:, :pad].float() == 7).all()) and bool((bo[:, pad + dim:].float() == 7).all())


# --------------------------------------------------------------------------
# The 8-bit product
# --------------------------------------------------------------------------
def run_linear(ts, sampler, x, xs, w, ws, out_kind, pad=0, stream=None):
    import torch
    m, k = x.shape
    n = w.shape[0]
    wide = -(-k // 16) * 16 + 32 * pad

    def rows(codes):  # what follows a row is NaN
        buf = torch.full((codes.shape[0], wide), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:, :k] = torch.from_numpy(codes).cuda()
        return buf.view(torch.float8_e4m3fn)[:, :k]
    out, buf = strided(m, n, out_kind, pad, fill=7)
    scales = []
    for s in (xs, ws):
        t = strided(*s.shape, "f32", pad, fill=float("nan"))[0]
        t.copy_(put(s))
        scales.append(t)
    ts.ts_linear_e4m3(sampler.handle, ts.LinearE4m3(rows(x), scales[0], rows(w), scales[1], out), stream)
    assert sampler.read_status() == 0
    if pad:
        assert bool((buf[:, :pad] == 7).all()) and bool((buf[:, pad + n:] == 7).all())
    return get(out)


def linear_case(rng, m, n, k):
    def c(rows):
        return okv.to_e4m3(np.clip(rng.normal(0, 100, (rows, k)), -448, 448))
    blocks = -(-k // 128)
    return c(m), rng.lognormal(-5, 1, (m, blocks)).astype(np.float32), c(n), rng.lognormal(-6, 0.5, (-(-n // 128), blocks)).astype(np.float32)


def linear_bound(size, k, kind, want):
    """A block's 128 exact products in fp32 sums, each within a step (2^-23) of the sizes'
    sum; the scales' product, its product with the sum and the blocks' additions."""
    off = size * (128 * 2.0 ** -23 + (-(-k // 128) + 3) * 2.0 ** -24)
    return off + HALF[kind] * (np.abs(want) + off) + TINY[kind]


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 1024), (2, 129, 130), (7, 100, 16), (16, 256, 384), (17, 640, 2048), (32, 1000, 1000), (33, 127, 4096),
         (64, 511, 512), (65, 1030, 272), (100, 384, 896), (128, 257, 1040), (129, 128, 640), (200, 2001, 144), (256, 1024, 1024), (300, 130, 2050),
         (513, 640, 768), (1025, 300, 1280), (777, 2001, 1040), (2050, 515, 400)]


@pytest.mark.parametrize("out_kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(ts, sampler, m, n, k, out_kind):
    """Every size by the kernel that it gets, and by each of the others."""
    rng = np.random.default_rng([m, n, k])
    x, xs, w, ws = linear_case(rng, m, n, k)
    want, size = olayer.linear(x, xs, w, ws)
    try:
        for path in range(4):
            sampler.set_option(ts.TS_OPT_LINEAR_PATH, path)
            got = run_linear(ts, sampler, x, xs, w, ws, out_kind, pad=(m + n) % 3)
            close(got, want, linear_bound(size, k, out_kind, want), path)
    finally:
        sampler.set_option(ts.TS_OPT_LINEAR_PATH, 0)


@pytest.mark.parametrize("m,n,k", [(1, 300, 1100), (30, 260, 4096), (61, 129, 900), (130, 700, 2048), (700, 650, 1500), (1500, 1100, 640)])
def test_linear_of_whole_numbers(ts, sampler, m, n, k):
    """Whole numbers whose sums stay below 2^24 have no roundings: equal, for every split."""
    rng = np.random.default_rng([m, k])
    x, w = rng.integers(-8, 9, (m, k)), rng.integers(-8, 9, (n, k))
    xs = 2.0 ** rng.integers(0, 2, (m, -(-k // 128)))
    ws = 2.0 ** rng.integers(0, 3, (-(-n // 128), -(-k // 128)))
    cx, cw = okv.to_e4m3(x), okv.to_e4m3(w)
    want, size = olayer.linear(cx, xs, cw, ws)
    assert size.max() < 2 ** 24
    try:
        for path in range(4):
            sampler.set_option(ts.TS_OPT_LINEAR_PATH, path)
            for split in (0, 1, 2, 4, 8):
                sampler.set_option(ts.TS_OPT_LINEAR_SPLIT, split)
                assert np.array_equal(run_linear(ts, sampler, cx, xs, cw, ws, "f32"), want), (path, split)
        sampler.set_option(ts.TS_OPT_LINEAR_SPLIT, 1)
        sampler.set_option(ts.TS_OPT_LINEAR_PATH, 2)
        for share in (1, 2, 4):
            sampler.set_option(ts.TS_OPT_LINEAR_SHARE, share)
            assert np.array_equal(run_linear(ts, sampler, cx, xs, cw, ws, "f32"), want), share
    finally:
        sampler.set_option(ts.TS_OPT_LINEAR_SHARE, 0)
        sampler.set_option(ts.TS_OPT_LINEAR_PATH, 0)
        sampler.set_option(ts.TS_OPT_LINEAR_SPLIT, 0)


def test_linear_keeps_small_sums_beside_large_products(ts, sampler):
    """448 x 448 once, its opposite, and ones between them: the sum of the ones is exact
    only where sums keep 24 bits."""
    k = 128
    x = np.ones((20, k))
    w = np.ones((130, k))
    x[:, 0], w[:, 0] = 448, 448
    x[:, 100], w[:, 100] = 448, -448
    one = np.ones((20, 1)), np.ones((2, 1))
    got = run_linear(ts, sampler, okv.to_e4m3(x), one[0], okv.to_e4m3(w), one[1], "f32")
    assert np.array_equal(got, np.full((20, 130), 126.0))


def test_linear_values_that_are_not_finite(ts, sampler):
    """NaN codes and scales reach their own rows and columns, and no others."""
    rng = np.random.default_rng(4)
    x, xs, w, ws = linear_case(rng, 40, 300, 300)
    x[3, 299], w[7, 0], xs[5, 1], ws[2, 0] = 0x7F, 0xFF, np.nan, np.inf
    got = run_linear(ts, sampler, x, xs, w, ws, "f32", pad=1)
    want, size = olayer.linear(x, xs, w, ws)
    bad = np.zeros((40, 300), bool)
    bad[3], bad[:, 7], bad[5], bad[:, 256:] = True, True, True, True
    assert not np.isfinite(got[bad]).any()
    close(got[~bad], want[~bad], linear_bound(size, 300, "f32", want)[~bad])


def test_linear_again_and_on_another_stream(ts, sampler):
    """The same bits from every run, and from two streams' calls at once."""
    import torch
    rng = np.random.default_rng(5)
    cases = [linear_case(rng, m, n, k) for m, n, k in ((33, 700, 3000), (300, 260, 2000), (1, 4096, 4096))]
    first = [run_linear(ts, sampler, *c, "f32") for c in cases]
    calls = []
    for x, xs, w, ws in cases:
        e4m3 = [torch.zeros((a.shape[0], -(-a.shape[1] // 16) * 16), dtype=torch.uint8, device="cuda") for a in (x, w)]
        for t, a in zip(e4m3, (x, w)):
            t[:, :a.shape[1]] = torch.from_numpy(a).cuda()
        views = [t.view(torch.float8_e4m3fn)[:, :x.shape[1]] for t in e4m3]
        out = torch.zeros((x.shape[0], w.shape[0]), device="cuda")
        calls.append((ts.LinearE4m3(views[0], put(xs), views[1], put(ws), out), out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for (call, _), st in zip(calls, streams):
            ts.ts_linear_e4m3(sampler.handle, call, st)
    torch.cuda.synchronize()
    for (_, out), want in zip(calls, first):
        assert np.array_equal(get(out), want)


# --------------------------------------------------------------------------
# Rotary positions
# --------------------------------------------------------------------------
def rotary_bound(x, want, amplitude, kind, rot):
    """Cosine and sine within 2^-22 and their product with the amplitude, two products and
    a sum of sizes up to |a| + |b|; elements that are copied have none of it."""
    size = np.zeros_like(want)
    size[..., :rot] = 2 * np.abs(x[..., :rot]).max(-1, keepdims=True) * abs(amplitude)
    off = size * (2.0 ** -22 + 4 * 2.0 ** -24)
    return off + np.where(size > 0, HALF[kind] * (np.abs(want) + off) + TINY[kind], 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 2, 2), (3, 2, 7, 4), (5, 3, 64, 64), (9, 5, 80, 40), (33, 4, 128, 128), (64, 16, 128, 64),
                                                  (130, 1, 48, 24), (7, 9, 96, 96), (40, 3, 256, 16), (2, 3, 1024, 1000), (3, 70, 20, 18),
                                                  (700, 2, 72, 72)])
def test_rotary(ts, sampler, tokens, heads, dim, rot, kind, interleaved):
    import torch
    rng = np.random.default_rng([tokens, heads, dim])
    freqs, _ = ts.ts_rotary_frequencies(rot, 10000.0)
    f = torch.from_numpy(freqs).cuda()
    qkv = put(rng.normal(0, 3, (tokens, heads + 2, dim)), kind)
    x = qkv[:, 1:1 + heads]
    pos = rng.integers(0, 200000, tokens).astype(np.int32)
    pos[rng.random(tokens) < 0.2] = -1
    p = torch.from_numpy(pos).cuda()
    out = put(np.full((tokens, heads, dim), 7.0), kind)
    kept = get(qkv)
    ts.ts_rotary(sampler.handle, ts.Rotary(x, out, p, f, interleaved=interleaved, amplitude=1.25))
    used = pos >= 0
    want = olayer.rotary(get(x)[used], pos[used], freqs, interleaved=interleaved, amplitude=1.25)
    got = get(out)
    close(got[used], want, rotary_bound(get(x)[used], want, 1.25, kind, rot))
    assert np.all(got[~used] == 7) and np.array_equal(get(qkv), kept)
    ts.ts_rotary(sampler.handle, ts.Rotary(x, x, p, f, interleaved=interleaved, amplitude=1.25))  # in place
    after = get(qkv)
    assert np.array_equal(after[:, 1:1 + heads][used], got[used]) and np.array_equal(after[:, 1:1 + heads][~used], kept[:, 1:1 + heads][~used])
    assert np.array_equal(after[:, [0, -1]], kept[:, [0, -1]]) and sampler.read_status() == 0


def test_rotary_far_positions(ts, sampler):
    """Positions up to 2^31 - 1 and frequencies of several turns, negative and zero ones."""
    import torch
    pos = np.array([0, 1, 2 ** 20, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1], np.int32)
    freqs = np.array([1.0, 7.5, -0.3, 0.0, 1e-9, 100.0])
    x = put(np.ones((6, 1, 12)))
    out = torch.empty_like(x)
    ts.ts_rotary(sampler.handle, ts.Rotary(x, out, torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda()))
    import fractions
    two_pi = fractions.Fraction("6.283185307179586476925286766559005768394338798750211641949889")
    got = get(out)
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs):
            turn = fractions.Fraction(float(f)) * int(p) / two_pi
            angle = float((turn - int(turn)) * two_pi)
            c, s = np.cos(angle), np.sin(angle)
            # the frequency in turns, to 2^-52 of it, times the position
            off = 2 * np.pi * abs(f) / (2 * np.pi) * 2.0 ** -52 * float(p) + 2.0 ** -22 + 4 * 2.0 ** -24
            assert abs(got[t, 0, i] - (c - s)) <= 2 * off and abs(got[t, 0, i + 6] - (c + s)) <= 2 * off, (p, f)


def test_rotary_rows(ts, sampler):
    """A map of rows: those are turned by their tokens' positions, the others stay; rows
    outside the tensor are reported and skipped."""
    import torch
    rng = np.random.default_rng(8)
    freqs, _ = ts.ts_rotary_frequencies(32)
    x = put(rng.normal(0, 1, (10, 2, 32)), "bf16")
    rows, pos = np.array([7, 2, -1, 9, 10, 0, 3], np.int32), np.array([5, 100, -1, 77, 3, -1, 0], np.int32)
    out = put(np.full((10, 2, 32), 7.0), "bf16")
    sampler.read_status()
    ts.ts_rotary(sampler.handle, ts.Rotary(x, out, torch.from_numpy(pos).cuda(), torch.from_numpy(freqs).cuda(), rows=torch.from_numpy(rows).cuda()))
    assert sampler.read_status() == ts.TS_ROW_BAD_SLOT
    got = get(out)
    for r, p in ((7, 5), (2, 100), (9, 77), (3, 0)):
        want = olayer.rotary(get(x)[r:r + 1], [p], freqs, interleaved=False)
        close(got[r:r + 1], want, rotary_bound(get(x)[r:r + 1], want, 1.0, "bf16", 32))
    assert np.all(got[[0, 1, 4, 5, 6, 8]] == 7)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind,cache_kind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,block,hnd", [(1, 2, 1, 64, 64, 16, False), (37, 6, 3, 80, 40, 24, False), (130, 16, 8, 128, 128, 16, True),
                                                               (50, 0, 2, 96, 96, 7, False), (21, 5, 5, 48, 24, 8, True), (300, 4, 1, 256, 64, 32, False),
                                                               (9, 4, 2, 64, 18, 16, False)])
def test_append_rotary(ts, sampler, tokens, heads, kv, dim, rot, block, hnd, kind, cache_kind, interleaved):
    """Queries as ts_rotary leaves them; keys turned and rounded once; values, and for wide
    caches keys, bit for bit what ts_rotary and then ts_kv_append leave."""
    import torch
    rng = np.random.default_rng([tokens, heads, dim])
    freqs, _ = ts.ts_rotary_frequencies(rot)
    f = torch.from_numpy(freqs).cuda()
    n_blocks = tokens // block + 3
    rows_in = put(rng.normal(0, 3, (tokens + 4, heads + 2 * kv, dim)), kind)
    q, k_new, v_new = rows_in[:, :heads], rows_in[:, heads:heads + kv], rows_in[:, heads + kv:]
    pos, slots = rng.integers(0, 9000, tokens).astype(np.int32), rng.permutation(n_blocks * block)[:tokens].astype(np.int64)
    rows = rng.permutation(tokens + 4)[:tokens].astype(np.int32)
    pos[::7], slots[::7], rows[::7] = -1, -1, -1
    if tokens > 20:
        slots[3], pos[4] = -1, -1  # either skips the token
    p, sl, rw = (torch.from_numpy(a).cuda() for a in (pos, slots, rows))

    def cache():
        shape = (n_blocks, kv, block, dim) if hnd else (n_blocks, block, kv, dim)
        made = [torch.full(shape, 0.5, device="cuda").to(kind_of(cache_kind)) for _ in range(2)]
        return [x.permute(0, 2, 1, 3) if hnd else x for x in made]
    scales = [put(rng.uniform(0.01, 0.03, kv)) for _ in range(2)] if cache_kind == "e4m3" else [None, None]
    k, v = cache()
    out = torch.full((tokens + 4, max(1, heads), dim), 7.0, device="cuda").to(kind_of(kind))
    call = ts.Rotary(q if heads else out, out, p, f, rows=rw, interleaved=interleaved, amplitude=0.75)
    if not heads:
        call.c.x, call.c.n_heads = None, 0
    sampler.read_status()
    ts.ts_kv_append_rotary(sampler.handle, ts.KvCache(k, v, *scales), ts.KvTokens(k_new, v_new, sl, rw), call)
    assert sampler.read_status() == 0

    used = (pos >= 0) & (slots >= 0)
    pos2, slots2, rows2 = (torch.from_numpy(np.where(used, a, -1).astype(a.dtype)).cuda() for a in (pos, slots, rows))
    want_out = torch.full_like(out, 7.0)
    if heads:
        ts.ts_rotary(sampler.handle, ts.Rotary(q, want_out, pos2, f, rows=rows2, interleaved=interleaved, amplitude=0.75))
    assert torch.equal(out, want_out)
    k2, v2 = cache()
    turned = k_new.clone()
    ts.ts_rotary(sampler.handle, ts.Rotary(k_new, turned, pos2, f, rows=rows2, interleaved=interleaved, amplitude=0.75))
    ts.ts_kv_append(sampler.handle, ts.KvCache(k2, v2, *scales), ts.KvTokens(turned, v_new, slots2, rows2))
    raw = (lambda t: codes(t)) if cache_kind == "e4m3" else get
    assert np.array_equal(raw(v), raw(v2))
    if cache_kind != "e4m3" or kind == "f32":
        assert np.array_equal(raw(k), raw(k2))
    kk = get(k).reshape(n_blocks * block, kv, dim) if not hnd else get(k.contiguous()).reshape(n_blocks * block, kv, dim)
    src = get(k_new)[rows[used]]
    want = olayer.rotary(src, pos[used], freqs, interleaved=interleaved, amplitude=0.75)
    if cache_kind == "e4m3":
        s = get(scales[0])[None, :, None]
        size = 2 * np.abs(src).max(-1, keepdims=True) * 0.75 * (2.0 ** -22 + 4 * 2.0 ** -24)
        off = (size + 2.0 ** -24 * np.abs(want)) / s
        y = np.clip(want / s, -448, 448)
        close(kk[slots[used]], y, off + HALF["e4m3"] * (np.abs(y) + off) + TINY["e4m3"])
    else:
        copied = rotary_bound(src, want, 0.75, kind, rot)
        close(kk[slots[used]], want, copied)
    rest = np.setdiff1d(np.arange(n_blocks * block), slots[used])
    assert np.all(kk[rest] == 0.5)


@pytest.mark.parametrize("dim", [18, 64, 72])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_append_rotary_rounds_as_append(ts, sampler, kind, dim):
    """Values of every size, infinities and NaN among them, and scales that are zero, tiny,
    huge, infinite or NaN: the bytes that ts_kv_append writes.  Keys at position 0 (an
    angle of zero) too, but for their zeros' signs and infinities (inf - 0 inf)."""
    import torch
    rng = np.random.default_rng(dim)
    tokens, kv = 40, 8
    x = (rng.normal(0, 1, (tokens, 2 * kv, dim)) * 10.0 ** rng.integers(-40, 38, (tokens, 2 * kv, 1))).astype(np.float32)
    x[3, :, 0], x[4, kv:, 1], x[5, kv:, 2], x[6, kv:] = 0.0, np.inf, np.nan, -np.inf
    pad = -dim % 16  # the cache's rows are whole pieces of 16 bytes
    rows = put(np.pad(x, ((0, 0), (0, 0), (0, pad))), kind)
    wide = dim + pad
    scale = put(np.array([0.02, 0.0, 1e-38, 1e38, np.inf, np.nan, 1e-45, 3e-28]))
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    slots = torch.arange(tokens, device="cuda")
    f = torch.ones(dim // 2, dtype=torch.float64, device="cuda")
    caches = []
    for fused in (True, False):
        k, v = (torch.zeros((3, 16, kv, wide), dtype=torch.uint8, device="cuda").view(kind_of("e4m3")) for _ in range(2))
        cache, t = ts.KvCache(k, v, scale, scale), ts.KvTokens(rows[:, :kv], rows[:, kv:], slots)
        if fused:
            call = ts.Rotary(rows[:, :kv], torch.empty_like(rows[:, :kv]), pos, f)
            ts.ts_kv_append_rotary(sampler.handle, cache, t, call)
        else:
            ts.ts_kv_append(sampler.handle, cache, t)
        caches.append((codes(k), codes(v)))
    assert np.array_equal(caches[0][1], caches[1][1])
    same = caches[0][0] == caches[1][0]
    zeros = ((caches[0][0] | caches[1][0]) & 0x7F) == 0
    assert np.all(same | zeros) and sampler.read_status() == 0


def test_append_rotary_bad_maps(ts, sampler):
    """Slots past the cache and rows outside the tokens: reported, skipped, the rest done."""
    import torch
    rng = np.random.default_rng(9)
    freqs, _ = ts.ts_rotary_frequencies(64)
    x = put(rng.normal(0, 1, (6, 4, 64)), "bf16")
    k, v = (torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 32, 5, 6, 1 << 40, 31], device="cuda")
    rows = torch.tensor([0, 1, 6, -2, 4, 5], dtype=torch.int32, device="cuda")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    sampler.read_status()
    ts.ts_kv_append_rotary(sampler.handle, ts.KvCache(k, v), ts.KvTokens(x[:, 2:3], x[:, 3:], slots, rows),
                           ts.Rotary(x[:, :2], out, pos, torch.from_numpy(freqs).cuda(), rows=rows))
    assert sampler.read_status() == ts.TS_ROW_BAD_SLOT
    there = [0, 31]
    assert torch.equal(v.view(32, 64)[there], x[[0, 5], 3]) and bool((v.view(32, 64)[1:31] == 0).all())
    assert bool((out[[1, 2, 3, 4]] == 0).all()) and torch.equal(out[0], x[0, :2]) and bool((out[5] != 0).any())


# --------------------------------------------------------------------------
# Together
# --------------------------------------------------------------------------
class Layer:
    """One layer of a decode step, as the header lists it."""

    def __init__(self, ts, sampler, streams=5, dim=256, heads=4, kv=2, hd=64, ffn=384, block=16):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(1)
        self.ts, self.handle = ts, sampler.handle
        bf, e4, f32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32

        def zeros(*shape, kind=bf):
            return torch.zeros(shape, device="cuda", dtype=kind)

        def weight(n, k):
            w = torch.randn((n, k), device="cuda", generator=gen) / k ** 0.5
            codes = torch.zeros((n, k), device="cuda", dtype=e4)
            scale = torch.zeros((-(-n // 128), -(-k // 128)), device="cuda")
            for i in range(scale.shape[0]):
                for j in range(scale.shape[1]):
                    at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                    scale[i, j] = w[at].abs().max() / 448
                    codes[at] = (w[at] / scale[i, j]).to(e4)
            return codes, scale

        def linear(rows, codes, n, k, out):
            self.weights.append(weight(n, k))
            return ts.LinearE4m3(rows, codes, *self.weights[-1], out)
        self.weights = []
        self.x, self.hidden = zeros(streams, dim), zeros(streams, dim)
        self.norms = [1 + 0.1 * torch.randn(dim, device="cuda", generator=gen) for _ in range(2)]
        self.a8, self.a8s = zeros(streams, dim, kind=e4), zeros(streams, 2, kind=f32)
        self.qkv, self.q = zeros(streams, heads + 2 * kv, hd), zeros(streams, heads, hd)
        self.attn = zeros(streams, heads, hd)
        self.o8, self.o8s = zeros(streams, heads * hd, kind=e4), zeros(streams, heads * hd // 128, kind=f32)
        self.up, self.f8, self.f8s = zeros(streams, 2 * ffn), zeros(streams, ffn, kind=e4), zeros(streams, ffn // 128, kind=f32)
        self.tables = ts.KvTables(streams, 4, streams * 4, block, max_tokens=streams)
        self.cache = ts.KvCache(zeros(streams * 4, block, kv, hd), zeros(streams * 4, block, kv, hd))
        self.freqs, _ = ts.ts_rotary_frequencies(hd)
        t = self.tables
        self.calls = [
            (ts.ts_kv_tables, t),
            (ts.ts_rms_norm, ts.RmsNorm(self.x, self.a8, self.norms[0], residual=self.hidden, residual_out=self.hidden, out_scale=self.a8s)),
            (ts.ts_linear_e4m3, linear(self.a8, self.a8s, (heads + 2 * kv) * hd, dim, self.qkv.view(streams, -1))),
            (ts.ts_kv_append_rotary, self.cache, ts.KvTokens(self.qkv[:, heads:heads + kv], self.qkv[:, heads + kv:], t.slots, t.requests),
             ts.Rotary(self.qkv[:, :heads], self.q, t.positions, torch.from_numpy(self.freqs).cuda(), rows=t.requests)),
            (ts.ts_paged_attention, self.cache, ts.PagedQuery(self.q, self.attn, t.block_table, t.lens)),
            (ts.ts_gate, ts.Gate(self.attn.view(streams, -1), self.o8, activation="none", out_scale=self.o8s)),
            (ts.ts_linear_e4m3, linear(self.o8, self.o8s, dim, heads * hd, self.x)),
            (ts.ts_rms_norm, ts.RmsNorm(self.x, self.a8, self.norms[1], residual=self.hidden, residual_out=self.hidden, out_scale=self.a8s)),
            (ts.ts_linear_e4m3, linear(self.a8, self.a8s, 2 * ffn, dim, self.up)),
            (ts.ts_gate, ts.Gate(self.up[:, ffn:], self.f8, self.up[:, :ffn], out_scale=self.f8s)),
            (ts.ts_linear_e4m3, linear(self.f8, self.f8s, dim, ffn, self.x))]
        self.shape = (streams, dim, heads, kv, hd, ffn)

    def step(self):
        for call, *args in self.calls:
            call(self.handle, *args)

    def plain(self, frames):
        """The layer's outputs for the frames so far, in 64 bits and without 8-bit rows."""
        streams, dim, heads, kv, hd, ffn = self.shape
        w = [get(c) * olayer.of_columns(np.repeat(get(s), 128, 0)[:c.shape[0]], c.shape[1]) for c, s in self.weights]
        keys, values = [], []
        for t, x in enumerate(frames):
            h, y = olayer.rms_norm(x, get(self.norms[0]), np.zeros_like(x), eps=1e-6)
            qkv = (y @ w[0].T).reshape(streams, heads + 2 * kv, hd)
            pos = np.full(streams, t)
            q = olayer.rotary(qkv[:, :heads], pos, self.freqs, interleaved=False).reshape(streams, kv, heads // kv, hd)
            keys.append(olayer.rotary(qkv[:, heads:heads + kv], pos, self.freqs, interleaved=False))
            values.append(qkv[:, heads + kv:])
            s = np.einsum("nkgd,ntkd->nkgt", q, np.stack(keys, 1)) * hd ** -0.5
            p = np.exp(s - s.max(-1, keepdims=True))
            attn = np.einsum("nkgt,ntkd->nkgd", p / p.sum(-1, keepdims=True), np.stack(values, 1)).reshape(streams, -1)
            h, y = olayer.rms_norm(attn @ w[1].T, get(self.norms[1]), h, eps=1e-6)
            up = y @ w[2].T
            out = (olayer.activation(up[:, :ffn], "silu") * up[:, ffn:]) @ w[3].T
        return h, out


def test_a_layer_of_the_operators(ts, sampler):
    """Frames through a whole layer, plain calls and a replayed graph: the same bits; and
    near the 64-bit layer without 8-bit rows: five roundings to e4m3 (half a step, 2^-4 of
    a value, in sums of independent terms about a third of that) leave the outputs' norm
    within a quarter."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    frames = [torch.randn((5, 256), device="cuda", generator=gen).bfloat16() for _ in range(20)]
    runs = []
    for replay in (False, True):
        layer = Layer(ts, sampler)
        graph = None
        if replay:
            lens, free, stack = layer.tables.lens.clone(), layer.tables.n_free.clone(), layer.tables.free_blocks.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                layer.step()
            torch.cuda.current_stream().wait_stream(side)
            layer.tables.lens.copy_(lens), layer.tables.n_free.copy_(free), layer.tables.free_blocks.copy_(stack)
            layer.tables.block_table.fill_(-1)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layer.step()
        seen = []
        for x in frames:
            layer.x.copy_(x)
            layer.hidden.zero_()
            graph.replay() if replay else layer.step()
            seen.append((layer.x.clone(), layer.hidden.clone()))
        torch.cuda.synchronize()
        assert sampler.read_status() == 0 and layer.tables.lens.tolist() == [20] * 5
        runs.append(seen)
    for a, b in zip(*runs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for t in (0, 1, 19):
        h, out = Layer(ts, sampler).plain([get(x) for x in frames[:t + 1]])
        for got, want in ((runs[0][t][0], out), (runs[0][t][1], h)):
            assert np.linalg.norm(get(got) - want) <= 0.25 * np.linalg.norm(want)


def test_two_graphs_at_once(ts, sampler):
    """Two captured layers of one sampler's row operators, replayed on two streams: they
    share nothing."""
    import torch
    rng = np.random.default_rng(6)
    runs = []
    for i in range(2):
        x = put(rng.normal(0, 1, (64, 1024)), "bf16")
        e, s = put(np.zeros((64, 1024)), "e4m3"), put(np.zeros((64, 8)))
        w, ws = put(rng.normal(0, 100, (640, 1024)), "e4m3"), put(rng.uniform(0.5, 1, (5, 8)))
        out = put(np.zeros((64, 640)))
        calls = [(ts.ts_rms_norm, ts.RmsNorm(x, e, out_scale=s)), (ts.ts_linear_e4m3, ts.LinearE4m3(e, s, w, ws, out))]
        for fn, c in calls:
            fn(sampler.handle, c)
        torch.cuda.synchronize()
        want = out.clone()
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
    for _, out, want, _ in runs:  # bits: weights beyond 448 are NaN codes
        assert torch.equal(out.view(torch.int32), want.view(torch.int32))


def test_plain_launches(ts):
    """Without programmatic dependent launch: the same bits."""
    import torch
    rng = np.random.default_rng(7)
    x, w, ws = put(rng.normal(0, 1, (20, 640)), "bf16"), put(rng.normal(0, 100, (300, 640)), "e4m3"), put(rng.uniform(0.5, 1, (3, 5)))
    got = []
    for pdl in (1, 0):
        s = ts.Sampler(0)
        s.set_option(ts.TS_OPT_PDL, pdl)
        e, sc, out = put(np.zeros((20, 640)), "e4m3"), put(np.zeros((20, 5))), put(np.zeros((20, 300)), "bf16")
        ts.ts_rms_norm(s.handle, ts.RmsNorm(x, e, out_scale=sc))
        ts.ts_linear_e4m3(s.handle, ts.LinearE4m3(e, sc, w, ws, out))
        torch.cuda.synchronize()
        got.append(out.view(torch.int16))
        s.close()
    assert torch.equal(*got)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_decode_loop_on_8_bit_weights(cache):
    """The example's steps on 8-bit weights: graph replays against plain calls, every
    stream's length follows its steps until it ends, all blocks come back."""
    import os
    import sys
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import decode_loop
    finally:
        sys.path.pop(0)
    runs = []
    for replay in (False, True):
        loop = decode_loop.DecodeLoop(streams=6, steps=29, cache=cache, weights="e4m3", seed=3)
        step = loop.capture().replay if replay else loop.step
        seen = []
        for _ in range(31):
            step()
            seen.append([t.clone() for t in (loop.batch.out_ids, loop.batch.finish_reason, loop.tables.lens, loop.h)])
        torch.cuda.synchronize()
        assert loop.sampler.read_status() == 0 and loop.tables.n_free.item() == loop.n_blocks
        runs.append(seen)
    for a, b in zip(*runs):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    done = torch.zeros(6, dtype=torch.bool, device="cuda")
    for i, (_, finish, lens, h) in enumerate(runs[0]):
        assert torch.equal(lens, torch.where(done, 0, i + 1).int()) and bool(torch.isfinite(h[~done]).all())
        done = finish > 0
    assert bool(done.all())
