"""The layer operators' C structs and their Python mirrors, what they refuse, the rotary
frequencies and the plain 64-bit versions' own pins (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import kv as okv
from oracle import layer as olayer
from test_abi import _c_layout

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ts():
    import codebook_token_sampling_gb300 as mod
    return mod


class _Stream:
    cuda_stream = 0


@pytest.fixture(scope="module")
def blank():
    """A handle of zeros: enough for calls that are refused, or that have nothing to do."""
    return ctypes.create_string_buffer(1 << 16)


def refused(ts, call, blank, *args):
    with pytest.raises(ts.SamplerError) as e:
        call(ctypes.addressof(blank), *args, _Stream)
    return e.value.status


def test_structs_match_the_header(ts, tmp_path):
    for struct, mirror in (("ts_norm_args", ts.TsNorm), ("ts_gate_args", ts.TsGate), ("ts_linear_args", ts.TsLinear),
                           ("ts_rotary_args", ts.TsRotary)):
        fields = [name for name, _ in mirror._fields_]
        want = [getattr(mirror, f).offset for f in fields] + [ctypes.sizeof(mirror)]
        assert _c_layout(tmp_path, struct, fields) == want, struct


def test_enum_values(ts, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ("TS_ACT_NONE", "TS_ACT_SILU", "TS_ACT_GELU", "TS_ACT_GELU_TANH")
    src = tmp_path / "acts.c"
    src.write_text('#include <stdio.h>\n#include "ts_sampler.h"\nint main(void) {'
                   + "".join(f'printf("%d\\n", {n});' for n in names) + "return 0; }\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "acts")],
                   check=True, capture_output=True)
    out = subprocess.run([str(tmp_path / "acts")], check=True, capture_output=True, text=True).stdout
    assert [int(x) for x in out.split()] == [getattr(ts, n) for n in names]


# --------------------------------------------------------------------------
# pins of the 64-bit versions
# --------------------------------------------------------------------------
def test_oracle_by_hand():
    h, y = olayer.rms_norm([[3.0, 4.0]], [1.0, 2.0], [[0.0, 0.0]], eps=0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]]) and np.array_equal(h, [[3.0, 4.0]])
    _, y = olayer.rms_norm([[1.0, 1.0]], [0.0, 1.0], [[1.0, 1.0]], eps=12.0, weight_offset=1.0)
    assert np.allclose(y, [[0.5, 1.0]])
    assert np.allclose(olayer.activation([0.0, 1.0], "silu"), [0, 1 / (1 + math.exp(-1))])
    assert np.allclose(olayer.activation([1.0, -40.0], "gelu"), [0.8413447460685429, 0])
    assert np.allclose(olayer.activation([1.0], "gelu_tanh"), 0.8411919906082768)
    turned = olayer.rotary(np.array([[[1.0, 0.0, 5.0]]]), [1], [math.pi / 2], interleaved=True)
    assert np.allclose(turned, [[[0.0, 1.0, 5.0]]])
    x = np.arange(4.0).reshape(1, 1, 4)
    assert np.allclose(olayer.rotary(x, [2], [math.pi / 4, 0.0], interleaved=False), [[[-2.0, 1.0, 0.0, 3.0]]])
    assert np.allclose(olayer.rotary(x, [2], [math.pi / 4, 0.0], interleaved=True), [[[-1.0, 0.0, 2.0, 3.0]]])


def test_oracle_blocks():
    y = np.zeros((2, 130), np.float32)
    y[0, 3], y[0, 129], y[1, 0] = -896.0, 1e-30, np.inf
    codes, scale = olayer.quantised_f32(y)
    assert scale[0].tolist() == [2.0, np.float32(2.0 ** -64) / np.float32(448)] and np.isnan(scale[1, 0]) and scale[1, 1] > 0
    assert okv.from_e4m3(codes[0, 3]) == -448 and codes[0, 129] == 0 and np.all(codes[1, :128] & 0x7F == 0x7F)
    assert np.array_equal(olayer.block_scales(y[:1].astype(float)).astype(np.float32), scale[:1])
    x = okv.to_e4m3(np.ones((1, 130)))
    out, size = olayer.linear(x, [[2.0, 3.0]], okv.to_e4m3(-np.ones((129, 130))), [[1.0, 10.0], [0.5, 0.0]])
    assert out[0, 0] == -(256 + 60) and out[0, 128] == -128 and size[0, 128] == 128


# --------------------------------------------------------------------------
# frequencies
# --------------------------------------------------------------------------
def test_frequencies(ts):
    i = np.arange(32)
    plain, amp = ts.ts_rotary_frequencies(64, 10000.0)
    f = 10000.0 ** (-2 * i / 64)
    assert np.allclose(plain, f, rtol=1e-15) and amp == 1.0 and plain[0] == 1.0
    linear, amp = ts.ts_rotary_frequencies(64, 10000.0, ts.TS_ROPE_LINEAR, factor=8.0)
    assert np.allclose(linear, f / 8, rtol=1e-15) and amp == 1.0
    ntk, amp = ts.ts_rotary_frequencies(64, 10000.0, ts.TS_ROPE_NTK, factor=8.0)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 8, rtol=1e-13) and amp == 1.0 and np.all(np.diff(ntk) < 0)
    parts, amp = ts.ts_rotary_frequencies(64, 10000.0, ts.TS_ROPE_BY_PARTS, factor=8.0, original_len=4096, low=1.0, high=32.0)
    turns = 4096 * f / (2 * math.pi)
    r = np.clip((turns - 1) / 31, 0, 1)
    assert np.allclose(parts, f * ((1 - r) / 8 + r), rtol=1e-14)
    assert parts[0] == 1.0 and np.isclose(parts[-1], f[-1] / 8) and np.isclose(amp, 0.1 * math.log(8) + 1)


@pytest.mark.parametrize("args", [
    dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=-2), dict(base=0.0), dict(base=math.inf), dict(base=-1.0), dict(scaling=4),
    dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan), dict(scaling=2, factor=2.0, rotary_dim=2),
    dict(scaling=3, factor=2.0, original_len=0.0), dict(scaling=3, factor=2.0, original_len=100, low=2.0, high=2.0),
    dict(scaling=3, factor=2.0, original_len=math.inf), dict(scaling=3, factor=2.0, original_len=10, low=math.nan)])
def test_frequencies_refusals(ts, args):
    with pytest.raises((ts.SamplerError, ValueError)):
        ts.ts_rotary_frequencies(**{"rotary_dim": 64, **args})


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def norm(ts, n=4, dim=256, out="bf16", **kw):
    x = torch.zeros((n, dim), dtype=torch.bfloat16)
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
    scale = torch.zeros((n, -(-dim // 128))) if out == "e4m3" else None
    return ts.RmsNorm(x, torch.zeros((n, dim)).to(kinds[out]), torch.ones(dim), residual=torch.zeros_like(x),
                      residual_out=torch.zeros_like(x), out_scale=scale, **kw)


def test_norm_refusals(ts, blank):
    bad, no = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    cases = [("n_rows", -1, bad), ("dim", 0, bad), ("dtype", 2, bad), ("dtype", 9, bad), ("out_dtype", 5, bad), ("weight_dtype", 2, bad),
             ("eps", -1e-6, bad), ("eps", math.nan, bad), ("eps", math.inf, bad), ("weight_offset", math.nan, bad), ("x_stride", 255, bad),
             ("out_stride", -1, bad), ("residual_stride", 0, bad), ("residual_out_stride", 10, bad), ("out_scale_stride", 1, bad),
             ("x", None, bad), ("out", None, bad), ("out_scale", None, bad), ("dim", 32769, bad)]
    for field, value, status in cases:
        call = norm(ts, out="e4m3")
        setattr(call.c, field, value)
        assert refused(ts, ts.ts_rms_norm, blank, call) == status, field
    for field in ("x", "residual", "residual_out", "weight", "out"):  # not aligned to their elements
        call = norm(ts, out="f32")
        setattr(call.c, field, getattr(call.c, field) + 1)
        assert refused(ts, ts.ts_rms_norm, blank, call) == bad, field
    for out, inside in (("out", "weight"), ("residual_out", "weight"), ("out", "residual"), ("out", "residual_out"), ("residual_out", "x"),
                        ("out_scale", "x"), ("out_scale", "residual"), ("out_scale", "out"), ("out", "x")):
        call = norm(ts, out="e4m3")
        setattr(call.c, out, getattr(call.c, inside) + 64)
        assert refused(ts, ts.ts_rms_norm, blank, call) == bad, (out, inside)
    call = norm(ts, n=1, dim=32776)
    assert refused(ts, ts.ts_rms_norm, blank, call) == no
    call = norm(ts)
    call.c.out_scale = call.c.x
    assert refused(ts, ts.ts_rms_norm, blank, call) == bad
    none = norm(ts)
    none.c.n_rows = 0
    ts.ts_rms_norm(ctypes.addressof(blank), none, _Stream)
    ts.ts_rms_norm(ctypes.addressof(blank), norm(ts, n=0), _Stream)


def test_norm_binding(ts):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    e4m3, w = torch.float8_e4m3fn, torch.ones(256)
    for bad in (dict(out=torch.zeros(4, 255)), dict(out=torch.zeros((4, 256), dtype=torch.float64)), dict(weight=torch.ones(255)),
                dict(weight=w.double()), dict(residual=x.float()), dict(residual_out=x[:3]), dict(out=x.to(e4m3)),
                dict(out_scale=torch.zeros(4, 2)), dict(out=x.to(e4m3), out_scale=torch.zeros(4, 1)), dict(x=x[:, ::2], out=x[:, ::2]),
                dict(x=x[:1].expand(4, 256)), dict(out=x.to("meta")), dict(out=x.to(e4m3), out_scale=torch.zeros((4, 2), dtype=torch.float64)),
                dict(weight=w[::2].repeat(2)[::2])):
        args = {"x": x, "out": torch.zeros_like(x), "weight": w, **bad}
        with pytest.raises(ValueError):
            ts.RmsNorm(args.pop("x"), args.pop("out"), args.pop("weight"), **args)
    wide = torch.zeros((4, 600), dtype=torch.bfloat16)
    made = ts.RmsNorm(wide[:, 8:264], x.to(e4m3), w, out_scale=torch.zeros(4, 3)[:, :2])
    assert made.c.x_stride == 600 and made.c.out_scale_stride == 3 and made.c.out_stride == 256


def gate(ts, n=4, dim=256, act="silu"):
    both = torch.zeros((n, 2 * dim), dtype=torch.bfloat16)
    return ts.Gate(both[:, dim:], torch.zeros((n, dim)).to(torch.float8_e4m3fn), both[:, :dim] if act != "none" else None, activation=act,
                   out_scale=torch.zeros((n, -(-dim // 128))))


def test_gate_refusals(ts, blank):
    bad = ts.TS_ERR_INVALID_ARG
    for field, value in (("n_rows", -1), ("dim", 0), ("dtype", 2), ("out_dtype", 3), ("act", -1), ("act", 4), ("up", None), ("gate", None),
                         ("out", None), ("out_scale", None), ("up_stride", 100), ("gate_stride", -5), ("out_stride", 0),
                         ("out_scale_stride", 1), ("out_dtype", 0)):
        call = gate(ts)
        setattr(call.c, field, value)
        assert refused(ts, ts.ts_gate, blank, call) == bad, field
    for field in ("up", "gate"):
        call = gate(ts)
        setattr(call.c, field, getattr(call.c, field) + 1)
        assert refused(ts, ts.ts_gate, blank, call) == bad
    for out, inside in (("out", "up"), ("out", "gate"), ("out_scale", "up"), ("out_scale", "gate"), ("out_scale", "out")):
        call = gate(ts)
        setattr(call.c, out, getattr(call.c, inside) + 16)
        assert refused(ts, ts.ts_gate, blank, call) == bad
    big = gate(ts, n=1, dim=1048584)
    assert refused(ts, ts.ts_gate, blank, big) == ts.TS_ERR_UNSUPPORTED
    ts.ts_gate(ctypes.addressof(blank), gate(ts, n=0), _Stream)
    up = torch.zeros((4, 256))
    for args in (dict(activation="relu", gate=up), dict(activation="silu"), dict(activation="none", gate=up), dict(gate=up.bfloat16()),
                 dict(gate=up[:, :128])):
        with pytest.raises(ValueError):
            ts.Gate(up, torch.zeros_like(up), **args)


def linear(ts, m=4, n=256, k=272, out=torch.bfloat16):
    def e4m3(*shape):
        return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return ts.LinearE4m3(e4m3(m, k), torch.zeros(m, -(-k // 128)), e4m3(n, k), torch.zeros(-(-n // 128), -(-k // 128)),
                         torch.zeros((m, n), dtype=out))


def test_linear_refusals(ts, blank):
    bad, no = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    for field, value, status in (("n_rows", -1, bad), ("in_dim", 0, bad), ("out_dim", 0, bad), ("out_dtype", 2, bad), ("x_stride", 256, bad),
                                 ("w_stride", 256, bad), ("x_stride", 280, bad), ("w_stride", 280, bad), ("out_stride", 255, bad),
                                 ("x_scale_stride", 2, bad), ("w_scale_stride", 2, bad), ("x", None, bad), ("x_scale", None, bad),
                                 ("w", None, bad), ("w_scale", None, bad), ("out", None, bad), ("x_stride", 1 << 40, no),
                                 ("w_stride", 1 << 41, no), ("w_stride", -16, bad)):
        call = linear(ts)
        setattr(call.c, field, value)
        assert refused(ts, ts.ts_linear_e4m3, blank, call) == status, field
    for field, by in (("x", 8), ("w", 8), ("x_scale", 2), ("w_scale", 1), ("out", 1)):
        call = linear(ts)
        setattr(call.c, field, getattr(call.c, field) + by)
        assert refused(ts, ts.ts_linear_e4m3, blank, call) == bad, field
    for inside in ("x", "w", "x_scale", "w_scale"):
        call = linear(ts)
        call.c.out = getattr(call.c, inside)
        assert refused(ts, ts.ts_linear_e4m3, blank, call) == bad, inside
    call = linear(ts, m=1, n=1, k=1048592)
    assert refused(ts, ts.ts_linear_e4m3, blank, call) == no
    ts.ts_linear_e4m3(ctypes.addressof(blank), linear(ts, m=0), _Stream)
    x = torch.zeros((4, 256), dtype=torch.uint8).view(torch.float8_e4m3fn)
    xs, ws, out = torch.zeros(4, 2), torch.zeros(1, 2), torch.zeros(4, 4)
    for args in ((x, xs, x.float(), ws, out), (x, xs[:, :1], x, ws, out), (x, xs, x[:, :128], ws, out), (x, xs, x, torch.zeros(2, 2), out),
                 (x, xs, x, ws, out.half()), (x, xs, x, ws, out[:3]), (x, xs, x.to("meta"), ws, out)):
        with pytest.raises(ValueError):
            ts.LinearE4m3(*args)


def rotary(ts, n=4, heads=3, dim=64, rot=64, rows=None, **kw):
    x = torch.zeros((n, heads, dim), dtype=torch.bfloat16)
    return ts.Rotary(x, torch.zeros_like(x), torch.zeros(n if rows is None else rows.numel(), dtype=torch.int32),
                     torch.ones(rot // 2, dtype=torch.float64), rows=rows, **kw)


def test_rotary_refusals(ts, blank):
    bad, no = ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED
    for field, value, status in (("n_tokens", -1, bad), ("n_heads", 0, bad), ("n_heads", 65537, no), ("head_dim", 0, bad), ("head_dim", 1025, no),
                                 ("rotary_dim", 0, bad), ("rotary_dim", 63, bad), ("rotary_dim", 66, bad), ("dtype", 2, bad),
                                 ("x", None, bad), ("out", None, bad), ("positions", None, bad), ("freqs", None, bad),
                                 ("amplitude", math.inf, bad), ("x_token_stride", -1, bad), ("out_head_stride", -64, bad)):
        call = rotary(ts)
        setattr(call.c, field, value)
        assert refused(ts, ts.ts_rotary, blank, call) == status, field
    for field in ("x", "out", "freqs"):
        call = rotary(ts)
        setattr(call.c, field, getattr(call.c, field) + 1)
        assert refused(ts, ts.ts_rotary, blank, call) == bad, field
    call = rotary(ts)
    call.c.out, call.c.out_token_stride = call.c.x, call.c.x_token_stride + 64
    assert refused(ts, ts.ts_rotary, blank, call) == bad
    call = rotary(ts, rows=torch.zeros(4, dtype=torch.int32))
    call.c.n_rows = -1
    assert refused(ts, ts.ts_rotary, blank, call) == bad
    ts.ts_rotary(ctypes.addressof(blank), rotary(ts, n=0), _Stream)
    x = torch.zeros((4, 3, 64), dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    for args in ((x, x.float(), pos, f), (x, x[:3], pos, f), (x.half(), x.half(), pos, f), (x, x, pos.long(), f), (x, x, pos[:3], f),
                 (x, x, pos, f.float()), (x, x, pos, torch.ones(33, dtype=torch.float64)), (x, x, pos, f[:0]),
                 (x.transpose(1, 2), x.transpose(1, 2), pos, f[:1]), (x, x, pos.to("meta"), f)):
        with pytest.raises(ValueError):
            ts.Rotary(*args)


def test_rotary_outputs_that_overlap(ts, blank):
    """Heads or rows of out on one another; one head's and one row's strides say nothing."""
    bad = ts.TS_ERR_INVALID_ARG
    for field, value in (("out_head_stride", 0), ("out_head_stride", 63), ("out_token_stride", 0), ("out_token_stride", 63)):
        call = rotary(ts)
        setattr(call.c, field, value)
        assert refused(ts, ts.ts_rotary, blank, call) == bad, (field, value)
    call = rotary(ts, rows=torch.zeros(4, dtype=torch.int32))
    call.c.out_token_stride = 0
    assert refused(ts, ts.ts_rotary, blank, call) == bad
    x = torch.zeros((4, 3, 64), dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    call = ts.Rotary(x, x[:1].expand(4, 3, 64), pos, f)
    assert refused(ts, ts.ts_rotary, blank, call) == bad


def test_append_rotary_refusals(ts, blank):
    bad = ts.TS_ERR_INVALID_ARG

    def cache(heads=2, dim=64, dtype=torch.bfloat16):
        k = torch.zeros((2, 16, heads, dim), dtype=dtype)
        return ts.KvCache(k, torch.zeros_like(k))

    def tokens(n=4, heads=2, dim=64, dtype=torch.bfloat16, rows=None):
        k = torch.zeros((n, heads, dim), dtype=dtype)
        return ts.KvTokens(k, k, torch.zeros(n, dtype=torch.int64), rows)
    rows = torch.zeros(4, dtype=torch.int32)
    for c, t, r in ((cache(), tokens(n=3), rotary(ts)), (cache(), tokens(rows=rows), rotary(ts)), (cache(), tokens(), rotary(ts, rows=rows)),
                    (cache(), tokens(rows=rows), rotary(ts, rows=rows.clone())), (cache(), tokens(rows=rows), rotary(ts, n=5, rows=rows))):
        assert refused(ts, ts.ts_kv_append_rotary, blank, c, t, r) == bad
    assert refused(ts, ts.ts_kv_append_rotary, blank, cache(dtype=torch.float32), tokens(), rotary(ts)) == ts.TS_ERR_UNSUPPORTED
    assert refused(ts, ts.ts_kv_append_rotary, blank, cache(dtype=torch.float32), tokens(dtype=torch.float32), rotary(ts)) == bad
    for field, value in (("x", None), ("n_heads", 0), ("freqs", None), ("rotary_dim", 65)):
        r = rotary(ts)
        setattr(r.c, field, value)
        assert refused(ts, ts.ts_kv_append_rotary, blank, cache(), tokens(), r) == bad, field
    t = tokens()
    t.c.slots = None
    assert refused(ts, ts.ts_kv_append_rotary, blank, cache(), t, rotary(ts)) == bad
    none = rotary(ts, n=0)
    none.c.x, none.c.n_heads = None, 0
    ts.ts_kv_append_rotary(ctypes.addressof(blank), cache(), tokens(n=0), none, _Stream)
    for c, t, r in ((cache(), tokens(heads=3), rotary(ts)), (cache(), tokens(dim=32), rotary(ts)), (cache(), tokens(), rotary(ts, dim=128))):
        with pytest.raises(ValueError):
            ts.ts_kv_append_rotary(ctypes.addressof(blank), c, t, r, _Stream)


def test_a_missing_handle_is_refused(ts):
    for call, args in ((ts.ts_rms_norm, (norm(ts),)), (ts.ts_gate, (gate(ts),)), (ts.ts_linear_e4m3, (linear(ts),)), (ts.ts_rotary, (rotary(ts),))):
        with pytest.raises(ts.SamplerError):
            call(None, *args, _Stream)
