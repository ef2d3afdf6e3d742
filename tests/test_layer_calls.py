"""Calls of the layer operators that the header allows or refuses, without a GPU."""
import ctypes

import pytest

from test_layer_binding import _Stream, blank, refused, rotary, ts  # noqa: F401  (fixtures among them)

torch = pytest.importorskip("torch")


def cache(ts, heads=2, dim=64):
    k = torch.zeros((2, 16, heads, dim), dtype=torch.bfloat16)
    return ts.KvCache(k, torch.zeros_like(k))


def tokens(ts, n=4, heads=2, dim=64, rows=None):
    k = torch.zeros((n if rows is None else rows.numel(), heads, dim), dtype=torch.bfloat16)
    return ts.KvTokens(k, torch.zeros_like(k), torch.zeros(n, dtype=torch.int64), rows)


def test_a_step_without_tokens_is_no_error(ts, blank):
    """An empty batch's tensors have no address: queries with heads and without rows."""
    call = rotary(ts, n=0)
    assert call.c.x is None and call.c.n_heads == 3
    ts.ts_kv_append_rotary(ctypes.addressof(blank), cache(ts), tokens(ts, n=0), call, _Stream)
    ts.ts_rotary(ctypes.addressof(blank), call, _Stream)
    for heads in (-1, 65537):
        call.c.n_heads = heads
        assert refused(ts, ts.ts_kv_append_rotary, blank, cache(ts), tokens(ts, n=0), call) in (ts.TS_ERR_INVALID_ARG, ts.TS_ERR_UNSUPPORTED)
    call = rotary(ts)
    call.c.x = None  # with tokens, they are missing
    assert refused(ts, ts.ts_kv_append_rotary, blank, cache(ts), tokens(ts), call) == ts.TS_ERR_INVALID_ARG
