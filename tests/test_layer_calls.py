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


# --------------------------------------------------------------------------
# Rotary outputs that lie on something else
# --------------------------------------------------------------------------
def rotary_of(ts, x, out, rows=None):
    n = x.shape[0] if rows is None else rows.numel()
    return ts.Rotary(x, out, torch.zeros(n, dtype=torch.int32), torch.ones(32, dtype=torch.float64), rows=rows)


def test_rotary_output_whose_rows_interleave(ts, blank):
    """Each stride holds a head, but a row's second head lies on the next row's first."""
    bf16 = torch.bfloat16
    x, buf = torch.zeros((4, 3, 64), dtype=bf16), torch.zeros(4096, dtype=bf16)
    for token, head in ((64, 64), (128, 64), (191, 64), (64, 128), (64, 255), (100, 100)):
        call = rotary_of(ts, x, buf.as_strided((4, 3, 64), (token, head, 1)))
        assert refused(ts, ts.ts_rotary, blank, call) == ts.TS_ERR_INVALID_ARG, (token, head)


def test_rotary_output_over_its_input(ts, blank):
    """By some elements, by a head, by a row: only x itself may be the output."""
    bf16 = torch.bfloat16
    buf = torch.zeros(8192, dtype=bf16)
    x = buf[2048:].as_strided((4, 3, 64), (192, 64, 1))
    for by in (8, -8, 64, -64, 192, -192, 3 * 192, -3 * 192, 3 * 192 + 191, -3 * 192 - 191):
        out = torch.as_strided(buf, (4, 3, 64), (192, 64, 1), 2048 + by)
        assert refused(ts, ts.ts_rotary, blank, rotary_of(ts, x, out)) == ts.TS_ERR_INVALID_ARG, by
    out = torch.as_strided(buf, (4, 3, 64), (200, 64, 1), 2048 + 64)  # of another pitch
    assert refused(ts, ts.ts_rotary, blank, rotary_of(ts, x, out)) == ts.TS_ERR_INVALID_ARG


def test_append_rotary_output_over_keys_values_and_cache(ts, blank):
    bf16, bad = torch.bfloat16, ts.TS_ERR_INVALID_ARG
    qkv = torch.zeros((4, 7, 64), dtype=bf16)  # 3 + 2 + 2 heads
    new = ts.KvTokens(qkv[:, 3:5], qkv[:, 5:7], torch.zeros(4, dtype=torch.int64))
    for first in (1, 2, 3, 4):
        out = qkv[:, first:first + 3]
        call = rotary_of(ts, torch.zeros((4, 3, 64), dtype=bf16), out)
        assert refused(ts, ts.ts_kv_append_rotary, blank, cache(ts), new, call) == bad, first
    pool = cache(ts)
    for t in (pool.k, pool.v):
        out = t.view(-1)[1024:].as_strided((4, 3, 64), (192, 64, 1))
        call = rotary_of(ts, torch.zeros((4, 3, 64), dtype=bf16), out)
        assert refused(ts, ts.ts_kv_append_rotary, blank, pool, tokens(ts), call) == bad


PROGRAM = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "ts_overlap.h"
using ts_host::Heads;
int main() {
  std::mt19937 rng(1);
  const auto any = [&](int lo, int hi) { return static_cast<int64_t>(rng() % (hi - lo + 1) + lo); };
  int both = 0, neither = 0, careful = 0;
  for (int n = 0; n < 400000; ++n) {
    const int64_t wide = any(1, 4), base = 1 << 20;
    const Heads a = {static_cast<uintptr_t>(base + any(0, 60)), any(1, 5), any(1, 5), any(0, 24), any(0, 24), wide};
    Heads b = {static_cast<uintptr_t>(base + any(0, 60)), any(1, 5), any(1, 5), any(0, 24), any(0, 24), wide};
    const bool alike = n % 2;
    if (alike) b.row = a.row, b.head = a.head;
    std::vector<int> used(400, 0);
    bool itself = false, meet = false;
    for (int pass = 0; pass < 2; ++pass) {
      const Heads &x = pass ? b : a;
      for (int64_t r = 0; r < x.rows; ++r)
        for (int64_t h = 0; h < x.heads; ++h)
          for (int64_t d = 0; d < x.wide; ++d) {
            int &u = used[x.from + r * x.row + h * x.head + d - base];
            if (!pass) itself = itself || u, u = 1;
            else meet = meet || u;
          }
    }
    if (itself && !a.meets_itself()) return std::printf("missed itself\n"), 1;
    if (meet && !(a.meets(b) && b.meets(a))) return std::printf("missed\n"), 1;
    if (alike && meet != a.meets(b)) return std::printf("not exact\n"), 1;
    both += meet, neither += !meet && !a.meets(b), careful += !meet && a.meets(b);
  }
  std::printf("%d %d %d\n", both, neither, careful);
  return 0;
}
"""


def test_overlaps_by_counting_bytes(tmp_path):
    """Random layouts against their bytes one by one: no overlap is missed, and those of
    equal strides are answered exactly."""
    import os
    import subprocess
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "codebook_token_sampling_gb300", "csrc")
    (tmp_path / "o.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(tmp_path / "o.cc"), "-o", str(tmp_path / "o")], check=True)
    done = subprocess.run([str(tmp_path / "o")], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
    assert all(int(x) > 1000 for x in done.stdout.split())
