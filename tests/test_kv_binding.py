"""The paged cache's C structs and their Python mirrors, and the plain 64-bit
versions' own pins (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import kv as okv
from test_abi import _c_layout


def test_structs_match_the_header(tmp_path):
    import codebook_token_sampling_gb300 as ts
    for struct, mirror in (("ts_kv_tables_args", ts.TsKvTables), ("ts_kv_cache", ts.TsKvCache),
                           ("ts_kv_tokens", ts.TsKvTokens), ("ts_paged_query", ts.TsPagedQuery)):
        fields = [name for name, _ in mirror._fields_]
        want = [getattr(mirror, f).offset for f in fields] + [ctypes.sizeof(mirror)]
        assert _c_layout(tmp_path, struct, fields) == want, struct


def test_e4m3_codes():
    values = okv.e4m3_values()
    assert values[0] == 0 and values[1] == 2.0 ** -9 and values[8] == 2.0 ** -6 and values[126] == 448
    assert np.all(np.diff(values) > 0)
    codes = np.arange(127, dtype=np.uint8)
    assert np.array_equal(okv.to_e4m3(values), codes)
    assert np.array_equal(okv.from_e4m3(codes), values)
    assert okv.to_e4m3([1e9, -1e9, 1.0625, 1.1875]).tolist() == [126, 254, 56, 58]  # ties to even codes
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).normal(0, 50, 5000).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(okv.to_e4m3(x), want)


def test_tables_by_hand():
    """Three requests of 2-token blocks: one ends (its block 5 goes on the
    stack), one crosses a block, one stays inside its block."""
    got = okv.tables([[4, -1], [5, -1], [6, -1]], [2, 2, 1], None, [0, 1, 0], [7, 8, -1, -1], 2, block_size=2, n_blocks=9,
                     max_tokens=4)
    assert got["block_table"].tolist() == [[4, 5], [5, -1], [6, -1]]
    assert got["free_blocks"].tolist() == [7, 8, 5, -1] and got["n_free"] == 2
    assert got["lens"].tolist() == [3, 0, 2] and got["token_starts"].tolist() == [0, 1, 1, 2]
    assert got["slots"].tolist() == [10, 13, -1, -1] and got["positions"].tolist() == [2, 1, -1, -1]
    assert got["requests"].tolist() == [0, 2, -1, -1] and got["status"] == 0


def test_tables_without_blocks():
    got = okv.tables([[-1], [0]], [0, 1], None, None, [], 0, block_size=2, n_blocks=1, max_tokens=2)
    assert got["lens"].tolist() == [0, 2] and got["status"] == okv.NO_BLOCKS and got["slots"].tolist() == [1, -1]


def test_attention_by_hand():
    """Two keys with scores 0 and ln 3: weights 1/4 and 3/4."""
    k = np.zeros((1, 2, 1, 1))
    k[0, 1, 0, 0] = np.log(3)
    v = np.array([8.0, 4.0]).reshape(1, 2, 1, 1)
    got = okv.attention(np.ones((1, 1, 1)), k, v, np.array([[0]]), [2], scale=1.0, n_blocks=1)
    assert np.isclose(got["out"][0, 0, 0], 5.0) and np.isclose(got["lse"][0, 0], np.log(4))
    none = okv.attention(np.ones((1, 1, 1)), k, v, np.array([[0]]), [2], scale=1.0, n_blocks=1, key_mask=[[0, 0]])
    assert none["out"][0, 0, 0] == 0 and none["lse"][0, 0] == -np.inf
    last = okv.attention(np.ones((1, 1, 1)), k, v, np.array([[0]]), [2], scale=1.0, n_blocks=1, window=1)
    assert last["out"][0, 0, 0] == 4.0


def test_table_rows_are_rows_of_their_own():
    """A table whose rows overlap in memory (one row expanded to all requests) is
    refused; strided rows and a single row keep their meaning."""
    import torch
    import codebook_token_sampling_gb300 as ts
    i32 = torch.int32

    def query(table):
        n = table.shape[0]
        q = torch.zeros((n, 2, 64), dtype=torch.bfloat16)
        return ts.PagedQuery(q, torch.empty_like(q), table, torch.zeros(n, dtype=i32))

    def tables(table):
        return ts.KvTables(*table.shape, 100, 16, max_tokens=4, block_table=table, device="cpu")
    row = torch.arange(8, dtype=i32)
    wide = torch.zeros((4, 20), dtype=i32)
    for make in (query, tables):
        for bad in (row.expand(4, -1), row.as_strided((3, 6), (1, 1)), wide[:, ::2], wide.t()[:8]):
            with pytest.raises(ValueError):
                make(bad)
        assert make(wide).c.table_stride == 20 and make(wide[:, 3:11]).c.table_stride == 20
        assert make(wide[::2]).c.table_stride == 40
        for one in (row.expand(1, -1), wide[1:2, :8], row.as_strided((1, 8), (0, 1))):
            made = make(one)
            assert made.c.table_stride >= 8 and made.c.max_blocks == 8


class _Stream:
    cuda_stream = 0


def test_tokens_and_queries_fit_the_cache():
    """Heads, row widths and devices are compared before a call reaches the
    library (which here refuses the NULL handle of those that fit)."""
    import torch
    import codebook_token_sampling_gb300 as ts

    def cache(heads, dim):
        k = torch.zeros((2, 16, heads, dim), dtype=torch.bfloat16)
        return ts.KvCache(k, torch.zeros_like(k))

    def tokens(heads, dim, device="cpu"):
        k = torch.zeros((3, heads, dim), dtype=torch.bfloat16, device=device)
        return ts.KvTokens(k, k, torch.zeros(3, dtype=torch.int64, device=device))

    def query(heads, dim, device="cpu"):
        q = torch.zeros((3, heads, dim), dtype=torch.bfloat16, device=device)
        i32 = {"dtype": torch.int32, "device": device}
        return ts.PagedQuery(q, torch.empty_like(q), torch.zeros((3, 2), **i32), torch.zeros(3, **i32))
    for call, make in ((ts.ts_kv_append, tokens), (ts.ts_paged_attention, query)):
        with pytest.raises(ts.SamplerError) as e:
            call(None, cache(4, 64), make(4, 64), _Stream)
        assert e.value.status == ts.TS_ERR_INVALID_ARG
        for other in (make(4, 128), make(4, 32), make(4, 64, "meta")):
            with pytest.raises(ValueError):
                call(None, cache(4, 64), other, _Stream)
    for heads in (2, 8):
        with pytest.raises(ValueError):
            ts.ts_kv_append(None, cache(4, 64), tokens(heads, 64), _Stream)


def test_key_masks_are_as_wide_as_the_tables():
    """A mask's columns count, not the stride of the rows that they are taken from."""
    import torch
    import codebook_token_sampling_gb300 as ts
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((2, 16, 4, 64), dtype=torch.bfloat16)
    cache = ts.KvCache(k, torch.zeros_like(k))
    i32 = {"dtype": torch.int32}
    wide = torch.ones((3, 1000), dtype=torch.uint8)

    def call(mask):
        ts.ts_paged_attention(None, cache, ts.PagedQuery(q, torch.empty_like(q), torch.zeros((3, 2), **i32),
                                                         torch.zeros(3, **i32), key_mask=mask), _Stream)
    for enough in (wide, wide[:, :32], wide[:, 7:39], None):
        with pytest.raises(ts.SamplerError):  # the NULL handle
            call(enough)
    for narrow in (wide[:, :31], wide[:, :10], wide[:, 999:]):
        with pytest.raises(ValueError):
            call(narrow)
