"""Plain 64-bit versions of the paged cache's operators (numpy; tests only).

They follow the definitions one request, one token and one block at a time and
share no code with the library."""
from __future__ import annotations

import numpy as np

BAD_SHAPE, BAD_SLOT, BAD_BLOCK, NO_BLOCKS = 1, 8, 32, 64


def e4m3_values() -> np.ndarray:
    """The 127 non-negative finite e4m3 values by code: 4 exponent bits with a
    bias of 7, 3 mantissa bits, subnormals at exponent 0."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def to_e4m3(x) -> np.ndarray:
    """The codes of fp32 values rounded to the nearest e4m3 value, ties to the
    even code, sizes beyond 448 to 448, NaN to code 0x7F."""
    x = np.asarray(x, np.float64)
    values = e4m3_values()
    size = np.minimum(np.abs(x), 448.0)
    size = np.where(np.isnan(x), 0.0, size)
    hi = np.clip(np.searchsorted(values, size), 1, 126)
    lo = hi - 1
    dlo, dhi = size - values[lo], values[hi] - size
    code = np.where((dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def from_e4m3(code) -> np.ndarray:
    code = np.asarray(code, np.uint8)
    mag = code & 0x7F
    v = np.append(e4m3_values(), np.nan)[mag]
    return np.where(code & 0x80, -v, v)


def tables(block_table, lens, n_new, finished, free_blocks, n_free, *, block_size, n_blocks,
           max_tokens) -> dict:
    """The state after ts_kv_tables and its maps; inputs are not changed."""
    table, stack = np.array(block_table), np.array(free_blocks)
    n, wide = table.shape
    n_new = [1] * n if n_new is None else [int(a) for a in n_new]
    finished = [0] * n if finished is None else [int(f) for f in finished]
    status = 0

    def blocks(x):
        return -(-x // block_size)

    top = int(n_free)
    if not 0 <= top <= stack.size:
        status |= BAD_SHAPE
        top = min(max(top, 0), stack.size)
    bad = []
    for i in range(n):
        length = int(lens[i])
        off = length < 0 or length > wide * block_size
        off = off or (not finished[i] and (n_new[i] < 0 or length + n_new[i] > wide * block_size))
        bad.append(off)
        if off:
            status |= BAD_SHAPE
        elif finished[i]:
            for b in range(blocks(length)):
                if top == stack.size:
                    status |= BAD_SHAPE
                else:
                    stack[top] = table[i, b]
                    top += 1
    held_top, needs, asked, used = top, 0, 0, 0
    lens_out, starts, slots, positions, requests = [], [0], [], [], []
    for i in range(n):
        length = int(lens[i])
        if bad[i] or finished[i]:
            lens_out.append(length if bad[i] else 0)
            starts.append(len(slots))
            continue
        a = n_new[i]
        need = blocks(length + a) - blocks(length)
        needs += need
        asked += a
        if a > 0 and ((need > 0 and needs > held_top) or asked > max_tokens):
            status |= NO_BLOCKS
            a = need = 0
        for j in range(need):
            used += 1
            table[i, blocks(length) + j] = stack[held_top - used]
        for t in range(length, length + a):
            b = int(table[i, t // block_size])
            if 0 <= b < n_blocks:
                slots.append(b * block_size + t % block_size)
            else:
                status |= BAD_BLOCK
                slots.append(-1)
            positions.append(t)
            requests.append(i)
        starts.append(len(slots))
        lens_out.append(length + a)
    fill = [-1] * (max_tokens - len(slots))
    return {"block_table": table, "free_blocks": stack, "n_free": held_top - used,
            "lens": np.array(lens_out, np.int64), "token_starts": np.array(starts),
            "slots": np.array(slots + fill, np.int64), "positions": np.array(positions + fill),
            "requests": np.array(requests + fill), "status": status}


def attention(q, k, v, block_table, lens, *, scale, n_blocks, window=0, softcap=0.0, key_mask=None,
              k_scale=None, v_scale=None) -> dict:
    """Outputs, lse and, per output, what an error bound needs: ``abs_v`` (the
    weighted mean of |v|), ``dot`` (the largest sum of |q k| scale over the keys),
    ``keys`` and ``max_v``.  q [n, heads, dim], k and v [block, token, head, dim]."""
    n, heads, dim = q.shape
    bs, kv_heads = k.shape[1], k.shape[2]
    group = heads // kv_heads
    out, abs_v = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse, dot = np.full((n, heads), -np.inf), np.zeros((n, heads))
    keys, max_v = np.zeros(n), np.zeros((n, heads))
    status = 0
    for r in range(n):
        length = int(lens[r])
        if not 0 <= length <= block_table.shape[1] * bs:
            status |= BAD_SHAPE
            out[r], lse[r] = np.nan, np.nan
            continue
        t = np.arange(length)
        if window:
            t = t[t >= length - window]
        if key_mask is not None:
            t = t[np.asarray(key_mask[r])[t] != 0]
        keys[r] = t.size
        if not t.size:
            continue
        b = np.asarray(block_table[r], np.int64)[t // bs]
        if np.any((b < 0) | (b >= n_blocks)):
            status |= BAD_BLOCK
            out[r], lse[r] = np.nan, np.nan
            continue
        for g in range(kv_heads):
            kk, vv = k[b, t % bs, g].astype(np.float64), v[b, t % bs, g].astype(np.float64)
            if k_scale is not None:
                kk = kk * float(k_scale[g])
            if v_scale is not None:
                vv = vv * float(v_scale[g])
            for h in range(g * group, (g + 1) * group):
                with np.errstate(invalid="ignore", over="ignore"):
                    qh = q[r, h].astype(np.float64)
                    s = kk @ qh * scale
                    dot[r, h] = np.max(np.abs(kk) @ np.abs(qh)) * abs(scale)
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    m = np.max(s)
                    if m == -np.inf:
                        continue
                    p = np.exp(s - m)
                    out[r, h] = p @ vv / p.sum()
                    abs_v[r, h] = p @ np.abs(vv) / p.sum()
                    lse[r, h] = m + np.log(p.sum())
                    max_v[r, h] = np.max(np.abs(vv))
    return {"out": out, "lse": lse, "abs_v": abs_v, "dot": dot, "keys": keys, "max_v": max_v,
            "status": status}
