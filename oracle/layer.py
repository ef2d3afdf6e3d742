"""Plain 64-bit versions of the layer operators around the paged cache (numpy; tests
only).  They follow the definitions row by row and share no code with the library."""
from __future__ import annotations

import math

import numpy as np

from .kv import from_e4m3, to_e4m3

BLOCK = 128


def block_scales(y) -> np.ndarray:
    """The scale of each 128 elements of the rows y: the largest size, 2^-64 at least,
    over 448; NaN where an element is not finite."""
    rows, dim = y.shape
    out = np.zeros((rows, -(-dim // BLOCK)))
    for r in range(rows):
        for b in range(out.shape[1]):
            a = np.abs(y[r, b * BLOCK:(b + 1) * BLOCK])
            out[r, b] = max(a.max(), 2.0 ** -64) / 448 if np.all(np.isfinite(a)) else np.nan
    return out


def of_columns(scale, dim) -> np.ndarray:
    """Block scales as one per column."""
    return np.repeat(scale, BLOCK, axis=1)[:, :dim]


def quantised_f32(y):
    """Codes and scales of fp32 rows, each step rounded to fp32 as the rule says."""
    y = np.asarray(y, np.float32)
    rows, dim = y.shape
    scale = np.zeros((rows, -(-dim // BLOCK)), np.float32)
    for b in range(scale.shape[1]):
        a = np.abs(y[:, b * BLOCK:(b + 1) * BLOCK])
        top = np.maximum(np.where(np.isnan(a), np.inf, a).max(1), np.float32(2.0 ** -64))
        scale[:, b] = np.where(np.isfinite(top), top / np.float32(448), np.float32(np.nan))
    with np.errstate(invalid="ignore"):
        q = y * of_columns(np.float32(1) / scale, dim)
    assert q.dtype == np.float32
    return to_e4m3(q), scale


def rms_norm(x, weight, residual=None, *, eps, weight_offset=0.0):
    """The sum h and its norm times the weight."""
    h = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    y = np.zeros_like(h)
    with np.errstate(all="ignore"):
        for r in range(h.shape[0]):
            y[r] = h[r] / np.sqrt(np.mean(h[r] * h[r]) + eps)
    if weight is not None:
        y = y * (np.asarray(weight, np.float64) + weight_offset)
    return h, y


def activation(g, kind) -> np.ndarray:
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "silu":
            return g / (1 + np.exp(-g))
        if kind == "gelu":
            return g * 0.5 * np.vectorize(math.erfc, otypes=[float])(-g / math.sqrt(2))
        if kind == "gelu_tanh":
            return g * 0.5 * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return np.ones_like(g)


def linear(x, x_scale, w, w_scale):
    """The product of e4m3 codes with block scales, and the same of sizes (for bounds)."""
    x, w = from_e4m3(x), from_e4m3(w)
    m, k = x.shape
    out, size = np.zeros((m, w.shape[0])), np.zeros((m, w.shape[0]))
    of_row = np.arange(w.shape[0]) // BLOCK
    for b in range(-(-k // BLOCK)):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        factor = np.asarray(x_scale, np.float64)[:, b, None] * np.asarray(w_scale, np.float64)[of_row, b][None, :]
        out += factor * (x[:, cols] @ w[:, cols].T)
        size += np.abs(factor) * (np.abs(x[:, cols]) @ np.abs(w[:, cols]).T)
    return out, size


def rotary(x, positions, freqs, *, interleaved, amplitude=1.0) -> np.ndarray:
    """Heads [tokens, heads, dim] with their first pairs turned, one pair at a time."""
    y = np.array(x, np.float64)
    half = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(positions, np.float64) * f
        c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
        u, v = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = u * c - v * s, v * c + u * s
    return y
