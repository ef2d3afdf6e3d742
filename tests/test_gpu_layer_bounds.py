"""The layer operators against the bounds that the header states: activations over every
size of gate, rotary angles of every frequency and position."""
import fractions

import numpy as np
import pytest

from oracle import layer as olayer
from test_gpu_layer import close, get, put, sampler, ts  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of fp32, of the value


# --------------------------------------------------------------------------
# Activations
# --------------------------------------------------------------------------
def activation(g, act):
    """In 64 bits, without the difference 1 + tanh that leaves nothing of small results."""
    if act != "gelu_tanh":
        return olayer.activation(g, act)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def activation_bound(g, act, out_kind):
    """(relative, absolute) error of an fp32 activation times 1.

    silu: the exponent's parts are kept, but for what ln 2 rounded to fp32 (2^-29) makes of
    127 of them (4 steps of 2^-24); the exponential within 2^-22.5 (3 steps); a correction, a
    sum, a reciprocal (2 steps), two products and the factor's: 13 steps, 2^-20.  gelu: the
    rational function within 6.3 steps, its polynomials of positive terms three and four, the
    reciprocal and the product 3, the exponential as above 7, a correction, a product, the
    difference from max(g, 0) and the factor's: 28 steps, below 2^-19; where the result has
    fewer than 32 bits the exponent's parts are not kept: the square rounded, its product
    with log2(e) / 2 rounded and that constant, 2.2 steps of g g / 2.  gelu_tanh: as silu,
    and its argument z's three roundings and two constants', 5 |z| steps.  Exponentials
    below 2^-126 and reciprocals of sums above 2^126 count as zero."""
    g = np.abs(g)
    if act == "silu":
        return 2.0 ** -20, (g + 1) * 2.0 ** -126
    if act == "gelu":
        return 2.0 ** -19 + (1.1 * STEP * np.minimum(g, 14.0) ** 2 if out_kind != "f32" else 0.0), 2.0 ** -126
    z = np.minimum(2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3), 90.0)
    return 2.0 ** -20 + 5 * STEP * z, (g + 1) * 2.0 ** -126


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [5000, 4999])
def test_activations_are_right_relative_to_their_size(ts, sampler, act, kind, dim):
    """Gates from -120 to 120, and of every power of two: also where the result is small."""
    rng = np.random.default_rng(dim)
    near = np.linspace(-14, 14, 30 * dim)
    far = rng.choice([-1.0, 1.0], 10 * dim) * 2.0 ** rng.uniform(-126, 7, 10 * dim)
    gate = put(np.concatenate([near, far]).reshape(-1, dim), kind)
    out = put(np.zeros(gate.shape))
    ts.ts_gate(sampler.handle, ts.Gate(put(np.ones(gate.shape), kind), out, gate, activation=act))
    g = get(gate)
    want = activation(g, act)
    rel, absolute = activation_bound(g, act, "f32")
    close(get(out), want, rel * np.abs(want) + absolute, act)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_small_results_in_16_bits(ts, sampler, act):
    """A gate of -8 to -4 leaves little, and a large factor makes it count: half a step of
    the result's type, and the fp32 bound before it."""
    gate = put(np.linspace(-8, -4, 64 * 256).reshape(64, 256), "bf16")
    up = put(np.full((64, 256), 3.0e4), "bf16")
    out = put(np.zeros((64, 256)), "bf16")
    ts.ts_gate(sampler.handle, ts.Gate(up, out, gate, activation=act))
    g = get(gate)
    want = activation(g, act) * get(up)
    rel, absolute = activation_bound(g, act, "bf16")
    off = rel * np.abs(want) + absolute * get(up)
    close(get(out), want, off + 2.0 ** -9 * (np.abs(want) + off) * 2, act)


# --------------------------------------------------------------------------
# Rotary angles
# --------------------------------------------------------------------------
TWO_PI = fractions.Fraction("6.2831853071795864769252867665590057683943387987502116419498891846156328125724179972560696506842341359")


def cosines_and_sines(ts, sampler, positions, freqs):
    """cos and sin of every position and frequency as ts_rotary turns (1, 0) by them, and in
    64 bits by exact products and their rests modulo a turn."""
    import torch
    n = len(freqs)
    x = put(np.tile(np.r_[np.ones(n), np.zeros(n)], (len(positions), 1, 1)))
    ts.ts_rotary(sampler.handle, ts.Rotary(x, x, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                                           torch.tensor(freqs, dtype=torch.float64, device="cuda")))
    want = np.zeros((len(positions), 2 * n))
    for t, p in enumerate(positions):
        for i, f in enumerate(freqs):
            turn = fractions.Fraction(float(f)) * int(p) / TWO_PI
            angle = float((turn - round(turn)) * TWO_PI)
            want[t, i], want[t, n + i] = np.cos(angle), np.sin(angle)
    return get(x)[:, 0], want


FAR = [0, 1, 2, 2 ** 20 - 1, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1]


def test_rotary_angles_of_any_frequency(ts, sampler):
    """The angle within 2^-31 turns below 2^64 radians per position, cosine and sine within
    2^-22."""
    rng = np.random.default_rng(5)
    freqs = [1.0, -0.3, 0.0, 1e-9, 5e-324, 100.0, -12345.678, 1e6, 2.0 ** 40 + 0.3, 2.0 ** 63, -1.8e19, *(2.0 ** rng.uniform(-40, 64, 85))]
    got, want = cosines_and_sines(ts, sampler, FAR, freqs)
    close(got, want, 2 * np.pi * 2.0 ** -31 + 2.0 ** -22)


def test_rotary_angles_in_all_quarters(ts, sampler):
    """Angles all around the circle and right beside its eighths: what is left beside whole
    quarters rounded to 24 bits (an eighth of a turn: pi / 4 2^-25), one step of the functions
    below 1, and the angle's 2^-31 turns; 2^-23 in all."""
    turns = np.r_[np.linspace(-1, 1, 4001), (np.arange(-8, 9) / 8)[:, None].repeat(9, 1).ravel() + np.tile(np.arange(-4, 5), 17) * 2.0 ** -33]
    for first in range(0, len(turns), 512):  # a head holds 512
        got, want = cosines_and_sines(ts, sampler, [1], list(2 * np.pi * turns[first:first + 512]))
        close(got, want, 2 * np.pi * 2.0 ** -31 + np.pi / 4 * 2.0 ** -25 + 2.0 ** -24, first)
