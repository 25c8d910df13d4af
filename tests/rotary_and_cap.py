"""Plain fp64 forms of the rotary embedding and of capped attention, for the
tests of those operators, and the tolerances that go with them.

A rounding to a type is off by at most half a step: HALF[dtype] of the value.
"""

from __future__ import annotations

import math

import numpy as np

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def rope_ref(x, pos, inv_freq, rot, sections, layout, factor, sign=1.0):
    """x [B, T, H, d] fp64, pos [axes, B, T]: each channel pair as a complex
    number times factor * exp(i * angle)."""
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = sign * pos[axis].transpose(1, 2, 0).astype(np.float64) * np.asarray(inv_freq, dtype=np.float64)   # [B, T, rot/2]
    turn = factor * np.exp(1j * ang)[:, :, None]
    y = np.array(x, dtype=np.float64)
    if layout == "halves":
        z = (x[..., : rot // 2] + 1j * x[..., rot // 2: rot]) * turn
        y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
    else:
        z = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def rope_tolerance(x, rot, layout, factor, dtype):
    """Elementwise: the sine and cosine (fp32 of an angle reduced in fp64, and
    a multiply by the factor) are within 6 fp32 half-steps of 1, the two
    products and their sum add 3 more of the pair's size, and the store rounds
    once to dtype."""
    size = np.abs(np.array(x, dtype=np.float64))
    a, b = (size[..., : rot // 2], size[..., rot // 2: rot]) if layout == "halves" else (size[..., 0:rot:2], size[..., 1:rot:2])
    pair = (a + b) * abs(factor)
    tol = np.zeros_like(size)
    if layout == "halves":
        tol[..., : rot // 2] = tol[..., rot // 2: rot] = pair
    else:
        tol[..., 0:rot:2] = tol[..., 1:rot:2] = pair
    tol = tol * 9 * HALF["fp32"]
    rotated = np.zeros_like(size)
    rotated[..., :rot] = 1.0
    # half a step of the result, whose size is at most the pair's; channels that pass through are exact
    size_of_result = np.where(rotated > 0, tol / (9 * HALF["fp32"]), 0.0)
    return tol + HALF[dtype] * size_of_result


def capped(s, cap):
    return cap * np.tanh(s / cap) if cap else s


def attend_ref(q, k, v, seen, cap, scale):
    """q [n, d], k, v [m, d] fp64, seen [n, m] bool -> [n, d]; a row that sees nothing is 0."""
    s = np.where(seen, capped(q @ k.T * scale, cap), -np.inf)
    top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0)) * seen
    total = p.sum(1, keepdims=True)
    return (p / np.where(total > 0, total, 1.0)) @ v


def attend_tolerance(q, k, v, cap, scale, dtype):
    """How far an output may be from attend_ref on the same inputs, one number
    for a head: the weights' relative error, twice (numerator and row sum),
    and the store's rounding, each times the largest |v|.

    Weights, bf16: each is rounded to 8 bits (half a step, 2^-8 of the value at most
    of its binade's lower end) and computed from a score that is off by at most
    (d + 16) fp32 half-steps of its terms plus the cap's own 1e-6 * cap and
    8e-6 of the score; the exponential on the FMA pipe adds 7.5e-5.
    Weights, fp32: the score's error and four half-steps of cap; the sums over
    m keys add their error, (8 + sqrt(m)) half-steps of a convex combination."""
    if not len(k):
        return 0.0
    vmax, m, d = float(np.abs(v).max()), len(k), q.shape[1]
    terms = float((np.abs(q) @ np.abs(k).T * scale).max())
    score = (d + 16) * HALF["fp32"] * terms
    if dtype == "bf16":
        s = min(terms, cap) if cap else terms
        w = 2.0 ** -8 + score + 1e-6 * cap + 8e-6 * s + 7.5e-5
        return (2 * w + 2.0 ** -8) * vmax
    w = score + 4 * cap * HALF["fp32"] + 4 * HALF["fp32"]
    return (2 * w + 2 * (8 + math.sqrt(m)) * HALF["fp32"]) * vmax
