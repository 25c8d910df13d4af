"""duo_gated_mix_train and duo_gated_mix_grad within bounds that a wrong window,
cap, gate or D leaves (tests/test_mix_bounds.py shows which), over the forms
that each launch takes: one CTA or a pair to a key tile, gates inside and
outside [0, 1] with sink tiles and bands, with and without a cap, sequences of
many tiles; and the gradient along its own direction against differences."""

import numpy as np
import pytest

from tests.gpu_helpers import f64, torch
from tests.mix_bounds import SIGMAS, excess, mix_bounds
from tests.test_gpu_mix_train import _case, _step

pytestmark = pytest.mark.gpu

MIXED = [0.3, 1.5, -0.75, 0.0, 1.0, 0.9, 2.0, -0.1]          # by KV head, in turn

CASES = [   # hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha, KV heads looked at
    (4, 2, 128, "bf16", 1, 700, 30.0, 3.0, 16, 64, [0.3, 0.8], None),
    (4, 4, 128, "bf16", 2, 257, 0.0, 1.0, 16, 64, [0.1, 0.9, 0.5, 0.25], None),
    (4, 2, 128, "bf16", 1, 300, 200.0, 3.0, 16, 64, [0.3, 0.8], None),           # no bound from the cap
    (4, 2, 128, "bf16", 3, 200, 30.0, 3.0, 100, 28, [0.3, 0.8], None),
    (4, 4, 128, "bf16", 1, 500, 0.0, 1.0, 16, 64, [1.5, -0.75, 2.0, -0.1], None),     # signed shares, no cap
    (4, 4, 128, "bf16", 1, 500, 20.0, 3.0, 100, 28, [1.5, -0.75, 2.0, -0.1], None),   # sink tiles under signed shares
    (2, 1, 128, "bf16", 1, 2100, 50.0, 3.0, 16, 64, [0.4], None),                # pairs, seventeen key tiles
    (2, 2, 128, "bf16", 1, 1500, 0.0, 1.0, 16, 64, [0.4, 1.25], None),
    (40, 40, 128, "bf16", 1, 1000, 30.0, 3.0, 16, 64, MIXED * 5, [0, 1, 18, 39]),      # a CTA to a key tile, eight tiles
    (48, 48, 128, "bf16", 1, 900, 0.0, 1.0, 100, 28, MIXED * 6, [1, 2, 24]),
    (64, 16, 128, "bf16", 2, 900, 50.0, 3.0, 0, 128, MIXED * 2, [0, 9]),
    (4, 2, 128, "bf16", 1, 400, 30.0, 3.0, 130, 200, [0.3, 0.8], None),          # a window past a tile: CUDA cores
    (4, 2, 64, "bf16", 1, 600, 30.0, 3.0, 16, 64, [0.3, -0.5], None),
    (8, 4, 64, "fp32", 2, 201, 20.0, 3.0, 16, 64, [0.1, 0.8, -0.5, 2.0], None),
    (4, 1, 128, "fp32", 1, 700, 0.0, 1.0, 3, 7, [0.5], None),
    (32, 32, 64, "fp32", 1, 640, 20.0, 3.0, 16, 64, MIXED * 4, [0, 1, 31]),      # tiles of 64 rows
    (32, 32, 128, "fp32", 1, 640, 0.0, 1.0, 16, 300, MIXED * 4, [2, 8]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:10]))
def test_mix_step_within_independent_roundings(duo, case):
    hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha, heads = case
    desc, q, k, v, do, al = _case(duo, hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha)
    got = dict(zip(("out", "dq", "dk", "dv", "dalpha"), (f64(x) for x in _step(duo, desc, cap, q, k, v, do, al))))
    heads = list(range(hkv)) if heads is None else heads
    G = hq // hkv
    rows = [j * G + g for j in heads for g in range(G)]
    tc = dtype == "bf16" and d == 128 and sink + recent <= 128
    pick = {"out": rows, "dq": rows, "dk": heads, "dv": heads}
    want, bounds = mix_bounds(f64(q)[:, :, rows], f64(k)[:, :, heads], f64(v)[:, :, heads], f64(do)[:, :, rows], f64(al)[heads], cap,
                              sink, recent, dtype, tc)
    for n, w in want.items():
        g = got[n][:, :, pick[n]] if n in pick else got[n][heads]
        assert excess(n, g, w, bounds[n]) is None, excess(n, g, w, bounds[n])


SHORT = [   # sequences of one tile: dS keeps what its rounding takes off, so dq and dk are off by their own rounding alone
    (1, 1, 2, 0.0, 3.0, 16, 64, [0.5]),
    (8, 1, 3, 20.0, 3.0, 16, 64, [0.25]),
    (4, 4, 5, 50.0, 3.0, 0, 1, [0.1, 0.9, 0.5, 0.7]),
    (8, 2, 17, 0.0, 1.0, 2, 4, [0.3, 0.8]),
    (8, 2, 64, 30.0, 3.0, 2, 4, [1.5, -0.75]),
    (8, 4, 100, 0.0, 3.0, 16, 64, [0.0, 1.0, 2.0, -0.5]),
    (16, 2, 128, 20.0, 3.0, 100, 28, [0.4, 1.25]),
    (4, 2, 128, 200.0, 3.0, 16, 64, [0.4, 0.6]),
    (4, 2, 127, 1e20, 3.0, 16, 8, [0.4, -0.6]),
]


@pytest.mark.parametrize("case", SHORT, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_short_sequences_within_the_outputs_rounding(duo, case):
    hq, hkv, N, cap, gain, sink, recent, alpha = case
    desc, q, k, v, do, al = _case(duo, hq, hkv, 128, "bf16", 3, N, cap, gain, sink, recent, alpha)
    got = dict(zip(("out", "dq", "dk", "dv", "dalpha"), (f64(x) for x in _step(duo, desc, cap, q, k, v, do, al))))
    want, bounds = mix_bounds(f64(q), f64(k), f64(v), f64(do), f64(al), cap, sink, recent, "bf16", True)
    for n, w in want.items():
        assert excess(n, got[n], w, bounds[n]) is None, excess(n, got[n], w, bounds[n])


@pytest.mark.parametrize("d,cap,sink,recent", [(64, 7.0, 4, 8), (64, 0.0, 16, 64), (128, 20.0, 0, 1)])
def test_gradient_along_its_direction_against_differences(duo, d, cap, sink, recent):
    """fp32: L = <dout, out> moved by +-h along the whole gradient of one input.  The kernel's L against fp64's at the same
    two places (the moved tensors as the kernel got them): only the outputs' roundings lie between.  The kernel's gradient against fp64's quotients at h
    and h / 2, extrapolated: the h^2 term is gone, the h^4 term is measured by a third quotient."""
    t = torch()
    desc, *x = _case(duo, 4, 2, d, "fp32", 1, 150, cap, 2.0, sink, recent, [0.3, 0.8])
    q, k, v, do, al = x
    got = _step(duo, desc, cap, *x)
    base = [f64(y) for y in (q, k, v, al)]
    _, bounds = mix_bounds(*base[:3], f64(do), base[3], cap, sink, recent, "fp32", False)
    noise = SIGMAS * float(np.sqrt((f64(do) ** 2 * bounds["out"].sigma ** 2).sum())) + \
        float(np.sqrt((f64(do) ** 2 * bounds["out"].lin ** 2).sum())) * SIGMAS

    def loss64(which, dx):
        y = [b.copy() for b in base]
        y[which] = y[which] + dx
        return float((mix_bounds(*y[:3], f64(do), y[3], cap, sink, recent, "fp32", False)[0]["out"] * f64(do)).sum())

    for which in range(4):
        grad = f64(got[1 + which])
        size = float(np.sqrt((grad ** 2).sum()))
        u = grad / size
        quotients = []
        for h in (2.0 ** -6, 2.0 ** -7, 2.0 ** -8):
            quotients.append((loss64(which, h * u) - loss64(which, -h * u)) / (2 * h))
        first, second = ((4 * b - a) / 3 for a, b in zip(quotients, quotients[1:]))
        assert abs(size - second) <= 2 * abs(first - second) + 2e-5 * size, (which, size, second)
        h = 8.0 / size                               # so that L moves by about 16, whichever input moves it
        vals, moved = [], []
        for sign in (1.0, -1.0):
            y = [z.clone() for z in (q, k, v, al)]
            y[which] += (sign * h * t.from_numpy(u).cuda()).float()
            vals.append(float((f64(_step(duo, desc, cap, y[0], y[1], y[2], do, y[3])[0]) * f64(do)).sum()))
            moved.append(loss64(which, f64(y[which]) - base[which]))
        signal = abs(moved[0] - moved[1])
        assert 2 * noise <= 0.02 * signal, (which, noise, signal)
        assert abs((vals[0] - vals[1]) - (moved[0] - moved[1])) <= 2 * noise
