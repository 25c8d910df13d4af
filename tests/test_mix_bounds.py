"""The bounds of tests/mix_bounds.py tell a right training step from a wrong
one: wrong results in fp64, without any rounding, leave them."""

import numpy as np
import pytest
import torch

from tests.mix_bounds import excess, mix_bounds

CASES = [   # hq, hkv, d, dtype, N, cap, gain, sink, recent, alpha
    (4, 2, 128, "bf16", 400, 30.0, 3.0, 16, 64, [0.3, 0.8]),
    (4, 2, 128, "bf16", 300, 0.0, 1.0, 16, 64, [0.4, 0.6]),
    (2, 2, 128, "bf16", 300, 20.0, 3.0, 0, 1, [1.5, -0.75]),
    (4, 2, 128, "bf16", 300, 30.0, 3.0, 100, 28, [0.5, 0.2]),
    (4, 2, 64, "bf16", 200, 30.0, 3.0, 16, 64, [0.3, 0.9]),
    (4, 2, 64, "fp32", 201, 20.0, 3.0, 16, 64, [0.3, 2.0]),
    (2, 1, 128, "fp32", 150, 0.0, 1.0, 3, 7, [0.5]),
]


def _inputs(case, seed=1):
    hq, hkv, d, dtype, N, cap, gain, sink, recent, alpha = case
    torch.manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = [torch.randn(1, N, h, d).mul(s).to(dt).double().numpy() for h, s in ((hq, gain), (hkv, 1.0), (hkv, 1.0), (hq, 1.0))]
    return x, np.asarray(alpha, dtype=np.float64), dtype == "bf16" and d == 128


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_bounds_are_far_below_the_results(case):
    x, al, tc = _inputs(case)
    res, bounds = mix_bounds(*x, al, case[5], case[7], case[8], case[3], tc)
    for n, r in res.items():
        rms = np.sqrt((r ** 2).mean())
        tol = np.median(6 * bounds[n].sigma + bounds[n].lin)
        assert tol <= (0.12 if tc else 0.05) * rms, (n, tol / rms)
    assert float(np.max(6 * bounds["dalpha"].sigma + bounds["dalpha"].lin)) <= 0.05 * float(np.abs(res["dalpha"]).max())


MUTATIONS = {
    "a window one token wider": dict(recent=1),
    "a sink token more": dict(sink=1),
    "a cap 5 % too large": dict(cap=1.05),
    "halved gates": dict(alpha=0.5),
    "D from attentions rounded to bf16": dict(stored_d=True),
}


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
@pytest.mark.parametrize("what", MUTATIONS)
def test_a_wrong_step_leaves_the_bounds(case, what):
    hq, hkv, d, dtype, N, cap, gain, sink, recent, alpha = case
    x, al, tc = _inputs(case)
    want, bounds = mix_bounds(*x, al, cap, sink, recent, dtype, tc)
    m = MUTATIONS[what]
    if "cap" in m and not cap:
        pytest.skip("no cap in this case")
    wrong, _ = mix_bounds(*x, al * m.get("alpha", 1.0), cap * m.get("cap", 1.0), sink + m.get("sink", 0), recent + m.get("recent", 0),
                          dtype, tc, stored_d=m.get("stored_d", False))
    left = [n for n in want if excess(n, wrong[n], want[n], bounds[n])]
    if "stored_d" in m:
        assert {"dq", "dk"} & set(left), left
    else:
        assert {"dq", "dk"} <= set(left) and "dalpha" in left or "alpha" in m and {"out", "dv", "dq", "dk"} <= set(left), left


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_zeros_and_wrong_signs_leave_the_bounds(case):
    x, al, tc = _inputs(case)
    want, bounds = mix_bounds(*x, al, case[5], case[7], case[8], case[3], tc)
    for n, r in want.items():
        assert excess(n, r, r, bounds[n]) is None
        for wrong in (np.zeros_like(r), -r, r * 1.05):
            assert excess(n, wrong, r, bounds[n]), n
