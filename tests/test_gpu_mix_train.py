"""duo_gated_mix_train and duo_gated_mix_grad against the formulas in fp64 and
against difference quotients."""

import numpy as np
import pytest

from tests.gpu_helpers import bits, f64, torch
from tests.rotary_and_cap import HALF, mix_ref

pytestmark = pytest.mark.gpu


def _case(duo, hq, hkv, d, dtype, B, N, cap, gain, sink=16, recent=64, alpha=None, seed=1):
    t = torch()
    t.manual_seed(seed)
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    q, k, v, do = (t.randn(B, N, h, d, device="cuda").mul(s).to(dt) for h, s in ((hq, gain), (hkv, 1.0), (hkv, 1.0), (hq, 1.0)))
    al = t.rand(hkv, device="cuda") if alpha is None else t.tensor(alpha, device="cuda", dtype=t.float32)
    desc = duo.desc_init(B, hq, hkv, d, duo.BF16 if dtype == "bf16" else duo.FP32, list(range(hkv)), hkv, sink=sink, recent=recent)
    return desc, q, k, v, do, al


def _step(duo, desc, cap, q, k, v, do, al):
    t = torch()
    N = q.shape[1]
    saved = t.full((duo.gated_mix_saved_bytes(desc, N),), 255, dtype=t.uint8, device="cuda")
    ws = t.full((duo.gated_mix_grad_workspace_bytes(desc, N),), 255, dtype=t.uint8, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    nan = float("nan")
    out, dq, dk, dv, da = t.full_like(q, nan), t.full_like(q, nan), t.full_like(k, nan), t.full_like(v, nan), t.full_like(al, nan)
    duo.gated_mix_train(desc, al, cap, q, k, v, N, out, saved, saved.numel(), status)
    duo.gated_mix_grad(desc, al, cap, q, k, v, N, saved, saved.numel(), do, dq, dk, dv, da, ws, ws.numel(), status)
    assert int(status) == 0
    return out, dq, dk, dv, da


def _check(got, want, tol):
    for name, g, w, e in zip(("out", "dq", "dk", "dv", "dalpha"), got, want, tol):
        err = np.abs(f64(g) - w)
        assert np.all(np.isfinite(f64(g))), name
        assert np.all(err <= e), f"{name}: largest error {err.max():.3e}, excess {np.max(err - e):.3e}"


CASES = [   # hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha
    (8, 2, 128, "bf16", 1, 700, 30.0, 3.0, 16, 64, None),
    (4, 4, 128, "bf16", 2, 257, 0.0, 1.0, 16, 64, [0.0, 1.0, 0.5, 0.25]),
    (8, 1, 128, "bf16", 1, 384, 5.0, 10.0, 16, 64, None),             # scores far past the cap
    (2, 2, 128, "bf16", 1, 300, 20.0, 3.0, 0, 1, [1.5, -0.75]),       # gates outside [0, 1], the smallest window
    (4, 2, 128, "bf16", 1, 1, 30.0, 3.0, 16, 64, None),
    (4, 2, 128, "bf16", 1, 300, 200.0, 3.0, 16, 64, None),            # a cap too high for exponentials without a maximum
    (4, 2, 128, "bf16", 3, 129, 30.0, 3.0, 100, 28, None),
    (32, 32, 128, "bf16", 5, 129, 30.0, 3.0, 16, 64, None),           # enough key tiles for a CTA each
    (64, 32, 128, "bf16", 4, 190, 0.0, 1.0, 16, 64, None),
    (4, 4, 128, "bf16", 1, 200, 30.0, 3.0, 130, 200, None),           # a window the tensor-core kernels do not take
    (8, 4, 64, "bf16", 2, 130, 30.0, 3.0, 16, 64, None),
    (8, 4, 64, "fp32", 2, 201, 20.0, 3.0, 16, 64, [0.0, 1.0, -0.5, 2.0]),
    (4, 1, 128, "fp32", 1, 150, 0.0, 1.0, 3, 7, None),
    (2, 2, 64, "fp32", 1, 1, 20.0, 1.0, 16, 64, None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_mix_step_matches_the_formulas(duo, case):
    hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha = case
    desc, q, k, v, do, al = _case(duo, hq, hkv, d, dtype, B, N, cap, gain, sink, recent, alpha)
    got = _step(duo, desc, cap, q, k, v, do, al)
    want, tol = mix_ref(f64(q), f64(k), f64(v), f64(do), f64(al), cap, sink, recent, dtype)
    _check(got, want, tol)
    again = _step(duo, desc, cap, q, k, v, do, al)                     # no atomics: the same bits
    for g, h in zip(got, again):
        assert np.array_equal(bits(g), bits(h))


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp32")])
@pytest.mark.parametrize("cap", [0.0, 30.0, 200.0])
def test_gates_of_sequences_inside_the_window_have_no_gradient(duo, d, dtype, cap):
    """Up to sink + recent tokens both attentions are the same, bit for bit."""
    case = _case(duo, 8, 4, d, dtype, 2, 80, cap, 2.0)
    assert np.all(f64(_step(duo, case[0], cap, *case[1:])[4]) == 0.0)


def test_forward_equals_the_plain_mix(duo):
    """Without a cap the training forward computes what duo_gated_mix computes
    (the same kernels and tiles: the same bits)."""
    t = torch()
    desc, q, k, v, do, al = _case(duo, 8, 4, 128, "bf16", 2, 333, 0.0, 1.0)
    out = _step(duo, desc, 0.0, q, k, v, do, al)[0]
    plain, status = t.empty_like(q), t.zeros(1, dtype=t.int32, device="cuda")
    duo.gated_mix(desc, al, q, k, v, 333, plain, status)
    assert np.array_equal(bits(out), bits(plain))


def test_gradients_against_difference_quotients(duo):
    """fp32, d 64: (L(x + h) - L(x - h)) / 2h of L = <dout, out>, for one entry
    of each input.  The quotient's own error: the rounding of L's terms over h,
    and the third derivative's h^2 / 6 (bounded by the fp64 quotient)."""
    t = torch()
    desc, q, k, v, do, al = _case(duo, 4, 2, 64, "fp32", 1, 90, 7.0, 2.0, 4, 8, [0.3, 0.8])
    got = _step(duo, desc, 7.0, q, k, v, do, al)
    base = [f64(x) for x in (q, k, v)] + [f64(al)]
    for which, at in ((0, (0, 77, 3, 5)), (1, (0, 40, 1, 9)), (2, (0, 2, 0, 63)), (3, (1,))):
        h, vals, loss64 = 2.0 ** -6, [], []
        for sign in (1, -1):
            x = [y.clone() for y in (q, k, v, al)]
            x[which][at] += sign * h
            out = _step(duo, desc, 7.0, x[0], x[1], x[2], do, x[3])[0]
            vals.append(float((f64(out) * f64(do)).sum()))
            y = [b.copy() for b in base]
            y[which][at] += sign * h
            loss64.append(float((mix_ref(y[0], y[1], y[2], f64(do), y[3], 7.0, 4, 8, "fp32")[0][0] * f64(do)).sum()))
        quotient, exact = (vals[0] - vals[1]) / (2 * h), (loss64[0] - loss64[1]) / (2 * h)
        grad = float(f64(got[1 + which])[at])
        terms = float(np.abs(f64(do)).sum()) * float(np.abs(base[2]).max())
        assert abs(quotient - exact) <= 64 * HALF["fp32"] * terms / h
        assert abs(grad - exact) <= h * h * 50 + 1e-5 * abs(exact)


def test_mix_step_captured_and_replayed_on_new_inputs(duo):
    """Both passes in one graph, replayed after the inputs were overwritten,
    while an eager step of the same tensors runs beside it."""
    t = torch()
    desc, q, k, v, do, al = _case(duo, 8, 4, 128, "bf16", 1, 300, 30.0, 3.0)
    N = 300
    saved = t.empty(duo.gated_mix_saved_bytes(desc, N), dtype=t.uint8, device="cuda")
    ws = t.empty(duo.gated_mix_grad_workspace_bytes(desc, N), dtype=t.uint8, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    out, dq, dk, dv, da = t.empty_like(q), t.empty_like(q), t.empty_like(k), t.empty_like(v), t.empty_like(al)
    _step(duo, desc, 30.0, q, k, v, do, al)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        duo.gated_mix_train(desc, al, 30.0, q, k, v, N, out, saved, saved.numel(), status)
        duo.gated_mix_grad(desc, al, 30.0, q, k, v, N, saved, saved.numel(), do, dq, dk, dv, da, ws, ws.numel(), status)
    new = _case(duo, 8, 4, 128, "bf16", 1, N, 30.0, 3.0, seed=9)[1:]
    for x, y in zip((q, k, v, do, al), new):
        x.copy_(y)
    graph.replay()
    eager = _step(duo, desc, 30.0, q, k, v, do, al)
    t.cuda.synchronize()
    for a, b in zip((out, dq, dk, dv, da), eager):
        assert np.array_equal(bits(a), bits(b))


def test_mix_step_of_no_tokens(duo):
    t = torch()
    desc, q, k, v, do, al = _case(duo, 4, 2, 128, "bf16", 1, 4, 30.0, 1.0)
    buf, status = t.empty(256, dtype=t.uint8, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
    out, dq, dk, dv, da = t.full_like(q, 7.0), t.full_like(q, 7.0), t.full_like(k, 7.0), t.full_like(k, 7.0), t.full_like(al, 7.0)
    duo.gated_mix_train(desc, al, 30.0, q, k, v, 0, out, buf, 0, status)
    duo.gated_mix_grad(desc, al, 30.0, q, k, v, 0, buf, 0, do, dq, dk, dv, da, buf, 0, status)
    assert all(bool((x == 7.0).all()) for x in (out, dq, dk, dv)) and not bool(da.any())


def test_rotary_training_step(duo):
    """rope -> gated mix -> loss <dout, out>, and back: dq and dk through the
    inverse rotation, against fp64 of the whole chain."""
    t = torch()
    B, N, hq, hkv, d, cap = 1, 200, 4, 2, 64, 10.0
    desc, q, k, v, do, al = _case(duo, hq, hkv, d, "fp32", B, N, cap, 2.0)
    inv = t.from_numpy(np.power(10000.0, -2.0 * np.arange(d // 2) / d).astype(np.float32)).cuda()
    rope = duo.rope_init(d, inv)
    qr, kr = t.empty_like(q), t.empty_like(k)
    duo.rope_qk(desc, rope, q, k, qr, kr, N)
    out, dqr, dkr, dv, da = _step(duo, desc, cap, qr, kr, v, do, al)
    dq, dk = t.empty_like(q), t.empty_like(k)
    duo.rope_qk(desc, rope, dqr, dkr, dq, dk, N, inverse=True)
    from tests.rotary_and_cap import rope_ref
    pos = np.arange(N)[None, None].repeat(B, 1)
    args = (bits(inv), d, [d // 2], "halves", 1.0)
    qr64, kr64 = rope_ref(f64(q), pos, *args), rope_ref(f64(k), pos, *args)
    want, tol = mix_ref(qr64, kr64, f64(v), f64(do), f64(al), cap, 16, 64, "fp32")
    want, tol = list(want), list(tol)
    for i in (1, 2):
        want[i] = rope_ref(want[i], pos, *args, sign=-1.0)
        # the rotated inputs' own rounding moves the gradient by its rate times 12 half-steps: 8 times the kernel's bound covers it
        tol[i] = 8 * np.maximum(tol[i], np.concatenate([tol[i][..., d // 2:], tol[i][..., : d // 2]], -1)) + 12 * HALF["fp32"]
    tol[0], tol[3], tol[4] = 8 * tol[0], 8 * tol[3], 8 * tol[4]
    _check((out, dq, dk, dv, da), want, tol)
