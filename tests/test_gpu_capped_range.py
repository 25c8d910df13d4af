"""Capped pre-fill and the capped training step where scores sit at +cap or
-cap and the values are far from 1: nothing overflows, nothing is flushed.

Every tolerance is relative to the values' size, so the same bounds hold for
values near 2^100 and near 2^-80."""

import numpy as np
import pytest

import oracle as O
from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, torch
from tests.rotary_and_cap import attend_ref, attend_tolerance, mix_ref

pytestmark = pytest.mark.gpu


def _rows(n, heads, signs, seed, size=4.0):
    """[1, n, heads, 128] rows along one direction, with signs [n], plus noise of size 1, in bf16.  Two such rows have a
    score of about +-180."""
    t = torch()
    u = t.randn(128, generator=t.Generator().manual_seed(1)).cuda()
    x = t.randn(1, n, heads, 128, generator=t.Generator().manual_seed(seed)).cuda()
    return (x + size * u * t.as_tensor(signs, dtype=t.float32).cuda()[None, :, None, None]).bfloat16()


def _values(n, heads, exponent, seed):
    t = torch()
    return t.randn(1, n, heads, 128, generator=t.Generator().manual_seed(seed)).cuda().mul(2.0 ** exponent).bfloat16()


@pytest.mark.parametrize("exponent", [0, 45, 100, 125, -60, -90])
@pytest.mark.parametrize("cap", [60.0, 50.0, 8.0])
def test_capped_prefill_of_saturated_scores(duo, cap, exponent):
    """Rows whose every score is near +cap, near -cap, and both, over the cache, the ring and the chunk."""
    t = torch()
    sh = S.LayerShape(8, 4, 128, "bf16")
    ret, chunks, scale = [0, 2], [300, 129], 128 ** -0.5
    lay = Layer(duo, sh, ret, 1, capacity=512)
    n = sum(chunks)
    q = _rows(n, 8, np.where(np.arange(n) % 3, 1.0, -1.0), 3)
    for pattern in (np.ones(n), np.where(np.arange(n) < 150, 1.0, -1.0)):   # every key alike; old keys against recent ones
        k, v = _rows(n, 4, pattern, 5), _values(n, 4, exponent, 6)
        for name in ("seq_len", "k_ring", "v_ring"):
            getattr(lay.caches, name).zero_()
        lay.caches.ring_pos.fill_(-1)
        ws = duo.Workspace(lay.desc, duo.OP_PREFILL, max(chunks), state=lay.caches.state)
        kk, vv, qq, c0 = f64(k)[0], f64(v)[0], f64(q)[0], 0
        for C in chunks:
            qc, kc, vc = (x[:, c0:c0 + C].contiguous() for x in (q, k, v))
            out = t.full_like(qc, float("nan"))
            duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, qc, kc, vc, C, out, ws.ptr, ws.nbytes)
            duo.append_kv(lay.desc, lay.caches.state, kc, vc, C)
            got, P, key = f64(out)[0], np.arange(c0, c0 + C)[:, None], np.arange(c0 + C)[None]
            for h in range(8):
                j = h // 2
                seen = key <= P if j in ret else (key <= P) & ((key < sh.sink) | (P - key < sh.recent))
                args = qq[c0:c0 + C, h], kk[:c0 + C, j], vv[:c0 + C, j]
                err = np.abs(got[:, h] - attend_ref(*args, seen, cap, scale))
                tol = attend_tolerance(*args, cap, scale, "bf16")
                assert np.all(err <= tol), f"c0={c0} h={h}: {err.max():.3e} > {tol:.3e}"
            c0 += C
    assert lay.status() == 0


@pytest.mark.parametrize("exponent", [0, 100, -80])
def test_key_splits_of_saturated_scores(duo, exponent):
    """A row's key ranges lie near +cap in some splits and near -cap in the others: one split may need lowered exponents
    and the next not, and the merge brings them together."""
    t = torch()
    sh = S.LayerShape(8, 2, 128, "bf16")
    lay = Layer(duo, sh, [0], 1, capacity=13000)
    n, C, cap, scale = 12800, 512, 60.0, 128 ** -0.5
    key = np.arange(n + C)
    for pattern in (np.where(key < 7000, -1.0, 1.0), np.where(key < 7000, 1.0, -1.0), -np.ones(n + C)):
        k, v = _rows(n + C, 2, pattern, 5), _values(n + C, 2, exponent, 6)
        q = _rows(C, 8, np.where(np.arange(C) % 3, 1.0, -1.0), 3)
        lay.caches.seq_len.zero_()
        duo.append_kv(lay.desc, lay.caches.state, k[:, :n].contiguous(), v[:, :n].contiguous(), n)
        ws = duo.Workspace(lay.desc, duo.OP_PREFILL, C, state=lay.caches.state)
        assert ws.nbytes > 256
        out = t.full_like(q, float("nan"))
        duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, q, k[:, n:].contiguous(), v[:, n:].contiguous(), C, out,
                                 ws.ptr, ws.nbytes)
        got, rows = f64(out)[0], np.array([0, 1, 2, 127, 128, 300, 301, 302, 511])
        kk, vv = f64(k)[0, :, 0], f64(v)[0, :, 0]
        seen = key[None] <= (n + rows)[:, None]
        for h in range(4):
            qq = f64(q)[0, rows, h]
            err = np.abs(got[rows, h] - attend_ref(qq, kk, vv, seen, cap, scale)).max()
            assert err <= attend_tolerance(qq, kk, vv, cap, scale, "bf16")
    assert lay.status() == 0


@pytest.mark.parametrize("exponent", [0, 60, -60])
@pytest.mark.parametrize("cap", [60.0, 20.0])
def test_mix_step_of_saturated_scores(duo, cap, exponent):
    """The causal attention of a row near +cap and its Lambda attention near -cap, and the other way round."""
    t = torch()
    N, hq, hkv = 400, 4, 2
    q, do = _rows(N, hq, np.where(np.arange(N) % 3, 1.0, -1.0), 3), _values(N, hq, 0, 4)
    k, v = _rows(N, hkv, np.where(np.arange(N) < 150, 1.0, -1.0), 5), _values(N, hkv, exponent, 6)
    al = t.tensor([0.25, 0.75], device="cuda")
    desc = duo.desc_init(1, hq, hkv, 128, duo.BF16, [0, 1], 2, sink=0, recent=64)
    saved = t.zeros(duo.gated_mix_saved_bytes(desc, N), dtype=t.uint8, device="cuda")
    ws = t.zeros(duo.gated_mix_grad_workspace_bytes(desc, N), dtype=t.uint8, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    got = [t.full_like(x, float("nan")) for x in (q, q, k, v, al)]
    duo.gated_mix_train(desc, al, cap, q, k, v, N, got[0], saved, saved.numel(), status)
    duo.gated_mix_grad(desc, al, cap, q, k, v, N, saved, saved.numel(), do, *got[1:], ws, ws.numel(), status)
    assert int(status) == 0
    want, tol = mix_ref(f64(q), f64(k), f64(v), f64(do), f64(al), cap, 0, 64, "bf16")
    for name, g, w, e in zip(("out", "dq", "dk", "dv", "dalpha"), got, want, tol):
        err = np.abs(f64(g) - w)
        assert np.all(err <= e), f"{name}: largest error {err.max():.3e}, excess {np.max(err - e):.3e}"


def test_a_second_pass_gives_the_same_weights(duo):
    """Values of ordinary size beside one column of huge ones: the ordinary columns agree with a call without it to the
    weights' rounding, and an infinite value reaches only the columns it stands in."""
    t = torch()
    sh = S.LayerShape(4, 4, 128, "bf16")
    lay = Layer(duo, sh, [0, 1, 2, 3], 1, capacity=256)
    C, cap = 200, 50.0
    q, k, v = _rows(C, 4, np.where(np.arange(C) % 3, 1.0, -1.0), 3), _rows(C, 4, np.ones(C), 5), _values(C, 4, 0, 6)
    outs = []
    for value in (None, 2.0 ** 120, float("inf")):
        w = v.clone()
        if value is not None:
            w[..., 77] = value
        out = t.empty_like(q)
        duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, q, k, w, C, out)
        outs.append(f64(out)[0])
        other = np.delete(outs[-1], 77, axis=-1)
        assert np.all(np.isfinite(other))
        # two sets of weights, each off by half a bf16 step and so is each row's sum, and two stores
        assert np.all(np.abs(other - np.delete(outs[0], 77, axis=-1)) <= 6 * 2.0 ** -8 * float(v.abs().max()))
    assert np.all(np.abs(outs[1][..., 77] / 2.0 ** 120 - 1.0) <= 2.0 ** -8)
    # a row past the diagonal's start has masked keys, whose weights of 0 meet the infinity
    assert not np.any(np.isfinite(outs[2][..., 77]))
    assert lay.status() == 0
