"""Caps far above the scores of a model, up to the largest accepted one, and
scores as far from 1 as such caps: scale / cap and its powers leave fp32's
normal range there, the scores do not."""

import numpy as np
import pytest

from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, torch

pytestmark = pytest.mark.gpu

# 1e30 and 2e38 are both so large that tanh(s / cap) * cap is s to the last bit
# of fp32 for every score below 1e20: two calls on the same inputs agree bit for
# bit where the kernels' order of sums is fixed
HUGE = (1e30, 2e38)


def _layer(duo, d, dtype, quant="none", ret=(0, 2), n=90):
    t = torch()
    sh = S.LayerShape(8, 4, d, dtype)
    lay = Layer(duo, sh, list(ret), 1, capacity=320, kv_quant={"none": duo.KV_PLAIN, "int8": duo.KV_INT8, "int4": duo.KV_INT4}[quant])
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    t.manual_seed(5)
    k, v = (t.randn(1, n, 4, d, device="cuda").to(dt) for _ in range(2))
    duo.append_kv(lay.desc, lay.caches.state, k, v, n)
    return lay, dt


@pytest.mark.parametrize("d,dtype,quant", [(64, "fp32", "none"), (128, "fp32", "none"), (64, "bf16", "none"), (128, "bf16", "none"),
                                           (128, "bf16", "int8"), (128, "bf16", "int4")])
def test_decode_under_a_huge_cap_is_the_plain_decode(duo, d, dtype, quant):
    t = torch()
    lay, dt = _layer(duo, d, dtype, quant)
    q = t.randn(1, 8, d, device="cuda").mul(4.0).to(dt)
    plain = t.empty_like(q)
    duo.decode_attn(lay.desc, lay.caches.state, q, plain, lay.ws.ptr, lay.ws.nbytes)
    for cap in HUGE:
        out = t.empty_like(q)
        duo.decode_attn_capped(lay.desc, lay.caches.state, cap, q, out, lay.ws.ptr, lay.ws.nbytes)
        # the same arithmetic, the keys dealt to splits and summed in another order at most: fp32 sums of 90 weights,
        # merged; where the weights are rounded to bf16 against another running maximum, two half-steps of them
        steps = 64 * 2.0 ** -24 if dtype == "fp32" else 3 * 2.0 ** -8
        assert np.abs(f64(out) - f64(plain)).max() <= steps * 4.5


@pytest.mark.parametrize("d,dtype,quant", [(64, "fp32", "none"), (128, "fp32", "none"), (64, "bf16", "none"), (128, "bf16", "none"),
                                           (128, "bf16", "int8")])
def test_prefill_under_huge_caps(duo, d, dtype, quant):
    t = torch()
    lay, dt = _layer(duo, d, dtype, quant)
    C = 200
    q, k, v = (t.randn(1, C, h, d, device="cuda").mul(s).to(dt) for h, s in ((8, 4.0), (4, 1.0), (4, 1.0)))
    ws = duo.Workspace(lay.desc, duo.OP_PREFILL, C, state=lay.caches.state)
    outs = []
    for cap in HUGE:
        outs.append(t.empty_like(q))
        duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, q, k, v, C, outs[-1], ws.ptr, ws.nbytes)
    assert np.array_equal(bits(outs[0]), bits(outs[1]))


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp32")])
def test_mix_step_under_huge_caps(duo, d, dtype):
    from tests.test_gpu_mix_train import _case, _step
    desc, *x = _case(duo, 8, 4, d, dtype, 1, 300, 0.0, 4.0)
    for a, b in zip(_step(duo, desc, HUGE[0], *x), _step(duo, desc, HUGE[1], *x)):
        assert np.array_equal(bits(a), bits(b))


# gain of q and of k, cap: scores near the cap, and far below it with products
# whose squares leave fp32
LARGE = [(2.0 ** 20, 1e12), (2.0 ** 30, 1e18), (2.0 ** 38, 1e26), (2.0 ** 10, 1e7)]


def _one_hot(q, k, cap):
    """Row by row the key of the largest capped score (causal), and whether it leads by 1e-4 of the cap or of itself, far
    more than any rounding of the scores."""
    s = q @ k.T * q.shape[-1] ** -0.5
    s = np.where(np.tril(np.ones(s.shape, bool)), cap * np.tanh(s / cap), -np.inf)
    two = np.sort(s, axis=1)[:, -2:]
    return s.argmax(1), two[:, 1] - two[:, 0] > 1e-4 * np.maximum(np.abs(two[:, 1]), np.abs(two[:, 0]))


@pytest.mark.parametrize("gain,cap", LARGE)
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp32")])
def test_scores_of_any_size(duo, d, dtype, gain, cap):
    """Scores so large that every softmax picks one key: the pre-fill and the training forward give that key's value."""
    t = torch()
    sh = S.LayerShape(4, 4, d, dtype)
    lay = Layer(duo, sh, [0, 1, 2, 3], 1, capacity=256)
    C, dt = 256, t.bfloat16 if dtype == "bf16" else t.float32
    t.manual_seed(3)
    q, k, v = (t.randn(1, C, 4, d, device="cuda").mul(s).to(dt) for s in (gain, gain, 1.0))
    out = t.empty_like(q)
    duo.prefill_chunk_capped(lay.desc, lay.caches.state, cap, q, k, v, C, out)
    al = t.ones(4, device="cuda")                       # the causal attention alone
    saved = t.empty(duo.gated_mix_saved_bytes(lay.desc, C), dtype=t.uint8, device="cuda")
    mixed, status = t.empty_like(q), t.zeros(1, dtype=t.int32, device="cuda")
    duo.gated_mix_train(lay.desc, al, cap, q, k, v, C, mixed, saved, saved.numel(), status)
    checked = 0
    for h in range(4):
        best, sure = _one_hot(f64(q)[0, :, h], f64(k)[0, :, h], cap)
        checked += int(sure.sum())
        want = f64(v)[0, best, h]
        for got in (out, mixed):
            got = f64(got)[0, :, h]
            assert np.all(np.isfinite(got))
            assert np.array_equal(got[sure], want[sure])
    assert checked > 256                                # not a test of nothing


@pytest.mark.parametrize("gain,cap", LARGE[1:3])
def test_gradients_of_scores_of_any_size_are_finite(duo, gain, cap):
    from tests.test_gpu_mix_train import _case, _step
    t = torch()
    desc, q, k, v, do, al = _case(duo, 4, 4, 128, "bf16", 1, 256, cap, 1.0)
    for x in _step(duo, desc, cap, q.mul(gain), k.mul(gain), v, do, al):
        assert bool(t.isfinite(x).all())
