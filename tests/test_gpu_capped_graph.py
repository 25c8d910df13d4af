"""A chunk's capped pre-fill with key splits, the rotated append and a capped
decode captured into one graph and replayed on new inputs, on a stream of the
caller's, beside the same calls made one by one."""

import numpy as np
import pytest

from head_split_kv_b200 import synthetic as S
from tests.gpu_helpers import Layer, bits, f64, torch

pytestmark = pytest.mark.gpu


# (an 8-bit cache's pre-fill takes V scales up to 4,095: no huge values there)
@pytest.mark.parametrize("quant,exponent", [("none", 0), ("none", 100), ("int8", 0)])
def test_captured_serving_step(duo, quant, exponent):
    """exponent 100: the pre-fill's values ask for the kernel's second pass, in the graph as outside it."""
    t = torch()
    sh = S.LayerShape(8, 2, 128, "bf16")
    n, C = 6400, 256
    kvq = duo.KV_PLAIN if quant == "none" else duo.KV_INT8
    one, two, warm = (Layer(duo, sh, [0], 1, capacity=n + 2 * C + 64, kv_quant=kvq) for _ in range(3))
    t.manual_seed(5)
    draw = lambda T: [t.randn(1, T, h, 128, device="cuda").mul(s).bfloat16() for h, s in ((8, 6.0), (2, 3.0), (2, 2.0 ** exponent))]  # noqa: E731
    _, k, v = draw(n)
    for lay in (one, two, warm):
        duo.append_kv(lay.desc, lay.caches.state, k, v, n)
    inv = t.linspace(1.0, 1e-3, 64, device="cuda")
    rope = duo.rope_init(128, inv)
    ws = [duo.Workspace(lay.desc, duo.OP_PREFILL, C, state=lay.caches.state) for lay in (one, two)]
    x = draw(C)
    outs = [[t.zeros(1, C, 8, 128, device="cuda", dtype=t.bfloat16) for _ in range(2)] + [t.zeros(1, 8, 128, device="cuda", dtype=t.bfloat16)]
            for _ in range(2)]

    def step(lay, w, out, stream=None):
        q, k, v = x
        st = lay.caches.state
        duo.prefill_chunk_capped(lay.desc, st, 20.0, q, k, v, C, out[0], w.ptr, w.nbytes, stream=stream)
        duo.append_kv_rope(lay.desc, st, rope, q, k, v, out[1], C, stream=stream)
        duo.decode_attn_capped(lay.desc, st, 20.0, out[1][:, -1], out[2], lay.ws.ptr, lay.ws.nbytes, stream=stream)

    step(warm, ws[1], outs[1])                                 # every kernel loaded before the capture
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        step(one, ws[0], outs[0])
    for _ in range(2):
        for a, b in zip(x, draw(C)):
            a.copy_(b)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        step(two, ws[1], outs[1])
        for i in (0, 1):
            assert np.all(np.isfinite(f64(outs[0][i]))) and np.array_equal(bits(outs[0][i]), bits(outs[1][i]))
        # decode deals its tiles to splits as they come: the weights' rounding, twice, and the store
        a, b = f64(outs[0][2]), f64(outs[1][2])
        assert np.abs(a - b).max() <= 6 * 2.0 ** -8 * np.abs(b).max() + 6 * 2.0 ** -8 * float(x[2].float().abs().max())
        for name in ("k_full", "v_full", "k_ring", "v_ring", "ring_pos", "seq_len"):
            assert np.array_equal(bits(getattr(one.caches, name)), bits(getattr(two.caches, name))), name
    assert one.status() == 0 and two.status() == 0
